"""The pre-norm MLP block of the examples against the same chain with the norm and
the activation as plain fp32 torch operations around the same linears."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _plain(mx, ex, x, r, dout, ds, p, fmt, values):
    """The chain with plain norm and activation; the backward pass reads the same
    8-bit values (`values`: s, gate, up as the checkpoints restore them)."""
    s = (x.float() + r.float()).bfloat16()
    sf = s.float()
    mean = sf.mean(1, keepdim=True)
    rstd = torch.rsqrt(((sf - mean) ** 2).mean(1, keepdim=True) + 1e-5)
    n = ((sf - mean) * rstd * p["norm"] + p["bias"]).bfloat16()
    gu, kept_gu = mx.linear_fwd_save(n, p["gate_up"], fmt)
    F = gu.shape[1] // 2
    h = (torch.nn.functional.silu(gu[:, :F].float()) * gu[:, F:].float()).bfloat16()
    out, kept_d = mx.linear_fwd_save(h, p["down"], fmt)
    dh, d_down = mx.linear_bwd_saved(dout, kept_d, F, fmt)
    gate, up = values["gate"].clone().requires_grad_(), values["up"].clone().requires_grad_()
    (torch.nn.functional.silu(gate) * up).backward(dh.float())
    dgu = torch.cat([gate.grad, up.grad], 1).bfloat16()
    dn, d_gate_up = mx.linear_bwd_saved(dgu, kept_gu, x.shape[1], fmt)
    xh = (values["s"] - mean) * rstd
    g = dn.float() * p["norm"]
    dx = ((g - xh * (g * xh).mean(1, keepdim=True) - g.mean(1, keepdim=True)) * rstd + ds.float()).bfloat16()
    return out, s, dx, {"norm": (dn.float() * xh).sum(0), "bias": dn.float().sum(0), "gate_up": d_gate_up, "down": d_down}


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4", "moss"])
def test_block_equals_the_chain_with_plain_norm_and_activation(fmt):
    """bf16 roundings of n and h may differ in single last places (fp32 sums in
    another order); each such difference can move a code of the quantization that
    follows to its neighbour, 2^-3 of a value at most, in fewer than one of 2^7
    elements: a relative error of the products below 2^-3 2^-3.5 = 0.011."""
    import fp4_precision_gemms_gb300 as mx
    import norm_mlp_step as ex

    mx.build()
    T, H, F = 512, 1024, 1536
    g = torch.Generator(device="cuda").manual_seed(5)
    x, r, dout, ds = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(4))
    p = ex.weights(H, F)
    out, s, kept = ex.forward(x, r, p, fmt)
    dx, grads = ex.backward(dout, ds, kept, p, fmt)
    values = {k: mx.act8_restore(kept[k], out_dtype=torch.float32) for k in ("s", "gate", "up")}
    out2, s2, dx2, grads2 = _plain(mx, ex, x, r, dout, ds, p, fmt, values)
    torch.cuda.synchronize()
    assert mx.last_device_status() == mx.MX_OK
    assert torch.equal(s, s2)
    pairs = [("out", out, out2), ("dx", dx, dx2)] + [(k, grads[k], grads2[k]) for k in grads2]
    for name, a, b in pairs:
        assert torch.isfinite(a).all(), name
        rel = (a.double() - b.double()).norm() / b.double().norm()
        assert rel <= 0.011, (name, rel.item())


def test_the_checkpoints_cost_little():
    """The gradients from the 8-bit checkpoints stay near those of the kept inputs:
    a code's relative error is 2^-4 at most, about 2^-5.5 in the mean square."""
    import fp4_precision_gemms_gb300 as mx

    mx.build()
    g = torch.Generator(device="cuda").manual_seed(6)
    s, dy = (torch.randn(512, 2048, generator=g, device="cuda").bfloat16() for _ in range(2))
    f = mx.norm_fwd(s, save=True)
    for a, b in zip(mx.norm_bwd(dy, f.saved, f.rstd, f.mean), mx.norm_bwd(dy, s, f.rstd, f.mean)):
        assert (a.double() - b.double()).norm() <= 2.0 ** -4 * b.double().norm()
    gate, up, dh = s[:, :1024], s[:, 1024:], dy[:, :1024]
    r = mx.act_fwd(gate, up, save=True)
    for a, b in zip(mx.act_bwd(dh, r.gate, r.up), mx.act_bwd(dh, gate, up)):
        assert (a.double() - b.double()).norm() <= 2.0 ** -4 * b.double().norm()
