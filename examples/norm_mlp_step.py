"""A training step of a pre-norm MLP block with every activation that its backward
pass needs held in 8 bits.

    s   = x + residual                      norm_fwd: one pass gives s, the norm, its
    n   = norm(s)                           maximum and the 8-bit checkpoint of s
    gu  = n W_gu^T                          linear_fwd_save (keeps n^T quantized)
    h   = silu(gu[:, :F]) * gu[:, F:]       act_fwd: h, its maximum, checkpoints of both
    out = h W_d^T                           linear_fwd_save; the block's output beside s

The maxima go to the linears as the tensor amax of their quantization (nvfp4, moss),
which then needs no pass of its own.  Backward, from dout and the gradient ds that
reaches s from the following layers:

    dh, dW_d     linear_bwd_saved
    dgu          act_bwd, from the checkpoints (one tensor, with its maximum)
    dn, dW_gu    linear_bwd_saved
    ds, dw, db   norm_bwd, from the checkpoint, joined with ds

    python examples/norm_mlp_step.py --tokens 8192 --hidden 4096 --ffn 14336 --fmt nvfp4
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp4_precision_gemms_gb300 as mx  # noqa: E402

AMAX_FORMATS = ("nvfp4", "moss")  # formats with a tensor scale


def weights(hidden: int, ffn: int, seed: int = 0, device="cuda") -> dict:
    g = torch.Generator(device=device).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    return {"norm": 1 + 0.1 * n(hidden), "bias": 0.1 * n(hidden),
            "gate_up": (0.02 * n(2 * ffn, hidden)).bfloat16(), "down": (0.02 * n(hidden, ffn)).bfloat16()}


def forward(x, residual, p, fmt):
    """(out, s, what the backward pass takes)."""
    word = lambda: torch.empty(1, dtype=torch.float32, device=x.device) if fmt in AMAX_FORMATS else None  # noqa: E731
    n_max, h_max = word(), word()
    norm = mx.norm_fwd(x, p["norm"], p["bias"], residual=residual, save=True, amax_out=n_max)
    gu, kept_gu = mx.linear_fwd_save(norm.y, p["gate_up"], fmt, x_amax=n_max)
    F = gu.shape[1] // 2
    act = mx.act_fwd(gu[:, :F], gu[:, F:], act="silu", save=True, amax_out=h_max)
    out, kept_d = mx.linear_fwd_save(act.h, p["down"], fmt, x_amax=h_max)
    return out, norm.sum, {"s": norm.saved, "mean": norm.mean, "rstd": norm.rstd, "gate": act.gate, "up": act.up,
                           "gate_up": kept_gu, "down": kept_d, "ffn": F, "hidden": x.shape[1]}


def backward(dout, ds, kept, p, fmt):
    """(gradient of s, {weight gradients})."""
    gu_max = torch.empty(1, dtype=torch.float32, device=dout.device) if fmt in AMAX_FORMATS else None
    dh, d_down = mx.linear_bwd_saved(dout, kept["down"], kept["ffn"], fmt)
    dgate, dup = mx.act_bwd(dh, kept["gate"], kept["up"], act="silu", amax_out=gu_max)
    dgu = dgate.as_strided((dgate.shape[0], 2 * dgate.shape[1]), (dgate.stride(0), 1))  # dgate and dup side by side
    assert dup.data_ptr() == dgate.data_ptr() + dgate.shape[1] * dgate.element_size()
    dn, d_gate_up = mx.linear_bwd_saved(dgu, kept["gate_up"], kept["hidden"], fmt, dy_amax=gu_max)
    dx, dw, db = mx.norm_bwd(dn, kept["s"], kept["rstd"], kept["mean"], p["norm"], dres=ds)
    return dx, {"norm": dw, "bias": db, "gate_up": d_gate_up, "down": d_down}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=14336)
    ap.add_argument("--fmt", default="nvfp4", choices=sorted(AMAX_FORMATS + ("mxfp8", "mxfp4")))
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    mx.build()
    p = weights(a.hidden, a.ffn)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, dout, ds = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16() for _ in range(4))
    dout, ds = dout * 1e-3, ds * 1e-3

    def step():
        out, s, kept = forward(x, r, p, a.fmt)
        return out, s, kept, backward(dout, ds, kept, p, a.fmt)

    for _ in range(3):
        _, _, kept, _ = step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        step()
    end.record()
    torch.cuda.synchronize()
    eight = sum(t.codes.numel() + t.sf.numel() for t in (kept["s"], kept["gate"], kept["up"]))
    print(f"{a.fmt}: {start.elapsed_time(end) / a.steps:.3f} ms per step; the norm's and the activation's inputs kept in "
          f"{eight / 2 ** 20:.1f} MiB (bf16: {(a.tokens * (a.hidden + 2 * a.ffn) * 2) / 2 ** 20:.1f} MiB)")
    if mx.last_device_status() != mx.MX_OK:
        raise SystemExit("device status word set")


if __name__ == "__main__":
    main()
