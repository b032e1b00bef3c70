"""The gated feed-forward block: h, the checkpoints and the gradients against the library's
own product in fp32 (which sums in the same order, so that g and u are the same numbers),
against 64-bit products of the dequantized operands, and against the calls it is made of."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

FORMATS = ("mxfp8", "mxfp4", "nvfp4", "moss", "nvfp4_local")
ACTS = ("silu", "gelu", "gelu_tanh")
BF, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    yield m
    assert m.last_device_status() == m.MX_OK


def data(T, K, F, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (n(T, K) * scale).to(BF), (n(2 * F, K) / math.sqrt(K)).to(BF)


def activation(z, act):
    z = z.double()
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def products(mx, x, gate, up):
    """g and u in fp32 by the plain GEMM, on the same kernel structure."""
    mx.set_gemm_variant("pair_ws")
    try:
        return mx.gemm(x, gate), mx.gemm(x, up)
    finally:
        mx.set_gemm_variant("auto")


def values(mx, q):
    """float64 values of an operand.  mx_dequantize takes one tensor scale: one by region is put on by rows."""
    if q.fmt != "nvfp4_local":
        return mx.dequantize(q).double()
    plain = mx.MXTensor("nvfp4", q.rows, q.k)
    plain.codes, plain.sf = q.codes, q.sf
    plain.scalars.fill_(1.0)
    return mx.dequantize(plain).double() * q.tensor_scale.double().repeat_interleave(128)[:q.rows, None]


SHAPES = [(1, 256, 32), (1, 512, 128), (2, 256, 8), (33, 256, 40), (64, 1024, 136), (130, 768, 200), (257, 512, 384), (300, 1280, 96),
          (700, 256, 20), (70, 256, 21), (40, 256, 131), (300, 512, 320), (129, 256, 64)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,F", SHAPES)
def test_h_and_checkpoints(mx, fmt, T, K, F):
    act = ACTS[(T + F) % 3]
    X, W = data(T, K, F)
    gate, up = mx.gated_weights(W, fmt)
    x = mx.quantize(X, fmt)
    top = torch.empty(1, device="cuda")
    h, g8, u8 = mx.gemm_gated(x, gate, up, act=act, save=True, amax_out=top)
    if F % 8 == 0:  # the plain product's own alignment rule
        g, u = products(mx, x, gate, up)
        for got, want in ((g8, mx.act8_save(g)), (u8, mx.act8_save(u))):
            assert torch.equal(got.codes, want.codes) and torch.equal(got.sf, want.sf)
        want = activation(g, act) * u.double()
        # half a step of bf16, and 2^-16 of the value for the approximate exponential
        assert ((h.double() - want).abs() <= (HALF + 2.0 ** -16) * want.abs() + 1e-37).all()
    # the same in 64 bits from the operands' values: K products and sums of 2^-23 of their size each
    a, b, c = (values(mx, q) for q in (x, gate, up))
    g, u = a @ b.T, a @ c.T
    eg, eu = ((a.abs() @ w.abs().T) * (K * 2.0 ** -23) for w in (b, c))
    want = activation(g, act) * u
    bound = 1.13 * eg * (u.abs() + eu) + (g.abs() + eg) * eu + (HALF + 2.0 ** -16) * want.abs() + 1e-30
    assert ((h.double() - want).abs() <= 1.01 * bound).all()
    for got, v, e in ((g8, g, eg), (u8, u, eu)):
        back = mx.act8_restore(got, out_dtype=F32).double()
        pad = torch.nn.functional.pad(v.abs() + e, (0, -F % 32)).view(T, -1, 32).amax(2)
        largest = pad.repeat_interleave(32, dim=1)[:, :F]
        assert ((back - v).abs() <= 2.0 ** -4 * (v.abs() + e) + e + largest * 2.0 ** -17).all()
        assert not got.codes[:, F:].any()  # the pad columns hold code 0
    assert float(top) == float(h.float().abs().max())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,F", [(1, 512, 128), (5, 256, 56), (300, 768, 384), (161, 256, 96), (96, 256, 16), (96, 512, 208),
                                   (70, 1024, 131)])
def test_forms_of_the_weights_agree(mx, fmt, T, K, F):
    """Quantized beforehand, within the call, or with the saved state: the same h.  (K is too short for few tokens'
    sums to be cut.)"""
    X, W = data(T, K, F, 1)
    h = mx.gated_fwd(X, mx.gated_weights(W, fmt), fmt)
    assert torch.equal(h, mx.gated_fwd(X, W, fmt))
    x = mx.quantize(X, fmt)
    assert torch.equal(h, mx.gemm_gated(x, *mx.gated_weights(W, fmt)).h)
    if T % 32 == 0 and F % 16 == 0:
        assert torch.equal(h, mx.gated_fwd_save(X, W, fmt).h)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 3, 15, 16, 17, 31, 33, 48, 64, 65])
@pytest.mark.parametrize("K,F", [(256, 128), (1280, 300), (4096, 264)])
def test_few_tokens(mx, fmt, T, K, F):
    """The kernel for few tokens against the one for many (which keeps checkpoints), and the tokens' quantization
    within the call against the one on its own: a row that is all zeros and a tensor that is among them."""
    X, W = data(T, K, F, T)
    X[T // 2] = 0
    if T == 3:
        X.zero_()
    if T == 15:
        X *= 2.0 ** -120  # block scales at their lower end
    gate, up = mx.gated_weights(W, fmt)
    top = torch.empty(1, device="cuda")
    for act in ACTS:
        many = mx.gemm_gated(mx.quantize(X, fmt), gate, up, act=act, save=True).h
        few = mx.gemm_gated(mx.quantize(X, fmt), gate, up, act=act, amax_out=top).h
        assert torch.equal(few, many) and float(top) == float(many.float().abs().max())
        # within the call the sums may be cut along K and joined: fp32 sums in another order, the bound of the 64-bit
        # test on both, so twice that
        whole = mx.gated_fwd(X, (gate, up), fmt, act=act, amax_out=top)
        assert float(top) == float(whole.float().abs().max())
        assert torch.equal(whole, mx.gated_fwd(X, (gate, up), fmt, act=act))  # one order
        a, b, c = (values(mx, q) for q in (mx.quantize(X, fmt), gate, up))
        g, u = a @ b.T, a @ c.T
        eg, eu = ((a.abs() @ w.abs().T) * (K * 2.0 ** -23) for w in (b, c))
        want = activation(g, act) * u
        bound = 1.13 * eg * (u.abs() + eu) + (g.abs() + eg) * eu + (HALF + 2.0 ** -16) * want.abs() + 1e-30
        assert ((whole.double() - want).abs() <= 1.01 * bound).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("special", [0.0, -0.0, float("inf"), float("-inf"), float("nan"), 3.3e38, 1e-40, 2.0 ** -126])
def test_few_tokens_with_special_values(mx, fmt, special):
    """The tokens' quantization within the call treats every value as the one on its own does (K is too short for the
    sums to be cut, so that the results are the same numbers)."""
    X, W = data(7, 256, 56, 4)
    X[2, 5] = special
    X[4, 32:80] = special
    X[5] *= 2.0 ** -100
    w = mx.gated_weights(W, fmt)
    got, want = mx.gated_fwd(X, w, fmt), mx.gemm_gated(mx.quantize(X, fmt), *w).h
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.float(), 1234.0), torch.nan_to_num(want.float(), 1234.0))


def test_few_tokens_of_a_wide_matrix(mx):
    """More values than the small quantization holds, rows of a wider matrix, and both captured."""
    for T, K in ((64, 8192 + 256), (64, 8192), (5, 256)):
        X, W = data(T, K + 64, 256, 3)
        X, W = X[:, 32:K + 32], W[:, :K].contiguous()
        for fmt in ("nvfp4", "mxfp8"):
            w = mx.gated_weights(W, fmt)
            many = mx.gemm_gated(mx.quantize(X.contiguous(), fmt), *w, save=True).h.double()
            want = mx.gated_fwd(X, w, fmt)
            # sums of K products in another order: their size is at most sqrt(K) here, 2^-23 K of it each
            assert ((want.double() - many).abs() <= 2 * HALF * many.abs() + K ** 1.5 * 2.0 ** -23 * (1 + many.abs())).all()
            if K == 256:  # too few steps to cut
                assert torch.equal(want.double(), many)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                h = mx.gated_fwd(X, w, fmt)
            for _ in range(2):
                h.zero_()
                g.replay()
                assert torch.equal(h, want)


def test_checkpoint_of_values_that_are_not_finite(mx):
    """Products that overflow: their codes are NaN, their groups' other values keep their own scale."""
    T, K, F = 130, 256, 96
    X, W = data(T, K, F, 12)
    X[5] *= 2.0 ** 100
    W[7] *= 2.0 ** 100  # gate feature 7
    W[F + 40] *= 2.0 ** 100  # up feature 40
    x, (gate, up) = mx.quantize(X, "mxfp8"), mx.gated_weights(W, "mxfp8")
    h, g8, u8 = mx.gemm_gated(x, gate, up, save=True)
    g, u = products(mx, x, gate, up)
    assert not torch.isfinite(g[5, 7]) and not torch.isfinite(u[5, 40])
    for got, want in ((g8, mx.act8_save(g)), (u8, mx.act8_save(u))):
        assert torch.equal(got.codes & 127, want.codes & 127) and torch.equal(got.sf, want.sf)
    room = torch.full((T, 8, 32), 77, dtype=torch.uint8, device="cuda")
    sf = torch.full((T * 3 + 1,), 77, dtype=torch.uint8, device="cuda")  # bytes at an odd address
    odd = mx.Act8(room[:, :3].reshape(T, 96).contiguous(), sf[1:].view(T, 3), F)
    kept = mx.gated_fwd_save(X[:128], W, "mxfp8", gate8=mx.Act8(odd.codes[:128], odd.sf[:128], F))
    assert torch.equal(kept.gate.codes & 127, g8.codes[:128] & 127) and torch.equal(kept.gate.sf, g8.sf[:128])
    assert (sf[0] == 77) and (sf[1 + 128 * 3:] == 77).all()


TRAIN = [(256, 256, 128), (256, 512, 384), (512, 768, 128 + 256), (256, 256, 640)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,F", TRAIN)
@pytest.mark.parametrize("act", ACTS)
def test_gradients_are_those_of_the_calls(mx, fmt, T, K, F, act):
    X, W = data(T, K, F, 2)
    dH = (torch.randn(T, F, device="cuda") * 1e-2).to(BF)
    kept = mx.gated_fwd_save(X, W, fmt, act=act)
    assert torch.equal(kept.h, mx.gated_fwd(X, W, fmt, act=act))
    x, (gate, up) = mx.quantize(X, fmt), mx.gated_weights(W, fmt)
    h, g8, u8 = mx.gemm_gated(x, gate, up, act=act, save=True)
    assert torch.equal(kept.gate.codes, g8.codes) and torch.equal(kept.up.sf, u8.sf)
    dX, dW = mx.gated_bwd(dH, kept, K, fmt, act=act)
    top = torch.empty(1, device="cuda")
    dg, du = mx.act_bwd(dH, g8, u8, act=act, amax_out=top)
    D = dg.as_strided((T, 2 * F), (2 * F, 1))
    _, saved = mx.linear_fwd_save(X, W, fmt)
    wX, wW = mx.linear_bwd_saved(D, saved, K, fmt, dy_amax=top if fmt in ("nvfp4", "moss") else None)
    assert torch.equal(dX, wX) and torch.equal(dW, wW)
    only, none = mx.gated_bwd(dH, kept, K, fmt, act=act, need_dw=False)
    assert torch.equal(only, dX) and none is None
    none, only = mx.gated_bwd(dH, kept, K, fmt, act=act, need_dx=False, dw_dtype=BF)
    assert torch.equal(only, dW.to(BF)) and none is None


@pytest.mark.parametrize("fmt,T,F,K", [("mxfp8", 128, 64, 256), ("mxfp8", 384, 192, 128), ("moss", 128, 320, 256),
                                       ("mxfp8", 128, 3392, 640), ("nvfp4_local", 256, 128, 256)])
def test_gradients_where_up_starts_within_a_scale_chunk(mx, fmt, T, F, K):
    X, W = data(T, K, F, 3)
    dH = (torch.randn(T, F, device="cuda") * 1e-2).to(BF)
    kept = mx.gated_fwd_save(X, W, fmt)
    top = torch.empty(1, device="cuda")
    dg, du = mx.act_bwd(dH, kept.gate, kept.up, amax_out=top)
    _, saved = mx.linear_fwd_save(X, W, fmt)
    wX, wW = mx.linear_bwd_saved(dg.as_strided((T, 2 * F), (2 * F, 1)), saved, K, fmt,
                                 dy_amax=top if fmt == "moss" else None)
    dX, dW = mx.gated_bwd(dH, kept, K, fmt)
    assert torch.equal(dX, wX) and torch.equal(dW, wW)


@pytest.mark.parametrize("fmt,opts", [("mxfp4", dict(wgrad_hadamard=True, wgrad_dy_rounding="sr", seed=7)),
                                      ("nvfp4", dict(wgrad_hadamard=True)), ("mxfp8", dict(wgrad_dy_rounding="sr", seed=3))])
def test_backward_options(mx, fmt, opts):
    T, K, F = 256, 256, 256
    X, W = data(T, K, F, 4)
    dH = (torch.randn(T, F, device="cuda") * 1e-2).to(BF)
    kept = mx.gated_fwd_save(X, W, fmt, **opts)
    dg, _ = mx.act_bwd(dH, kept.gate, kept.up)
    _, saved = mx.linear_fwd_save(X, W, fmt, **opts)
    wX, wW = mx.linear_bwd_saved(dg.as_strided((T, 2 * F), (2 * F, 1)), saved, K, fmt, **opts)
    dX, dW = mx.gated_bwd(dH, kept, K, fmt, **opts)
    assert torch.equal(dX, wX) and torch.equal(dW, wW)


def test_gradients_against_differences(mx):
    """Along random directions the loss <h, c> in 64 bits moves as the gradients say, up to the formats' rounding:
    each operand of each product is off by 2^-4 of its size (E4M3 codes), independently from value to value, and a
    gradient's product with a random direction keeps a share sqrt(2 / n) of that at most: 0.1 holds by far."""
    T, K, F = 256, 256, 128
    X, W = data(T, K, F, 5)
    c = torch.randn(T, F, device="cuda").to(BF)
    kept = mx.gated_fwd_save(X, W, "mxfp8")
    dX, dW = mx.gated_bwd(c, kept, K, "mxfp8")

    def loss(x, w):
        gu = x @ w.T
        return (activation(gu[:, :F], "silu") * gu[:, F:] * c.double()).sum()

    x, w = X.double(), W.double()
    for grad, base, other in ((dX, x, 0), (dW, w, 1)):
        v = grad.double() / grad.double().norm()  # the steepest direction: the derivative is the gradient's norm
        e = 1e-4
        args = lambda s: (x + s * v, w) if other == 0 else (x, w + s * v)  # noqa: E731
        slope = (loss(*args(e)) - loss(*args(-e))) / (2 * e)
        assert abs(float(slope) / float(grad.double().norm()) - 1) < 0.1


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_given_buffers_and_strides(mx, fmt):
    """Rows of X, dH and h inside wider matrices; what lies beside h's rows stays."""
    T, K, F = 256, 256, 200 if fmt == "mxfp8" else 128
    X, W = data(T, K, F, 6)
    wide = torch.zeros(T, K + 24, dtype=BF, device="cuda")
    wide[:, 8:8 + K] = X
    room = torch.full((T + 2, F + 32), 5.0, dtype=BF, device="cuda")
    out = room[1:T + 1, 8:8 + F]
    h = mx.gated_fwd(wide[:, 8:8 + K], W, fmt, out=out)
    assert h is out and torch.equal(h, mx.gated_fwd(X, W, fmt))
    mask = torch.ones_like(room, dtype=torch.bool)
    mask[1:T + 1, 8:8 + F] = False
    assert (room[mask] == 5.0).all()
    if F % 64 == 0:
        kept = mx.gated_fwd_save(X, W, fmt)
        ws = torch.empty(mx.gated_workspace_bytes(T, K, F, fmt, "bwd"), dtype=torch.uint8, device="cuda")
        dh = torch.randn(T, F + 3, device="cuda").to(BF)[:, 1:F + 1]  # rows at odd addresses
        a = mx.gated_bwd(dh, kept, K, fmt, workspace=ws)
        b = mx.gated_bwd(dh.contiguous(), kept, K, fmt)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    else:  # FP8, whole tiles: rows at odd addresses and a workspace off the sector's grid take the separate passes
        F = 128
        X, W = data(T, K, F, 6)
        kept = mx.gated_fwd_save(X, W, fmt)
        dh = torch.randn(T, F + 3, device="cuda").to(BF)[:, 1:F + 1]
        n = mx.gated_workspace_bytes(T, K, F, fmt, "bwd")
        ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
        want = mx.gated_bwd(dh.contiguous(), kept, K, fmt)
        for a in (mx.gated_bwd(dh, kept, K, fmt), mx.gated_bwd(dh.contiguous(), kept, K, fmt, workspace=ws[16:])):
            assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_empty(mx, fmt):
    X, W = data(0, 256, 128)
    top = torch.full((1,), 3.0, device="cuda")
    assert mx.gated_fwd(X, W, fmt, amax_out=top).shape == (0, 128) and float(top) == 0.0
    kept = mx.gated_fwd_save(X, W, fmt)
    dX, dW = mx.gated_bwd(torch.empty(0, 128, dtype=BF, device="cuda"), kept, 256, fmt)
    assert dX.shape == (0, 256) and not dW.any()
    X, W = data(4, 256, 0)
    assert mx.gated_fwd(X, W, fmt).shape == (4, 0)


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_captured_and_on_other_streams(mx, fmt):
    """Two captured steps, replayed on new inputs and in turn with eager calls on another stream."""
    T, K, F = 256, 256, 256
    X, W = data(T, K, F, 7)
    dH = (torch.randn(T, F, device="cuda") * 1e-2).to(BF)

    def step():
        kept = mx.gated_fwd_save(X, W, fmt)
        return (kept.h, *mx.gated_bwd(dH, kept, K, fmt))

    step()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    side = torch.cuda.Stream()
    for seed in range(3):
        X.copy_(data(T, K, F, 20 + seed)[0])
        for g, _ in graphs:
            g.replay()
        side.wait_stream(torch.cuda.current_stream())
        kept = mx.gated_fwd_save(X, W, fmt, stream=side)
        dX, dW = mx.gated_bwd(dH, kept, K, fmt, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, (kept.h, dX, dW)))


@pytest.mark.parametrize("T,K,F", [(1, 4096, 256), (48, 2048, 640), (200, 512, 256)])
def test_calls_at_once_and_one_behind_another(mx, T, K, F):
    """Two streams with workspaces of their own, each with many calls behind one another in the same workspace."""
    W = mx.gated_weights(data(T, K, F, 30)[1], "nvfp4")
    X = [data(T, K, F, 31 + i)[0] for i in range(4)]
    want = [mx.gated_fwd(x, W, "nvfp4") for x in X]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    n = mx.gated_workspace_bytes(T, K, F, "nvfp4", "fwd_quantized")
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    got = []
    for i in range(24):
        for k, s in enumerate(streams):
            j = (i + k) % 4
            got.append((j, mx.gated_fwd(X[j], W, "nvfp4", workspace=spaces[k], stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(h, want[j]) for j, h in got)


def test_past_2g_values(mx):
    """h and the checkpoints of more than 2^31 values: the last rows are what the same call makes of them alone."""
    K, F, tail = 128, 14336, 64
    T = (1 << 31) // F + 300
    X, W = data(T, K, F, 8)
    x, (gate, up) = mx.quantize(X, "mxfp8"), mx.gated_weights(W, "mxfp8")
    h, g8, u8 = mx.gemm_gated(x, gate, up, save=True)
    s, sg, su = mx.gemm_gated(mx.quantize(X[-tail:].contiguous(), "mxfp8"), gate, up, save=True)
    assert torch.equal(h[-tail:], s)
    assert torch.equal(g8.codes[-tail:], sg.codes) and torch.equal(u8.sf[-tail:], su.sf)


def test_used_as_a_training_step(mx):
    """Norm, block, down projection and back, clipping and the optimizer's step, whose copies and maxima the next
    forward pass reads: the same numbers as with the separate calls and fp32 weights kept by hand."""
    T, K, F, fmt = 256, 256, 256, "nvfp4"
    g = torch.Generator(device="cuda").manual_seed(9)
    master = [(torch.randn(s, generator=g, device="cuda") / math.sqrt(s[1])) for s in ((2 * F, K), (K, F))]
    copies = [m.to(BF) for m in master]
    opt = mx.AdamW(master, lr=1e-2, state="8bit", copies=copies, rounding="sr", seed=11)
    x = torch.randn(T, K, generator=g, device="cuda").to(BF)
    dout = (torch.randn(T, K, generator=g, device="cuda") * 1e-2).to(BF)
    tops = torch.empty(2, device="cuda")
    for step in range(3):
        n_top, h_top = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        n = mx.norm_fwd(x, kind="rms", amax_out=n_top)
        w_top = tops[0:1] if step else None
        kept = mx.gated_fwd_save(n.y, copies[0], fmt, x_amax=n_top, w_amax=w_top, amax_out=h_top)
        assert torch.equal(kept.h, mx.gated_fwd_save(n.y, copies[0], fmt).h)  # the reported maxima are the tensors' own
        out, kept_d = mx.linear_fwd_save(kept.h, copies[1], fmt, x_amax=h_top, w_amax=tops[1:2] if step else None)
        assert torch.equal(out, mx.linear_fwd(kept.h, copies[1], fmt))
        dh, d_down = mx.linear_bwd_saved(dout, kept_d, F, fmt)
        _, d_gu = mx.gated_bwd(dh, kept, K, fmt)
        scale = mx.grad_norm([d_gu, d_down], max_norm=0.1)
        norm = math.sqrt(float((d_gu.double() ** 2).sum() + (d_down.double() ** 2).sum()))
        assert abs(float(scale[0]) / norm - 1) < 1e-6
        before = [c.clone() for c in copies]
        opt.step([d_gu, d_down], grad_scale=scale[1:], amax_out=tops)
        assert all(torch.equal(c, m.to(BF)) and not torch.equal(c, b) for c, m, b in zip(copies, master, before))
        assert [float(t) for t in tops] == [float(c.abs().max()) for c in copies]
