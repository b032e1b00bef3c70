"""The gated block for few tokens where its tests with small shapes do not reach: tokens' quantization of
several values a thread bit for bit, more tiles than SMs, ranges that hold part of a tile, whole ones and
part of another, rows too wide for the small quantization, and two host threads."""
import math
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

FORMATS = ("mxfp8", "mxfp4", "nvfp4", "moss", "nvfp4_local")
BF = torch.bfloat16
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    yield m
    assert m.last_device_status() == m.MX_OK


def data(T, K, F, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return n(T, K).to(BF), (n(2 * F, K) / math.sqrt(K)).to(BF)


def values(mx, q):
    """float64 values of an operand.  mx_dequantize takes one tensor scale: one by region is put on by rows."""
    if q.fmt != "nvfp4_local":
        return mx.dequantize(q).double()
    plain = mx.MXTensor("nvfp4", q.rows, q.k)
    plain.codes, plain.sf = q.codes, q.sf
    plain.scalars.fill_(1.0)
    return mx.dequantize(plain).double() * q.tensor_scale.double().repeat_interleave(128)[:q.rows, None]


def near(mx, h, x, gate, up):
    """h within the error of fp32 sums of K products in any order: 2^-23 of the products' sizes each, then SiLU and
    the product in fp32 and one rounding to bf16."""
    a, b, c = (values(mx, q) for q in (x, gate, up))
    g, u = a @ b.T, a @ c.T
    eg, eu = ((a.abs() @ w.abs().T) * (x.k * 2.0 ** -23) for w in (b, c))
    want = g / (1 + torch.exp(-g)) * u
    bound = 1.13 * eg * (u.abs() + eu) + (g.abs() + eg) * eu + (HALF + 2.0 ** -16) * want.abs() + 1e-30
    return bool(((h.double() - want).abs() <= 1.01 * bound).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,F", [(48, 4096, 12288), (64, 8192, 13312), (33, 4096, 12288)])
def test_quantization_bit_for_bit(mx, fmt, T, K, F):
    """Widths whose tiles are not cut: the same numbers as from operands quantized by themselves.  Some rows hold
    values of their own kind, each in another part of the tensor."""
    X, W = data(T, K, F, T)
    X[3] = 0
    X[T // 2] *= 2.0 ** -60
    X[T - 1, K - 16:] = 0
    X[T - 2, ::2] *= 2.0 ** -8
    w = mx.gated_weights(W, fmt)
    top, want_top = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    got = mx.gated_fwd(X, w, fmt, amax_out=top)
    want = mx.gemm_gated(mx.quantize(X, fmt), *w, amax_out=want_top).h
    assert torch.equal(got, want) and torch.equal(top, want_top)
    X[T - 1, K - 40] = math.inf  # the last values of the last thread's range
    X[T - 2, 5] = math.nan
    got, want = mx.gated_fwd(X, w, fmt), mx.gemm_gated(mx.quantize(X, fmt), *w).h
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, 7.0, 8.0, 9.0), torch.nan_to_num(want, 7.0, 8.0, 9.0))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 17, 64])
@pytest.mark.parametrize("K,tiles", [(768, 160), (768, 224), (768, 320), (2048, 40), (2048, 153), (4096, 9), (256, 305)])
def test_tiles_and_ranges(mx, fmt, T, K, tiles):
    """Few tiles, some more than SMs, twice as many and some: with K = 768 a tile has three or six steps, so that
    ranges start and end inside one.  Every call adds up in the same order."""
    F = tiles * 128 - 24
    X, W = data(T, K, F, tiles)
    gate, up = mx.gated_weights(W, fmt)
    top = torch.empty(1, device="cuda")
    h = mx.gated_fwd(X, (gate, up), fmt, amax_out=top)
    assert near(mx, h, mx.quantize(X, fmt), gate, up)
    assert float(top) == float(h.float().abs().max())
    assert torch.equal(h, mx.gated_fwd(X, (gate, up), fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,F", [(48, 14336, 1024), (64, 16384, 40), (5, 2 ** 17, 256)])
def test_wide_rows(mx, fmt, T, K, F):
    """More values than one cluster's registers hold, weights in the call and beforehand."""
    X, W = data(T, K, F, 5)
    gate, up = mx.gated_weights(W, fmt)
    h = mx.gated_fwd(X, (gate, up), fmt)
    assert near(mx, h, mx.quantize(X, fmt), gate, up)
    assert torch.equal(h, mx.gated_fwd(X, W, fmt))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mx.gated_fwd(X, (gate, up), fmt)
    for _ in range(2):
        out.zero_()
        g.replay()
        assert torch.equal(out, h)


def test_two_host_threads(mx):
    """Forward, saved state and backward from two threads on streams of their own, against the same calls alone."""
    fmt, K, F, T = "nvfp4", 512, 512, 256

    def work(seed, got):
        X, W = data(T, K, F, seed)
        few = X[:48]
        dH = (X[:, :F] * 1e-2).contiguous()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            w = mx.gated_weights(W, fmt)
            for _ in range(20):
                kept = mx.gated_fwd_save(X, W, fmt)
                dX, dW = mx.gated_bwd(dH, kept, K, fmt)
                got.append((kept.h, kept.gate.codes, kept.up.sf, dX, dW, mx.gated_fwd(few, w, fmt)))
        stream.synchronize()

    results = [[], []]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(50 + i, results[i])) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        alone = []
        work(50 + i, alone)
        assert len(results[i]) == 20
        for r in results[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, alone[0]))


@pytest.mark.parametrize("fmt", FORMATS)
def test_wide_rows_are_cut(mx, fmt):
    """Eight tiles of a long K are cut whatever quantizes the tokens: every tile's counter, at the workspace's end,
    has been set to zero and counted its pieces."""
    T, K, F = 48, 14336, 1024
    X, W = data(T, K, F, 6)
    w = mx.gated_weights(W, fmt)
    ws = torch.full((mx.gated_workspace_bytes(T, K, F, fmt, "fwd_quantized"),), 0x5A, dtype=torch.uint8, device="cuda")
    want = mx.gated_fwd(X, w, fmt)
    for _ in range(2):
        assert torch.equal(mx.gated_fwd(X, w, fmt, workspace=ws), want)
        counts = ws[-256:].view(torch.int32)[:F // 128]
        assert ((counts > 1) & (counts <= 152)).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4", "nvfp4_local"])
@pytest.mark.parametrize("K,tiles", [(4096, 32), (4096, 64), (1024, 8), (768, 200)])
def test_one_workspace_for_every_batch(mx, fmt, K, tiles):
    """A workspace for 64 tokens serves the batches that shrink and grow behind one another, cut or not."""
    X, W = data(64, K, 128 * tiles, 8)
    for weights in (mx.gated_weights(W, fmt), W):
        ws = torch.full((mx.gated_workspace_bytes(64, K, 128 * tiles, fmt, "fwd" if weights is W else "fwd_quantized"),), 0x5A,
                        dtype=torch.uint8, device="cuda")
        for T in (64, 1, 48, 7, 16, 33, 64, 2):
            assert torch.equal(mx.gated_fwd(X[:T], weights, fmt, workspace=ws), mx.gated_fwd(X[:T], weights, fmt))
