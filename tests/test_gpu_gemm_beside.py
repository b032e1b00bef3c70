"""Nothing beside the rows of a product is written, by any of its kernels."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    yield m
    m.set_gemm_variant("auto")
    assert m.last_device_status() == m.MX_OK


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("N", [1, 3, 4, 8, 12, 21, 32, 50, 130, 260, 262, 264])
@pytest.mark.parametrize("variant", ["cta_n128", "cta_n256", "pair", "pair_ws", "auto"])
def test_beside(mx, fmt, dtype, N, variant):
    K, M = 512, 300
    g = torch.Generator(device="cuda").manual_seed(N)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    a, b = mx.quantize(n(M, K), fmt), mx.quantize(n(N, K), fmt)
    ld, first = -(-N // 8) * 8 + 16, 8
    room = torch.full(((M + 2) * ld,), 5.0, dtype=dtype, device="cuda")
    out = room[ld + first:ld + first + (M - 1) * ld + N].as_strided((M, N), (ld, 1))
    mx.set_gemm_variant(variant)
    try:
        mx.gemm(a, b, out_dtype=dtype, out=out)
    finally:
        mx.set_gemm_variant("auto")
    want = mx.dequantize(a).double() @ mx.dequantize(b).double().T
    size = mx.dequantize(a).double().abs() @ mx.dequantize(b).double().abs().T
    half = 2.0 ** -8 if dtype is BF else 2.0 ** -24
    assert ((out.double() - want).abs() <= half * want.abs() + 1.01 * K * 2.0 ** -23 * size).all()
    out.fill_(5.0)
    assert (room == 5.0).all()
