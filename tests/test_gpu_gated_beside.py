"""Nothing beside h's rows is written: what lies between one row's last column and the next row, before the first
row and behind the last one stays, whatever the number of columns."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
COLUMNS = [1, 2, 3, 7, 8, 9, 12, 20, 31, 32, 33, 36, 61, 64, 65, 100, 127, 130, 161, 200, 253, 257]


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    yield m
    assert m.last_device_status() == m.MX_OK


def data(T, K, F):
    g = torch.Generator(device="cuda").manual_seed(F)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return n(T, K).to(BF), (n(2 * F, K) / math.sqrt(K)).to(BF)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("F", COLUMNS)
@pytest.mark.parametrize("T", [1, 40, 65, 130, 300])
def test_beside(mx, fmt, F, T):
    K = 256
    X, W = data(T, K, F)
    weights = mx.gated_weights(W, fmt)
    x = mx.quantize(X, fmt)
    want = mx.gated_fwd(X, weights, fmt)
    ld, first = -(-F // 8) * 8 + 8, 8
    for call in (lambda out: mx.gated_fwd(X, weights, fmt, out=out), lambda out: mx.gemm_gated(x, *weights, save=True, out=out)):
        room = torch.full(((T + 2) * ld,), 5.0, dtype=BF, device="cuda")
        out = room[ld + first:ld + first + (T - 1) * ld + F].as_strided((T, F), (ld, 1))
        call(out)
        assert torch.equal(out, want)
        out.fill_(5.0)
        assert (room == 5.0).all()
