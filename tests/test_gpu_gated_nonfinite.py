"""The gated block's backward pass where dH or a checkpoint holds values that are not finite: the
pass that encodes D as it makes it gives what act_bwd and linear_bwd_saved give one after the other."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
T, K, F = 256, 256, 128
BLOCK = slice(32, 64)
# rows and columns of dH that hold the value
WHERE = {"one": (5, 40), "block": (6, BLOCK), "even columns of a block": (7, slice(32, 64, 2)),
         "odd columns of a block": (8, slice(33, 64, 2)), "row": (9, slice(None)), "even columns of a row": (10, slice(0, F, 2)),
         "column": (slice(None), 3), "even rows of a block of a column": (slice(32, 64, 2), 70),
         "all but one of a block": (11, slice(33, 64)), "all": (slice(None), slice(None))}


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    yield m
    assert m.last_device_status() == m.MX_OK


def same(a, b):
    """Equal bit for bit, any NaN being one."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a, 0.0, math.inf, -math.inf),
                                                                       torch.nan_to_num(b, 0.0, math.inf, -math.inf))


def both_ways(mx, fmt, X, W, dH, kept):
    """(dX, dW) of gated_bwd, and of the calls it is made of."""
    got = mx.gated_bwd(dH, kept, K, fmt)
    dg, _ = mx.act_bwd(dH, kept.gate, kept.up)
    _, saved = mx.linear_fwd_save(X, W, fmt)
    return got, mx.linear_bwd_saved(dg.as_strided((T, 2 * F), (2 * F, 1)), saved, K, fmt)


def data(mx, fmt):
    g = torch.Generator(device="cuda").manual_seed(31)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    X, W, dH = n(T, K).to(BF), (n(2 * F, K) / math.sqrt(K)).to(BF), (n(T, F) * 1e-2).to(BF)
    return X, W, dH, mx.gated_fwd_save(X, W, fmt)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", WHERE, ids=str)
def test_dh(mx, fmt, value, where):
    X, W, dH, kept = data(mx, fmt)
    dH[WHERE[where]] = value
    got, want = both_ways(mx, fmt, X, W, dH, kept)
    assert same(got[0], want[0]) and same(got[1], want[1])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("where", ["one", "even columns of a block", "odd columns of a block", "row", "column"])
@pytest.mark.parametrize("half", ["gate", "up"])
def test_checkpoint(mx, fmt, where, half):
    """Codes that stand for NaN, as the forward pass leaves them for products that overflow."""
    X, W, dH, kept = data(mx, fmt)
    getattr(kept, half).codes[WHERE[where]] = 0x7F
    got, want = both_ways(mx, fmt, X, W, dH, kept)
    assert same(got[0], want[0]) and same(got[1], want[1])


@pytest.mark.parametrize("where", WHERE, ids=str)
def test_rowwise_operand(mx, where):
    """MXFP8, whose products hide a row's codes behind its NaN: the operand itself, in the workspace behind the room
    for D [T, 2 F] and for its maximum."""
    X, W, dH, kept = data(mx, "mxfp8")
    dH[WHERE[where]] = math.nan
    ws = torch.zeros(mx.gated_workspace_bytes(T, K, F, "mxfp8", "bwd"), dtype=torch.uint8, device="cuda")
    mx.gated_bwd(dH, kept, K, "mxfp8", workspace=ws)
    dg, _ = mx.act_bwd(dH, kept.gate, kept.up)
    want = mx.quantize(dg.as_strided((T, 2 * F), (2 * F, 1)), "mxfp8")
    at = 4 * T * F + 256
    codes, sf = ws[at:at + 2 * T * F], ws[at + 2 * T * F:at + 2 * T * F + want.sf.numel()]
    assert torch.equal(codes & 127, want.codes.view(-1).view(torch.uint8) & 127)  # a NaN's sign aside
    assert torch.equal(sf, want.sf.view(-1).view(torch.uint8))
