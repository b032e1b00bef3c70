"""What mx_gemm_gated refuses, before it looks for a device."""
import pytest

import fp4_precision_gemms_gb300 as mx

BAD, UNSUP, ALIGN = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED, mx.MX_ERR_ALIGNMENT
P = 1 << 20  # an address that is never read: every call here is refused


@pytest.fixture(scope="module")
def L():
    mx.build()
    return mx.lib()


def operand(rows=64, k=256, fmt=0, codes=P, sf=P, ts=P, had=0, block=32):
    return mx._CTensor(codes, sf, ts, ts, rows, k, fmt, block, had, 0)


def a8(rows=32, cols=64, codes=P, sf=P):
    return mx._CAct8(codes, sf, rows, cols)


def call(L, **k):
    d = dict(a=operand(32), gate=operand(), up=operand(), act=0, h=P, ldh=64, gate8=None, up8=None, amax=None)
    assert set(k) <= set(d)
    d.update(k)
    return L.mx_gemm_gated(*d.values(), None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(a=None)), (BAD, dict(gate=None)), (BAD, dict(up=None)), (BAD, dict(act=3)), (BAD, dict(act=-1)), (BAD, dict(h=None)),
    (BAD, dict(ldh=56)), (ALIGN, dict(ldh=68)), (ALIGN, dict(h=P + 8)), (ALIGN, dict(amax=P + 2)), (BAD, dict(up=operand(63))),
    (BAD, dict(gate8=a8())), (BAD, dict(up8=a8())), (BAD, dict(gate8=a8(31), up8=a8())), (BAD, dict(gate8=a8(), up8=a8(32, 63))),
    (ALIGN, dict(gate8=a8(codes=P + 8), up8=a8())), (BAD, dict(gate8=a8(sf=None), up8=a8())),
    (ALIGN, dict(a=operand(32, 192), gate=operand(64, 192), up=operand(64, 192))),
    (UNSUP, dict(a=operand(32, 0), gate=operand(64, 0), up=operand(64, 0))), (UNSUP, dict(a=operand(1 << 31)))])
def test_refuses(L, want, kw):
    assert call(L, **kw) == want


@pytest.mark.parametrize("which", ["a", "gate", "up"])
@pytest.mark.parametrize("want,bad", [(BAD, dict(k=512)), (BAD, dict(fmt=3)), (BAD, dict(fmt=9)), (BAD, dict(codes=None)),
                                      (BAD, dict(sf=None)), (ALIGN, dict(codes=P + 8)), (ALIGN, dict(sf=P + 4)), (BAD, dict(block=16)),
                                      (UNSUP, dict(had=1)), (BAD, dict(rows=-1))])
def test_refuses_operands(L, which, want, bad):
    assert call(L, **{which: operand(**{"rows": 32 if which == "a" else 64, **bad})}) == want
