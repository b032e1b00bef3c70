"""What the gated feed-forward block's calls refuse, before anything is launched."""
import ctypes as C

import pytest
import torch

import fp4_precision_gemms_gb300 as mx

OK, BAD, UNSUP, ALIGN, WS = 0, mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED, mx.MX_ERR_ALIGNMENT, mx.MX_ERR_WORKSPACE
P = 1 << 20  # an address that is never read: every call here is refused


@pytest.fixture(scope="module")
def L():
    mx.build()
    return mx.lib()


def operand(rows=64, k=256, fmt=0, codes=P, sf=P, ts=P, had=0, block=32):
    return mx._CTensor(codes, sf, ts, ts, rows, k, fmt, block, had, 0)


def a8(rows=32, cols=64, codes=P, sf=P):
    return mx._CAct8(codes, sf, rows, cols)


def fwd(L, **k):
    d = dict(X=P, ldx=256, T=32, Kin=256, F=64, fmt=0, act=0, W=P, gate=None, up=None, h=P, ldh=64, amax=None, ws=P, n=1 << 30)
    assert set(k) <= set(d)
    d.update(k)
    return L.mx_gated_fwd(*d.values(), None)


COMMON = [(BAD, dict(T=-1)), (BAD, dict(F=-1)), (BAD, dict(Kin=-1)), (BAD, dict(fmt=9)), (BAD, dict(act=3)), (BAD, dict(T=1 << 31)),
          (BAD, dict(X=None)), (BAD, dict(ldx=255)), (ALIGN, dict(ldx=260)), (ALIGN, dict(X=P + 8)), (ALIGN, dict(Kin=0)),
          (ALIGN, dict(Kin=192, ldx=192)), (ALIGN, dict(fmt=2, Kin=128, ldx=128)), (BAD, dict(h=None)), (BAD, dict(ldh=56)),
          (ALIGN, dict(ldh=68)), (ALIGN, dict(h=P + 4)), (ALIGN, dict(amax=P + 1)), (ALIGN, dict(W=P + 2)), (WS, dict(ws=None)),
          (WS, dict(n=100)), (ALIGN, dict(ws=P + 8))]


@pytest.mark.parametrize("want,kw", COMMON + [(BAD, dict(W=None)), (BAD, dict(gate=operand(), up=operand())),
                                              (BAD, dict(W=None, gate=operand()))])
def test_fwd_refuses(L, want, kw):
    assert fwd(L, **kw) == want


@pytest.mark.parametrize("want,bad", [(BAD, dict(rows=63)), (BAD, dict(k=512)), (BAD, dict(fmt=3)), (BAD, dict(codes=None)),
                                      (ALIGN, dict(codes=P + 8)), (BAD, dict(block=16)), (UNSUP, dict(had=1))])
def test_fwd_refuses_operands(L, want, bad):
    assert fwd(L, W=None, gate=operand(**bad), up=operand()) == want
    assert fwd(L, W=None, gate=operand(), up=operand(**bad)) == want


def save(L, opts=None, **k):
    d = dict(X=P, ldx=256, W=P, T=32, Kin=256, F=64, fmt=0, act=0, x_amax=None, w_amax=None, o=None, h=P, ldh=64, gate8=a8(),
             up8=a8(), amax=None, ws=P, n=1 << 30, saved=P, ns=1 << 30)
    assert set(k) <= set(d)
    d.update(k)
    d["o"] = C.byref(mx._CBwdOpts(*opts)) if opts else None
    return L.mx_gated_fwd_save(*d.values(), None)


@pytest.mark.parametrize("want,kw", COMMON + [
    (BAD, dict(W=None)), (BAD, dict(gate8=None)), (BAD, dict(up8=a8(31))), (BAD, dict(gate8=a8(32, 63))), (BAD, dict(up8=a8(codes=None))),
    (ALIGN, dict(gate8=a8(codes=P + 8))), (ALIGN, dict(T=33, gate8=a8(33), up8=a8(33))),
    (ALIGN, dict(F=56, ldh=56, gate8=a8(32, 56), up8=a8(32, 56))), (WS, dict(saved=None)), (WS, dict(ns=100)),
    (UNSUP, dict(fmt=4, x_amax=P)), (UNSUP, dict(fmt=4, w_amax=P)), (UNSUP, dict(fmt=3, opts=(1, 0, 0, 0, 0))),
    (UNSUP, dict(fmt=2, x_amax=P, opts=(1, 0, 0, 0, 0)))])
def test_fwd_save_refuses(L, want, kw):
    assert save(L, **kw) == want


def bwd(L, opts=None, **k):
    d = dict(dH=P, lddh=64, T=128, Kin=256, F=64, fmt=0, act=0, gate8=a8(128), up8=a8(128), o=None, saved=P, ns=1 << 30, dX=P, xt=1,
             dW=P, wt=0, ws=P, n=1 << 30)
    assert set(k) <= set(d)
    d.update(k)
    d["o"] = C.byref(mx._CBwdOpts(*opts)) if opts else None
    return L.mx_gated_bwd(*d.values(), None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(T=-1)), (BAD, dict(fmt=-1)), (BAD, dict(act=-1)), (BAD, dict(dH=None)), (BAD, dict(lddh=63)), (BAD, dict(gate8=None)),
    (BAD, dict(up8=None)), (BAD, dict(gate8=a8(127))), (ALIGN, dict(up8=a8(128, codes=P + 8))), (BAD, dict(xt=2)), (BAD, dict(wt=-1)),
    (ALIGN, dict(dH=P + 1)), (ALIGN, dict(dX=P + 8)), (ALIGN, dict(dW=P + 2)), (ALIGN, dict(ws=P + 8)), (ALIGN, dict(Kin=192)),
    (ALIGN, dict(T=96, gate8=a8(96), up8=a8(96))), (ALIGN, dict(F=48, gate8=a8(128, 48), up8=a8(128, 48))),
    (ALIGN, dict(fmt=2)), (WS, dict(ws=None)), (WS, dict(n=1000)), (WS, dict(saved=None)), (WS, dict(ns=1000)),
    (ALIGN, dict(saved=P + 4)), (BAD, dict(opts=(0, 2, 0, 0, 0))), (UNSUP, dict(fmt=3, opts=(1, 0, 0, 0, 0)))])
def test_bwd_refuses(L, want, kw):
    assert bwd(L, **kw) == want


def test_workspace_sizes(L):
    assert L.mx_gated_workspace_bytes(32, 256, 64, 0, 3) == 0
    assert L.mx_gated_workspace_bytes(-1, 256, 64, 0, 0) == 0
    assert L.mx_gated_workspace_bytes(32, 256, 64, 7, 0) == 0
    for fmt in range(5):
        w = [L.mx_gated_workspace_bytes(256, 512, 384, fmt, k) for k in range(3)]
        assert w[0] > w[2] > 0 and w[1] >= 256 * 384 * 4 + L.mx_linear_workspace_bytes(256, 512, 768, fmt, 2)


def test_without_a_gpu(L):
    if torch.cuda.is_available():
        pytest.skip("needs a host without a GPU")
    assert L.mx_gemm_gated(operand(), operand(), operand(), 0, P, 64, None, None, None, None) == mx.MX_ERR_NO_DEVICE
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(128, 256, dtype=torch.bfloat16)
    for call in (lambda: mx.gated_fwd(x, w, "mxfp8"), lambda: mx.gated_fwd_save(x, w, "mxfp8"), lambda: mx.gated_weights(w, "mxfp8")):
        with pytest.raises(mx.MXError) as e:
            call()
        assert e.value.code == mx.MX_ERR_NO_DEVICE


@pytest.mark.gpu
def test_python_side_refusals():
    x = torch.zeros(32, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(128, 256, dtype=torch.bfloat16, device="cuda")
    q = mx.gated_weights(w, "mxfp8")
    calls = [lambda: mx.gated_fwd(x.float(), w, "mxfp8"), lambda: mx.gated_fwd(x, w.float(), "mxfp8"),
             lambda: mx.gated_fwd(x, w[:127], "mxfp8"), lambda: mx.gated_fwd(x, w[:, :128], "mxfp8"),
             lambda: mx.gated_fwd(x, w, "fp8"), lambda: mx.gated_fwd(x, w, "mxfp8", act="relu"),
             lambda: mx.gated_fwd(x, q, "nvfp4"), lambda: mx.gated_fwd(x, (q[0], w), "mxfp8"),
             lambda: mx.gated_fwd(x, w, "mxfp8", out=torch.zeros(32, 63, dtype=torch.bfloat16, device="cuda")),
             lambda: mx.gated_fwd(x, w, "mxfp8", out=torch.zeros(32, 64, device="cuda")),
             lambda: mx.gated_fwd(x, w, "mxfp8", workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")),
             lambda: mx.gated_fwd(x.t().contiguous().t(), w, "mxfp8"),
             lambda: mx.gemm_gated(mx.quantize(x, "mxfp8", hadamard=True), *q),
             lambda: mx.gated_fwd_save(x, w, "mxfp8", x_amax=torch.zeros(2, device="cuda")),
             lambda: mx.gated_fwd_save(x, w, "mxfp8", saved=torch.zeros(8, dtype=torch.uint8, device="cuda")),
             lambda: mx.gated_weights(w.t(), "mxfp8"), lambda: mx.gated_weights(w[:3], "mxfp8")]
    kept = mx.gated_fwd_save(x, w, "mxfp8")
    dh = torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda")
    calls += [lambda: mx.gated_bwd(dh, kept, 256, "mxfp8"),  # 32 tokens: the weight gradient multiplies along them
              lambda: mx.gated_bwd(dh[:16], kept, 256, "mxfp8", need_dw=False),
              lambda: mx.gated_bwd(dh.float(), kept, 256, "mxfp8", need_dw=False),
              lambda: mx.gated_bwd(dh, kept, 256, "mxfp8", need_dw=False, dx_dtype=torch.float16),
              lambda: mx.gated_bwd(dh, kept, 256, "mxfp8", need_dw=False, dX=torch.zeros(32, 512, dtype=torch.bfloat16, device="cuda")[:, :256])]
    for call in calls:
        with pytest.raises(mx.MXError):
            call()
    mx.gated_bwd(dh, kept, 256, "mxfp8", need_dw=False)
