"""What the gradient norm and the AdamW step refuse, before anything is launched."""
import ctypes as C

import pytest
import torch

import fp4_precision_gemms_gb300 as mx

BAD, UNSUP, ALIGN, WS = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED, mx.MX_ERR_ALIGNMENT, mx.MX_ERR_WORKSPACE
P = 1 << 20  # an address that is never read: every call here is refused
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    mx.build()
    return mx.lib()


def step(L, count=1, scale=P, amax=P, tensor=None, opts=None, tensors=True, with_opts=True):
    t = dict(param=P, grad=P, m=P, v=P, m_sf=P, v_sf=P, copy=None, n=100, weight_decay=0.1, p_dtype=0, g_dtype=0, bits=32)
    o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, t=1, lr_at=None, t_at=None, seed=0, rounding=0)
    for d, given in ((t, tensor or {}), (o, opts or {})):
        assert set(given) <= set(d)
        d.update(given)
    row, oo = mx._CAdamwTensor(**t), mx._CAdamwOpts(**o)
    return L.mx_adamw_step(C.pointer(row) if tensors else None, count, C.byref(oo) if with_opts else None, scale, amax, None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(count=-1)), (BAD, dict(tensors=False)), (BAD, dict(with_opts=False)), (BAD, dict(count=1 << 40)),
    (ALIGN, dict(scale=P + 2)), (ALIGN, dict(amax=P + 1)),
] + [(BAD, dict(tensor=t)) for t in (
    dict(param=None), dict(m=None), dict(v=None), dict(n=-1), dict(n=(1 << 34) + 1), dict(bits=16), dict(bits=0),
    dict(p_dtype=2), dict(g_dtype=-1), dict(weight_decay=NAN), dict(weight_decay=INF), dict(bits=8, m_sf=None),
    dict(bits=8, v_sf=None))
] + [(ALIGN, dict(tensor=t)) for t in (
    dict(param=P + 2), dict(grad=P + 2), dict(m=P + 2), dict(v=P + 1), dict(copy=P + 1), dict(bits=8, m=P + 8),
    dict(bits=8, v=P + 4), dict(p_dtype=1, param=P + 1))
] + [(UNSUP, dict(tensor=dict(p_dtype=1, copy=P)))
] + [(BAD, dict(opts=o)) for o in (
    dict(lr=NAN), dict(lr=INF), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=NAN), dict(eps=-1.0),
    dict(eps=NAN), dict(t=0), dict(t=-3), dict(rounding=2))
] + [(ALIGN, dict(opts=o)) for o in (dict(lr_at=P + 2), dict(t_at=P + 4))])
def test_adamw_refuses(L, want, kw):
    assert step(L, **kw) == want


def norm(L, count=1, max_norm=1.0, out=P, ws=P, n=1 << 20, grads=True, **g):
    row = mx._CGrad(**{**dict(data=P, n=100, dtype=0), **g.get("grad", {})})
    return L.mx_grad_norm(C.pointer(row) if grads else None, count, max_norm, out, ws, n, None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(count=-1)), (BAD, dict(grads=False)), (BAD, dict(out=None)), (BAD, dict(max_norm=0.0)),
    (BAD, dict(max_norm=-1.0)), (BAD, dict(max_norm=NAN)), (ALIGN, dict(out=P + 1)), (WS, dict(ws=None)),
    (WS, dict(n=8)), (ALIGN, dict(ws=P + 4)), (BAD, dict(grad=dict(data=None))), (BAD, dict(grad=dict(n=-1))),
    (BAD, dict(grad=dict(n=(1 << 34) + 1))), (BAD, dict(grad=dict(dtype=3))), (ALIGN, dict(grad=dict(data=P + 1)))])
def test_grad_norm_refuses(L, want, kw):
    assert norm(L, **kw) == want


def test_sizes(L):
    assert L.mx_grad_norm_workspace_bytes(-1) == 0
    a, b = L.mx_grad_norm_workspace_bytes(0), L.mx_grad_norm_workspace_bytes(5000)
    assert 0 < a <= b < 1 << 20


def test_python_side_without_a_gpu():
    if torch.cuda.is_available():
        pytest.skip("needs a host without a GPU")
    x = torch.zeros(4)
    with pytest.raises(mx.MXError) as e:
        mx.AdamW([x])
    assert e.value.code == mx.MX_ERR_NO_DEVICE
    with pytest.raises(mx.MXError):
        mx.grad_norm([x])
    for kw in (dict(params=[]), dict(params=[x], state="4bit"), dict(params=[x], rounding="up"),
               dict(params=[x], weight_decay=[0.1, 0.2]), dict(params=[x], copies=[])):
        with pytest.raises(mx.MXError):
            mx.AdamW(**kw)


@pytest.mark.gpu
def test_python_side_refusals():
    p = torch.zeros(64, device="cuda")
    for kw in (dict(params=[p, p]), dict(params=[p[:40], p[32:]]), dict(params=[p.view(8, 8).t()]),
               dict(params=[p.half()]), dict(params=[p.bfloat16()], copies=[p.bfloat16()]),
               dict(params=[p], copies=[torch.zeros(64, device="cuda")]),
               dict(params=[p], copies=[torch.zeros(63, device="cuda", dtype=torch.bfloat16)])):
        with pytest.raises(mx.MXError):
            mx.AdamW(**kw)
    opt = mx.AdamW([p])
    g = torch.zeros(64, device="cuda")
    one = torch.zeros(1, device="cuda")
    for a, kw in (([], {}), ([g, g], {}), ([g[:63]], {}), ([g.half()], {}), ([g.cpu()], {}), ([g.view(8, 8).t()], {}),
                  ([g], dict(grad_scale=one.double())), ([g], dict(grad_scale=torch.zeros(2, device="cuda"))),
                  ([g], dict(amax_out=torch.zeros(2, device="cuda"))), ([g], dict(t=0)), ([g], dict(lr=float("nan"))),
                  ([g], dict(lr=one.double()))):
        with pytest.raises(mx.MXError):
            opt.step(a, **kw)
    assert opt.t == 0 and not p.any()
    p.data = torch.zeros(32, device="cuda")  # another size
    with pytest.raises(mx.MXError):
        opt.step([g])
    with pytest.raises(mx.MXError):
        mx.grad_norm([])
    with pytest.raises(mx.MXError):
        mx.grad_norm([g], max_norm=0.0)
    with pytest.raises(mx.MXError):
        mx.grad_norm([g], out=torch.zeros(3, device="cuda"))
