"""What the norm, activation and checkpoint calls refuse, before anything is
launched: argument errors are found on the host and need no GPU (bad arguments
are refused before the device is looked at), sizes are plain functions."""
import ctypes as C

import pytest
import torch

import fp4_precision_gemms_gb300 as mx
from conftest import gpu_available

BAD, UNSUP, ALIGN, WS = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED, mx.MX_ERR_ALIGNMENT, mx.MX_ERR_WORKSPACE
P = 1 << 20  # an address that is never read: every call here is refused


@pytest.fixture(scope="module")
def L():
    mx.build()
    return mx.lib()


def a8(rows=4, cols=64, codes=P, sf=P):
    return mx._CAct8(codes, sf, rows, cols)


def test_sizes(L):
    for rows, cols, G in ((1, 1, 1), (3, 32, 1), (5, 33, 2), (8192, 14336, 448), (2 ** 20, 4099, 129)):
        assert L.mx_act8_codes_bytes(rows, cols) == rows * G * 32
        assert L.mx_act8_sf_bytes(rows, cols) == rows * G
    for rows, cols in ((0, 64), (64, 0), (-1, 64), (64, -1), (1, 2 ** 31), (2 ** 60, 64)):
        assert L.mx_act8_codes_bytes(rows, cols) == 0
        assert L.mx_norm_bwd_workspace_bytes(rows, cols) == 0
    assert L.mx_norm_bwd_workspace_bytes(64, 2048) == 0  # few short rows need none
    for rows in (1, 100, 10 ** 6):
        n = L.mx_norm_bwd_workspace_bytes(rows, 4096)
        assert n >= 2 * 4096 * 4 and n <= 1 << 28


def norm_fwd(L, **k):
    d = dict(x=P, ldx=64, residual=None, ldr=0, xt=1, rows=4, cols=64, kind=0, w=P, b=P, wt=0, eps=1e-5, sum_out=None,
             lds=0, y=P, ldy=64, yt=1, mean=P, rstd=P, save=None, amax=P)
    assert set(k) <= set(d)
    d.update(k)
    return L.mx_norm_fwd(*d.values(), None)


def norm_bwd(L, **k):
    d = dict(dy=P, ldy=64, yt=1, x=P, ldx=64, x8=None, mean=P, rstd=P, w=P, wt=0, rows=4, cols=64, kind=0, dres=None,
             ldres=0, dx=P, lddx=64, xt=1, dw=P, db=P, amax=None, ws=P, n=1 << 30)
    assert set(k) <= set(d)
    d.update(k)
    return L.mx_norm_bwd(*d.values(), None)


def act_fwd(L, **k):
    d = dict(gate=P, ldg=64, up=P, ldu=64, rows=4, cols=64, act=0, dt=1, h=P, ldh=64, gate8=None, up8=None, amax=None)
    assert set(k) <= set(d)
    d.update(k)
    return L.mx_act_fwd(*d.values(), None)


def act_bwd(L, **k):
    d = dict(dh=P, ldh=64, gate=P, ldg=64, up=P, ldu=64, gate8=None, up8=None, rows=4, cols=64, act=0, dt=1, dgate=P,
             lddg=64, dup=P, lddu=64, amax=None)
    assert set(k) <= set(d)
    d.update(k)
    return L.mx_act_bwd(*d.values(), None)


@pytest.mark.parametrize("why,code,args", [
    ("null x", BAD, dict(x=None)), ("null y", BAD, dict(y=None)), ("negative rows", BAD, dict(rows=-1)),
    ("negative cols", BAD, dict(cols=-1)), ("too many cols", BAD, dict(cols=2 ** 31)), ("short stride", BAD, dict(ldx=63)),
    ("short y stride", BAD, dict(ldy=8)), ("bad x type", BAD, dict(xt=2)), ("bad y type", BAD, dict(yt=-1)),
    ("bad weight type", BAD, dict(wt=5)), ("bad kind", BAD, dict(kind=2)), ("negative eps", BAD, dict(eps=-1.0)),
    ("NaN eps", BAD, dict(eps=float("nan"))), ("residual without sum", BAD, dict(residual=P, ldr=64)),
    ("sum without residual", BAD, dict(sum_out=P, lds=64)), ("checkpoint of another shape", BAD, dict(save=a8(cols=32))),
    ("checkpoint without codes", BAD, dict(save=a8(codes=None))), ("misaligned codes", ALIGN, dict(save=a8(codes=P + 8))),
    ("misaligned x", ALIGN, dict(x=P + 1)), ("misaligned fp32 y", ALIGN, dict(y=P + 2, yt=0)),
    ("misaligned weight", ALIGN, dict(w=P + 2)), ("misaligned statistics", ALIGN, dict(rstd=P + 2)),
    ("misaligned amax", ALIGN, dict(amax=P + 1)), ("overflowing extent", BAD, dict(rows=2 ** 40, ldx=2 ** 40))])
def test_norm_fwd_refuses(L, why, code, args):
    assert norm_fwd(L, **args) == code, why


@pytest.mark.parametrize("why,code,args", [
    ("null dy", BAD, dict(dy=None)), ("null dx", BAD, dict(dx=None)), ("no input at all", BAD, dict(x=None)),
    ("x and a checkpoint", BAD, dict(x8=a8())), ("no rstd", BAD, dict(rstd=None)), ("no mean", BAD, dict(mean=None)),
    ("bad kind", BAD, dict(kind=-1)), ("bad type", BAD, dict(xt=7)), ("short stride", BAD, dict(ldx=2)),
    ("short dres", BAD, dict(dres=P, ldres=1)), ("another checkpoint", BAD, dict(x=None, x8=a8(rows=5))),
    ("misaligned dx", ALIGN, dict(dx=P + 1)), ("misaligned dw", ALIGN, dict(dw=P + 2)),
    ("misaligned workspace", ALIGN, dict(ws=P + 4)), ("no workspace", WS, dict(ws=None, rows=100)),
    ("short workspace", WS, dict(n=16, rows=100))])
def test_norm_bwd_refuses(L, why, code, args):
    assert norm_bwd(L, **args) == code, why


def test_norm_bwd_takes_no_workspace_a_byte_short(L):
    n = L.mx_norm_bwd_workspace_bytes(100, 64)
    assert n > 0 and norm_bwd(L, rows=100, n=n - 1) == WS


@pytest.mark.parametrize("why,code,args", [
    ("null gate", BAD, dict(gate=None)), ("null h", BAD, dict(h=None)), ("bad act", BAD, dict(act=3)),
    ("bad type", BAD, dict(dt=2)), ("short stride", BAD, dict(ldu=1)), ("up8 without up", BAD, dict(up=None, up8=a8())),
    ("another checkpoint", BAD, dict(gate8=a8(rows=3))), ("misaligned", ALIGN, dict(gate=P + 1)),
    ("misaligned amax", ALIGN, dict(amax=P + 2))])
def test_act_fwd_refuses(L, why, code, args):
    assert act_fwd(L, **args) == code, why


@pytest.mark.parametrize("why,code,args", [
    ("null dh", BAD, dict(dh=None)), ("null dgate", BAD, dict(dgate=None)), ("null dup", BAD, dict(dup=None)),
    ("dup without up", BAD, dict(up=None)), ("gate kept, up saved", BAD, dict(up=None, up8=a8())),
    ("gate twice", BAD, dict(gate8=a8())), ("gate saved, up kept", BAD, dict(gate=None, gate8=a8())),
    ("nothing", BAD, dict(gate=None)), ("bad act", BAD, dict(act=-1)),
    ("another checkpoint", BAD, dict(gate=None, up=None, gate8=a8(), up8=a8(cols=65))),
    ("misaligned", ALIGN, dict(dup=P + 1))])
def test_act_bwd_refuses(L, why, code, args):
    assert act_bwd(L, **args) == code, why


def test_act8_refuses(L):
    assert L.mx_act8_save(P, 64, 1, None, None) == BAD
    assert L.mx_act8_save(None, 64, 1, a8(), None) == BAD
    assert L.mx_act8_save(P, 63, 1, a8(), None) == BAD
    assert L.mx_act8_save(P, 64, 3, a8(), None) == BAD
    assert L.mx_act8_save(P + 2, 64, 0, a8(), None) == ALIGN
    assert L.mx_act8_save(P, 64, 1, a8(codes=P + 1), None) == ALIGN
    assert L.mx_act8_save(P, 64, 1, a8(sf=None), None) == BAD
    assert L.mx_act8_restore(None, P, 64, 1, None) == BAD
    assert L.mx_act8_restore(a8(), None, 64, 1, None) == BAD
    assert L.mx_act8_restore(a8(rows=-1), P, 64, 1, None) == BAD


@pytest.mark.skipif(gpu_available(), reason="checks the no-GPU error path")
def test_valid_calls_without_a_gpu_say_so(L):
    assert norm_fwd(L) == mx.MX_ERR_NO_DEVICE and norm_bwd(L) == mx.MX_ERR_NO_DEVICE
    assert act_fwd(L) == mx.MX_ERR_NO_DEVICE and act_bwd(L) == mx.MX_ERR_NO_DEVICE
    assert L.mx_act8_save(P, 64, 1, a8(), None) == mx.MX_ERR_NO_DEVICE
    with pytest.raises(mx.MXError):
        mx.norm_fwd(torch.zeros(2, 32))


@pytest.mark.gpu
def test_the_binding_refuses_tensors_that_do_not_fit():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    v, rs = torch.ones(64, device="cuda"), torch.ones(4, device="cuda")
    g = mx.act8_save(x)
    y, ry = torch.zeros(100, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(100, device="cuda")
    calls = [
        lambda: mx.norm_fwd(x[0]), lambda: mx.norm_fwd(x.half()), lambda: mx.norm_fwd(x.t()),
        lambda: mx.norm_fwd(x[:1].expand(4, 64)),  # rows that share memory have no row stride
        lambda: mx.norm_fwd(x, v[:63]), lambda: mx.norm_fwd(x, v, v.bfloat16()), lambda: mx.norm_fwd(x, kind="batch"),
        lambda: mx.norm_fwd(x, residual=x.float()), lambda: mx.norm_fwd(x, sum_out=x), lambda: mx.norm_fwd(x, v.cpu()),
        lambda: mx.norm_fwd(x, amax_out=v), lambda: mx.norm_fwd(x, save=mx.Act8.empty(4, 32)),
        lambda: mx.norm_bwd(x, x, rs), lambda: mx.norm_bwd(x, x, rs[:3], rs), lambda: mx.norm_bwd(x, x.float(), rs, rs, dx=x),
        lambda: mx.norm_bwd(y, y, ry, ry, workspace=torch.empty(4, dtype=torch.uint8, device="cuda")),
        lambda: mx.norm_bwd(x, mx.Act8(g.codes, g.sf, 65), rs, rs),
        lambda: mx.act_fwd(x, x[:, :32]), lambda: mx.act_fwd(x, act="relu"), lambda: mx.act_fwd(x, x.float()),
        lambda: mx.act_bwd(x, g, x), lambda: mx.act_bwd(x, x, g), lambda: mx.act_bwd(x, x, dup=x),
        lambda: mx.act_bwd(x.float(), x), lambda: mx.act8_save(x, out=mx.Act8.empty(3, 64)),
        lambda: mx.act8_restore(mx.Act8(g.codes[:, :32], g.sf, 64)),
        lambda: mx.norm_fwd(x.cpu())]
    for i, f in enumerate(calls):
        with pytest.raises(mx.MXError):
            f()
            pytest.fail(f"call {i} was not refused")
