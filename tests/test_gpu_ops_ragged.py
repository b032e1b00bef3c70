"""Rows at any address: every offset and stride modulo 16 bytes, rows shorter than
a 16-byte word, odd widths up to the widest kernels, in place, with sentinels
around every output.  Values outside the matrix are NaN, so that one used by
mistake shows."""
import pytest
import torch

import ops_ref as ref
import workloads

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def _at(t, offset, gap):
    """t in rows `gap` elements apart that start `offset` elements past a 16-byte
    boundary, NaN all around."""
    rows, cols = t.shape
    base = torch.full((rows * (cols + gap) + 64,), float("nan"), dtype=t.dtype, device=t.device)
    v = base[16 + offset:].as_strided((rows, cols), (cols + gap, 1))
    v.copy_(t)
    return v, base


def _room(rows, cols, dtype, offset, gap):
    base = torch.full((rows * (cols + gap) + 64,), 7.0, dtype=dtype, device="cuda")
    v = base[16 + offset:].as_strided((rows, cols), (cols + gap, 1))
    return v, base


def _untouched(base, v):
    """Only the view's own elements differ from the sentinel."""
    mask = torch.ones_like(base, dtype=torch.bool)
    mask[v.storage_offset():].as_strided(v.shape, v.stride()).fill_(False)
    return bool((base[mask] == 7.0).all())


OFFSETS = [(o, g) for o in (0, 1, 2, 3, 5, 7) for g in (0, 1, 4, 9)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(40, 1), (40, 3), (33, 7), (9, 31), (5, 300), (4, 1001)])
def test_activation_and_checkpoint_at_every_offset(mx, shape, dtype):
    """The same bits as from dense rows on a boundary, at every offset."""
    rows, cols = shape
    d = [workloads.draw(k, shape, 700 + i, device="cuda").to(dtype) for i, k in enumerate(("student_t3", "normal", "normal"))]
    pad = torch.zeros(rows, (cols + 7) // 8 * 8 + 8, dtype=dtype, device="cuda")  # rows on 16-byte boundaries
    flat = [pad.clone()[:, :cols].copy_(t) for t in d]
    want = mx.act_fwd(flat[0], flat[1], save=True)
    wg, wu = mx.act_bwd(flat[2], flat[0], flat[1])
    w8g, w8u = mx.act_bwd(flat[2], want.gate, want.up)
    for o, g in OFFSETS:
        (gate, _), (up, _), (dh, _) = _at(d[0], o, g), _at(d[1], (o + 3) % 8, g), _at(d[2], (o * 5) % 8, g + 1)
        h, hb = _room(rows, cols, dtype, (o + 1) % 8, g)
        r = mx.act_fwd(gate, up, save=True, out=h)
        assert torch.equal(h, want.h) and _untouched(hb, h)
        assert torch.equal(r.gate.codes, want.gate.codes) and torch.equal(r.up.sf, want.up.sf)
        (dg, gb), (du, ub) = _room(rows, cols, dtype, o, g), _room(rows, cols, dtype, (o + 5) % 8, g)
        mx.act_bwd(dh, gate, up, dgate=dg, dup=du)
        assert torch.equal(dg, wg) and torch.equal(du, wu) and _untouched(gb, dg) and _untouched(ub, du)
        mx.act_bwd(dh, r.gate, r.up, dgate=dg, dup=du)
        assert torch.equal(dg, w8g) and torch.equal(du, w8u) and _untouched(gb, dg) and _untouched(ub, du)
        back, bb = _room(rows, cols, dtype, o, g)
        mx.act8_restore(r.gate, out=back)
        assert torch.equal(back, mx.act8_restore(want.gate, out_dtype=dtype)) and _untouched(bb, back)
        mx.act_bwd(dh, gate, up, dgate=gate, dup=dh)  # in place: over gate and over dh
        assert torch.equal(gate, wg) and torch.equal(dh, wu)


@pytest.mark.parametrize("types", [(BF, BF), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("shape", [(70, 1), (70, 3), (70, 7), (70, 31), (66, 300), (70, 513), (67, 1001), (5, 8191)])
def test_norm_at_offsets(mx, shape, types):
    tx, ty = types
    rows, cols = shape
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda t: torch.randn(rows, cols, generator=g, device="cuda").add(0.3).to(t)  # noqa: E731
    x, r, dy, dres = n(tx), n(tx), n(ty), n(tx)
    wide = torch.randn(2, cols + 1, generator=g, device="cuda")
    w, b = 1 + 0.1 * wide[0, 1:], wide[1, 1:].contiguous()
    w_odd = torch.empty(cols + 1, device="cuda")[1:].copy_(w)  # parameters at an odd address too
    s = (x.float() + r.float()).to(tx)
    y, mean, rstd = ref.norm_fwd(s, w, b, "layer", 1e-5)
    by, bm, br = ref.norm_fwd_bounds(s, w, b, "layer", 1e-5, ty)
    m32, r32 = mean.float(), rstd.float()
    for i, (o, gap) in enumerate(OFFSETS[:: 1 if cols < 400 else 5]):
        (xv, _), (rv, _) = _at(x, o, gap), _at(r, (o + 3) % 8, gap)
        (out, ob), (sm, sb) = _room(rows, cols, ty, (o + 1) % 8, gap), _room(rows, cols, tx, (o + 6) % 8, gap)
        f = mx.norm_fwd(xv, w_odd if i % 2 else w, b, residual=rv, sum_out=sm, out=out, save=True)
        assert torch.equal(sm, s) and _untouched(ob, out) and _untouched(sb, sm)
        ref.assert_within(out, y, by, "y")
        ref.assert_within(f.mean, mean, bm, "mean")
        ref.assert_within(f.rstd, rstd, br, "rstd")
        assert torch.equal(f.saved.codes, mx.act8_save(s).codes)
        (dv, _), (sv, _), (qv, _) = _at(dy, (o * 3) % 8, gap), _at(s, (o + 2) % 8, gap), _at(dres, (o + 7) % 8, gap)
        for kept in (sv, f.saved):
            vals = s if torch.is_tensor(kept) else ref.decode(kept.codes, kept.sf, cols)
            want = ref.norm_bwd(dy, vals, m32, r32, w, "layer", dres)
            bound = ref.norm_bwd_bounds(dy, vals, m32, r32, w, "layer", dres, tx)
            dx, db_ = _room(rows, cols, tx, o, gap)
            got = mx.norm_bwd(dv, kept, r32, m32, w_odd if i % 2 else w, dres=qv, dx=dx)
            assert _untouched(db_, dx)
            for a, v, bd, name in zip(got, want, bound, ("dx", "dw", "db")):
                ref.assert_within(a, v, bd, name)


@pytest.mark.parametrize("cols", [8193, 9001, 12287, 16383, 16385])
@pytest.mark.parametrize("types", [(BF, BF), (F32, F32)])
def test_norm_at_odd_widths_above_8192(mx, cols, types):
    tx, ty = types
    rows = 70
    g = torch.Generator(device="cuda").manual_seed(4)
    s, dy, dres = (torch.randn(rows, cols, generator=g, device="cuda").to(t) for t in (tx, ty, tx))
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    f = mx.norm_fwd(s, w, None, save=True, out_dtype=ty)
    y, mean, rstd = ref.norm_fwd(s, w, None, "layer", 1e-5)
    by, _, _ = ref.norm_fwd_bounds(s, w, None, "layer", 1e-5, ty)
    ref.assert_within(f.y, y, by, "y")
    assert torch.equal(f.saved.codes, mx.act8_save(s).codes)
    m32, r32 = mean.float(), rstd.float()
    for kept in (s, f.saved):
        vals = s if torch.is_tensor(kept) else ref.decode(kept.codes, kept.sf, cols)
        got = mx.norm_bwd(dy, kept, r32, m32, w, dres=dres, dx_dtype=tx)
        want = ref.norm_bwd(dy, vals, m32, r32, w, "layer", dres)
        bound = ref.norm_bwd_bounds(dy, vals, m32, r32, w, "layer", dres, tx)
        for a, v, bd, name in zip(got, want, bound, ("dx", "dw", "db")):
            ref.assert_within(a, v, bd, name)


def test_a_call_first_made_inside_a_capture(mx):
    """No kernel needs a first call outside a graph: a fresh process captures one."""
    import subprocess
    import sys

    code = """
import sys; sys.path.insert(0, '.')
import torch, fp4_precision_gemms_gb300 as mx
x = torch.randn(200, 4096, device='cuda').bfloat16(); torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    am = torch.empty(1, device='cuda')
    f = mx.norm_fwd(x, save=True, amax_out=am)
    dx, dw, db = mx.norm_bwd(f.y, f.saved, f.rstd, f.mean)
    a = mx.act_fwd(x[:, :2048], x[:, 2048:], save=True)
g.replay(); torch.cuda.synchronize()
e = mx.norm_fwd(x, save=True)
assert torch.equal(e.y, f.y) and am.item() == e.y.abs().max().item()
assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), mx.norm_bwd(e.y, e.saved, e.rstd, e.mean)))
print('captured')
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert "captured" in r.stdout, r.stderr[-2000:]
