"""Layer norm and RMS norm, forward and backward, against their plain forms in
64 bits within first-order rounding bounds; gradients also against differences."""
import pytest
import torch

import ops_ref as ref
import workloads

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
COLS = [1, 7, 32, 33, 64, 100, 128, 255, 256, 520, 1000, 1024, 1531, 2048, 4096, 4099, 5120, 8192, 12288, 16384, 16400,
        33000]


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def _x(rows, cols, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(torch.randn(1, cols, generator=g, device="cuda"))
    return (x + 0.3).to(dtype)


def _wb(cols, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(dtype),
            (0.3 * torch.randn(cols, generator=g, device="cuda")).to(dtype))


def _check_fwd(r, s, w, b, kind, eps, y_dtype, amax):
    y, mean, rstd = ref.norm_fwd(s, w, b, kind, eps)
    by, bm, br = ref.norm_fwd_bounds(s, w, b, kind, eps, y_dtype)
    assert r.y.dtype is y_dtype
    ref.assert_within(r.y, y, by, "y")
    ref.assert_within(r.rstd, rstd, br, "rstd")
    if kind == "layer":
        ref.assert_within(r.mean, mean, bm, "mean")
    else:
        assert r.mean is None
    if amax is not None:
        assert amax.item() == r.y.float().abs().max().item()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("types", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("cols", COLS)
def test_forward(mx, cols, types, kind):
    """Residual addition, checkpoint, maximum and statistics together."""
    tx, ty = types
    rows = 5 if cols > 2000 else 37
    x, r = _x(rows, cols, tx, 1), _x(rows, cols, tx, 2)
    w, b = _wb(cols, F32, 3)
    amax = torch.full((1,), 9e9, device="cuda")
    out = mx.norm_fwd(x, w, b, kind=kind, residual=r, save=True, amax_out=amax, out_dtype=ty)
    s = (x.float() + r.float()).to(tx)
    assert torch.equal(out.sum, s)
    _check_fwd(out, s, w, b, kind, 1e-5, ty, amax)
    alone = mx.act8_save(s)
    assert torch.equal(out.saved.codes, alone.codes) and torch.equal(out.saved.sf, alone.sf)


@pytest.mark.parametrize("how", ["dense", "wide", "odd"])
@pytest.mark.parametrize("wdtype", [BF, F32, None])
@pytest.mark.parametrize("cols", [31, 128, 200, 1024, 4096, 4104])
def test_forward_layouts_and_parameters(mx, cols, wdtype, how):
    rows = 23
    x = ref.layout(_x(rows, cols, BF, 4), how)
    w, b = _wb(cols, wdtype, 5) if wdtype else (None, None)
    wide = torch.full((rows, cols + 24), 5.0, dtype=BF, device="cuda")
    at = 8 if how == "wide" else 3
    out = mx.norm_fwd(x, w, b, out=wide[:, at:at + cols])
    _check_fwd(out, x, w, b, "layer", 1e-5, BF, None)
    assert (wide[:, :at] == 5).all() and (wide[:, at + cols:] == 5).all()
    if w is not None:  # weight without bias, bias without weight
        _check_fwd(mx.norm_fwd(x, w, None), x, w, None, "layer", 1e-5, BF, None)
        _check_fwd(mx.norm_fwd(x, None, b), x, None, b, "layer", 1e-5, BF, None)


@pytest.mark.parametrize("rows", [1, 2, 3, 151, 1217, 9001])
@pytest.mark.parametrize("cols", [48, 128, 1024])
def test_forward_row_counts(mx, rows, cols):
    x = _x(rows, cols, BF, 6)
    w, b = _wb(cols, F32, 7)
    _check_fwd(mx.norm_fwd(x, w, b), x, w, b, "layer", 1e-5, BF, None)


@pytest.mark.parametrize("cols", [129, 1024, 4096])
def test_a_large_mean_does_not_cost_the_variance(mx, cols):
    """Rows of 1000 +- 1: the variance is summed around the mean."""
    x = 1000.0 + _x(9, cols, F32, 8)
    out = mx.norm_fwd(x, out_dtype=F32)
    _check_fwd(out, x, None, None, "layer", 1e-5, F32, None)
    assert (out.y.double().std(1, correction=0) - 1).abs().max() < 1e-3


@pytest.mark.parametrize("cols", [33, 512, 4096])
def test_constant_and_non_finite_rows(mx, cols):
    x = _x(6, cols, BF, 9)
    x[1] = 0.0
    x[2] = 3.0
    x[3, cols // 2] = float("nan")
    x[4, 0] = float("inf")
    out = mx.norm_fwd(x, save=True)
    assert (out.y[1] == 0).all() and (out.y[2] == 0).all()
    assert torch.isnan(out.y[3]).all() and torch.isnan(out.y[4]).all()
    keep = [0, 1, 2, 5]
    y, _, _ = ref.norm_fwd(x[keep], None, None, "layer", 1e-5)
    ref.assert_within(out.y[keep], y, ref.norm_fwd_bounds(x[keep], None, None, "layer", 1e-5, BF)[0], "others")
    assert torch.isnan(mx.act8_restore(out.saved)[3, cols // 2])
    amax = torch.zeros(1, device="cuda")
    mx.norm_fwd(x, amax_out=amax)
    assert torch.isnan(amax).all()


@pytest.mark.parametrize("cols", [40, 1000, 4096, 4099])
def test_in_place(mx, cols):
    """The stream updated in place, the output over the input."""
    x, r = _x(300, cols, BF, 10), _x(300, cols, BF, 11)
    w, b = _wb(cols, F32, 12)
    want = mx.norm_fwd(x, w, b, residual=r)
    r2 = r.clone()
    got = mx.norm_fwd(x, w, b, residual=r2, sum_out=r2)
    assert torch.equal(r2, want.sum) and torch.equal(got.y, want.y)
    x2 = want.sum.clone()
    assert torch.equal(mx.norm_fwd(x2, w, b, out=x2).y, want.y)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("source", ["x", "act8"])
@pytest.mark.parametrize("types", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("cols", COLS)
def test_backward(mx, cols, types, source, kind):
    tx, ty = types
    rows = 5 if cols > 2000 else 37
    s = _x(rows, cols, tx, 20)
    w, _ = _wb(cols, F32, 21)
    dy = workloads.draw("student_t3", (rows, cols), 22, 1e-3, device="cuda").to(ty)
    dres = workloads.draw("student_t3", (rows, cols), 23, 1e-3, device="cuda").to(tx)
    _, mean, rstd = ref.norm_fwd(s, w, None, kind, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    kept = mx.act8_save(s) if source == "act8" else s
    sv = ref.decode(kept.codes, kept.sf, cols) if source == "act8" else s
    amax = torch.full((1,), 9e9, device="cuda")
    dx, dw, db = mx.norm_bwd(dy, kept, rstd, mean if kind == "layer" else None, w, kind=kind, dres=dres, need_db=True,
                             dx_dtype=tx, amax_out=amax)
    want = ref.norm_bwd(dy, sv, mean, rstd, w, kind, dres)
    bound = ref.norm_bwd_bounds(dy, sv, mean, rstd, w, kind, dres, tx)
    assert dx.dtype is tx and dw.dtype is F32 and db.dtype is F32
    for g, v, b, n in zip((dx, dw, db), want, bound, ("dx", "dw", "db")):
        ref.assert_within(g, v, b, n)
    assert amax.item() == dx.float().abs().max().item()


@pytest.mark.parametrize("rows", [1, 2, 7, 64, 153, 1217, 5003])
@pytest.mark.parametrize("cols", [64, 200, 1024, 1531])
def test_backward_row_counts(mx, rows, cols):
    """The reductions over few and many rows, with and without each output; the
    same call twice gives the same bits."""
    s = _x(rows, cols, BF, 24)
    w, _ = _wb(cols, BF, 25)
    dy = workloads.draw("student_t3", (rows, cols), 26, 1e-3, device="cuda")
    _, mean, rstd = ref.norm_fwd(s, w, None, "layer", 1e-5)
    mean, rstd = mean.float(), rstd.float()
    got = mx.norm_bwd(dy, s, rstd, mean, w)
    want = ref.norm_bwd(dy, s, mean, rstd, w, "layer", None)
    bound = ref.norm_bwd_bounds(dy, s, mean, rstd, w, "layer", None, BF)
    for g, v, b, n in zip(got, want, bound, ("dx", "dw", "db")):
        ref.assert_within(g, v, b, n)
    for dw, db in ((True, True), (True, False), (False, True), (False, False)):
        part = mx.norm_bwd(dy, s, rstd, mean, w, need_dw=dw, need_db=db)
        assert torch.equal(part[0], got[0])
        assert (part[1] is None) != dw and (part[2] is None) != db
        assert not dw or torch.equal(part[1], got[1])
        assert not db or torch.equal(part[2], got[2])


@pytest.mark.parametrize("how", ["dense", "wide", "odd"])
@pytest.mark.parametrize("cols", [31, 128, 200, 1024, 4096])
def test_backward_layouts_and_in_place(mx, cols, how):
    rows = 40
    s, dyv = _x(rows, cols, BF, 27), workloads.draw("student_t3", (rows, cols), 28, 1e-3, device="cuda")
    _, mean, rstd = ref.norm_fwd(s, None, None, "layer", 1e-5)
    mean, rstd = mean.float(), rstd.float()
    want = ref.norm_bwd(dyv, s, mean, rstd, None, "layer", None)
    bound = ref.norm_bwd_bounds(dyv, s, mean, rstd, None, "layer", None, BF)
    dy = ref.layout(dyv, how)
    wide = torch.full((rows, cols + 24), 5.0, dtype=BF, device="cuda")
    at = 8 if how == "wide" else 3
    got = mx.norm_bwd(dy, ref.layout(s, how), rstd, mean, dx=wide[:, at:at + cols])
    for g, v, b in zip(got, want, bound):
        ref.assert_within(g, v, b, how)
    assert (wide[:, :at] == 5).all() and (wide[:, at + cols:] == 5).all()
    apart = mx.norm_bwd(dy, ref.layout(s, how), rstd, mean, dx=torch.empty_strided((rows, cols), dy.stride(), dtype=BF,
                                                                                   device="cuda"))
    got2 = mx.norm_bwd(dy, ref.layout(s, how), rstd, mean, dx=dy)  # dx over dy
    assert torch.equal(dy, apart[0]) and torch.equal(got2[1], apart[1]) and torch.equal(got2[2], apart[2])


@pytest.mark.parametrize("shape", [(64, 2048), (65, 2048), (64, 2056), (3, 9), (64, 31)])
@pytest.mark.parametrize("over", ["dy", "x", None])
def test_backward_around_the_few_row_rule(mx, shape, over):
    """Both sides of the rule that picks the one-launch kernel, dx apart from,
    over dy and over x, from the input and from the checkpoint."""
    rows, cols = shape
    s, dy = _x(rows, cols, BF, 60), workloads.draw("student_t3", (rows, cols), 61, 1e-3, device="cuda")
    w, _ = _wb(cols, F32, 62)
    _, mean, rstd = ref.norm_fwd(s, w, None, "layer", 1e-5)
    mean, rstd = mean.float(), rstd.float()
    for kept in (s.clone(), mx.act8_save(s)):
        sv = s if torch.is_tensor(kept) else ref.decode(kept.codes, kept.sf, cols)
        d = dy.clone()
        dx = d if over == "dy" else kept if over == "x" and torch.is_tensor(kept) else None
        got = mx.norm_bwd(d, kept, rstd, mean, w, dx=dx, dx_dtype=BF)
        want = ref.norm_bwd(dy, sv, mean, rstd, w, "layer", None)
        bound = ref.norm_bwd_bounds(dy, sv, mean, rstd, w, "layer", None, BF)
        for g, v, b, n in zip(got, want, bound, ("dx", "dw", "db")):
            ref.assert_within(g, v, b, n)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("cols", [5, 40])
def test_gradients_against_differences(mx, cols, kind):
    """Central differences, step 1e-5 in 64 bits, of L = sum(dy y) + sum(dres s):
    their own error is about 1e-10 times the third derivatives, which rows of
    spread 1 keep below 1e4; the call's fp32 error adds 1e-5 of the largest
    gradient at these sizes."""
    rows, h = 3, 1e-5
    s, dres = _x(rows, cols, F32, 30), _x(rows, cols, F32, 31)
    w, b = _wb(cols, F32, 32)
    dy = _x(rows, cols, F32, 33)
    f = mx.norm_fwd(s, w, b, kind=kind, out_dtype=F32)
    dx, dw, db = mx.norm_bwd(dy, s, f.rstd, f.mean, w, kind=kind, dres=dres, need_db=True)

    def loss(s_, w_, b_):
        return ((dy.double() * ref.norm_fwd(s_, w_, b_, kind, 1e-5)[0]).sum() + (dres.double() * s_).sum()).item()

    base = [s.double(), w.double(), b.double()]
    for at, grad in enumerate((dx, dw, db)):
        num = torch.zeros_like(grad, dtype=torch.float64)
        for i in range(grad.numel()):
            v = []
            for sign in (1, -1):
                args = [t.clone() for t in base]
                args[at].view(-1)[i] += sign * h
                v.append(loss(*args))
            num.view(-1)[i] = (v[0] - v[1]) / (2 * h)
        assert (grad.double() - num).abs().max() <= 2e-5 * num.abs().max() + 1e-6


@pytest.mark.parametrize("shape", [(0, 64), (5, 0), (0, 0)])
def test_empty(mx, shape):
    rows, cols = shape
    x = torch.empty(shape, dtype=BF, device="cuda")
    amax = torch.full((1,), 3.0, device="cuda")
    out = mx.norm_fwd(x, save=True, amax_out=amax)
    assert out.y.shape == shape and amax.item() == 0
    dx, dw, db = mx.norm_bwd(x, x, torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"),
                             dw=torch.full((cols,), 3.0, device="cuda"), db=torch.full((cols,), 3.0, device="cuda"))
    assert dx.shape == shape and (dw == 0).all() and (db == 0).all()


def test_training_without_affine_rows_independent(mx):
    """A row's results do not depend on the rows around it."""
    x = _x(700, 4096, BF, 40)
    whole = mx.norm_fwd(x, save=True)
    part = mx.norm_fwd(x[13:14], save=True)
    assert torch.equal(whole.y[13:14], part.y) and torch.equal(whole.rstd[13:14], part.rstd)
    assert torch.equal(whole.saved.codes[13:14], part.saved.codes)


@pytest.mark.parametrize("row", [0, 1, 3])
@pytest.mark.parametrize("types", [(BF, 4096), (F32, 16384)])
def test_a_wait_that_runs_out_is_reported(mx, types, row):
    """The hook lets one thread of every CTA give up; the status word says so,
    nothing hangs, and the next calls are right."""
    dtype, cols = types
    x = _x(2000, cols, dtype, 50)
    good = mx.norm_fwd(x)
    want = mx.norm_bwd(x, x, good.rstd, good.mean, dres=x)
    for call in (lambda: mx.norm_fwd(x, residual=x), lambda: mx.norm_fwd(x, kind="rms"),
                 lambda: mx.norm_bwd(x, x, good.rstd, good.mean, dres=x)):
        mx.set_norm_fail_at(row)
        try:
            call()
        finally:
            mx.set_norm_fail_at(-1)
        assert mx.last_device_status() == mx.MX_ERR_TIMEOUT
    assert torch.equal(mx.norm_fwd(x).y, good.y)
    got = mx.norm_bwd(x, x, good.rstd, good.mean, dres=x)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert mx.last_device_status() == mx.MX_OK
