"""Which memory the operands of a norm call may share: matrices in place, vectors
not, at a shape of every kernel.  Overlapping vectors are refused on the host."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
# few short rows (64x64: dw has the statistics' size too), narrow rows, a CTA's rows, wide rows
SHAPES = [(64, 64), (1, 2048), (200, 256), (70, 4096), (3, 16400)]


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def _refused(mx, outputs, call):
    before = [t.clone() for t in outputs]
    launches = mx.launch_count()
    with pytest.raises(mx.MXError) as e:
        call()
    assert e.value.code == mx.MX_ERR_INVALID_ARG and mx.launch_count() == launches
    assert all(torch.equal(a, b) for a, b in zip(before, outputs))


@pytest.mark.parametrize("shape", SHAPES)
def test_vectors_that_overlap_are_refused(mx, shape):
    rows, cols = shape
    x, dy = (workloads.draw("student_t3", shape, 970 + i, device="cuda") for i in range(2))
    words = torch.ones(2 * max(rows, cols) + 8, device="cuda")  # every vector below lies in here
    at = lambda n, i=0: words[i:i + n]  # noqa: E731
    far = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    w, mean, rstd, one = far(cols), far(rows), far(rows), far(1)
    for k in (0, cols - 1):  # the same memory, and one shared word
        for name in ("dw", "db"):
            _refused(mx, [words], lambda: mx.norm_bwd(dy, x, rstd, mean, at(cols), **{name: at(cols, k)}))
        _refused(mx, [words], lambda: mx.norm_bwd(dy, x, rstd, mean, w, dw=at(cols), db=at(cols, k)))
        _refused(mx, [words], lambda: mx.norm_bwd(dy, x, rstd, mean, at(cols), amax_out=at(1, k)))
        _refused(mx, [words], lambda: mx.norm_bwd(dy, x, rstd, mean, w, dw=at(cols), amax_out=at(1, k)))
        _refused(mx, [words], lambda: mx.norm_fwd(x, w, at(cols), amax_out=at(1, k)))
    _refused(mx, [words], lambda: mx.norm_bwd(dy, x, at(rows), mean, w, dw=at(cols)))
    _refused(mx, [words], lambda: mx.norm_bwd(dy, x, rstd, at(rows), w, db=at(cols, rows - 1)))
    _refused(mx, [words], lambda: mx.norm_bwd(dy, x, rstd, mean, at(cols).view(BF)[:cols], dw=at(cols, (cols - 1) // 2)))
    _refused(mx, [words], lambda: mx.norm_fwd(x, at(cols), mean=at(rows), rstd=rstd))
    _refused(mx, [words], lambda: mx.norm_fwd(x, at(cols), rstd=at(rows, cols - 1), mean=mean))
    _refused(mx, [words], lambda: mx.norm_fwd(x, w, mean=at(rows), rstd=at(rows, rows - 1)))
    _refused(mx, [words], lambda: mx.norm_fwd(x, w, mean=mean, rstd=at(rows), amax_out=at(1, rows - 1)))
    # side by side is apart, and an RMS norm reads no mean
    mx.norm_bwd(dy, x, rstd, mean, at(cols), dw=at(cols, cols), amax_out=one)
    mx.norm_bwd(dy, x, rstd, at(rows), w, kind="rms", dw=at(cols))


@pytest.mark.parametrize("shape", SHAPES)
def test_matrices_in_place_give_the_same_bits(mx, shape):
    rows, cols = shape
    x, r, dy, ds = (workloads.draw(k, shape, 980 + i, device="cuda")
                    for i, k in enumerate(("student_t3", "normal", "student_t3", "normal")))
    w = workloads.draw("normal", (1, cols), 990, device="cuda").float()[0]
    f = mx.norm_fwd(x, w, residual=r)
    a, b = x.clone(), r.clone()
    g = mx.norm_fwd(a, w, residual=b, sum_out=b, out=a)
    assert torch.equal(f.y, a) and torch.equal(f.sum, b) and torch.equal(f.rstd, g.rstd)
    want = mx.norm_bwd(dy, f.sum, f.rstd, f.mean, w, dres=ds)
    for k in range(3):
        t = [dy.clone(), f.sum.clone(), ds.clone()]
        got = mx.norm_bwd(t[0], t[1], f.rstd, f.mean, w, dres=t[2], dx=t[k])
        assert all(torch.equal(p, q) for p, q in zip(want, got)), k
