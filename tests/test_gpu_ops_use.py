"""How the norm, activation and checkpoint calls are used: on side streams, in
CUDA graphs, with offsets past 2^31 elements, and with their maxima handed to the
quantization that follows."""
import pytest
import torch

import ops_ref as ref
import workloads

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def _all(mx, x, r, w, b, dh):
    """Every call once; a flat list of outputs."""
    am = torch.empty(1, device="cuda")
    f = mx.norm_fwd(x, w, b, residual=r, save=True, amax_out=am)
    half = x.shape[1] // 2
    a = mx.act_fwd(f.y[:, :half], f.y[:, half:], save=True)
    dg, du = mx.act_bwd(dh, a.gate, a.up)
    dy = torch.cat([dg, du], 1)
    dx, dw, db = mx.norm_bwd(dy, f.saved, f.rstd, f.mean, w, dres=x)
    return [f.y, f.sum, am, f.saved.codes, f.saved.sf, a.h, a.gate.codes, a.up.sf, dg, du, dx, dw, db,
            mx.act8_restore(f.saved)]


def _args(seed=0, rows=301, cols=2048):
    d = lambda k, s, i: workloads.draw(k, s, 500 + seed + i, device="cuda")  # noqa: E731
    return [d("student_t3", (rows, cols), 0), d("normal", (rows, cols), 1), d("normal", (1, cols), 2).float()[0],
            d("normal", (1, cols), 3).float()[0], d("student_t3", (rows, cols // 2), 4)]


def test_side_stream_and_graph_give_the_same_bits(mx):
    args = _args()
    want = _all(mx, *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x, r, w, b, dh = args
    am = torch.empty(1, device="cuda")
    f = mx.norm_fwd(x, w, b, residual=r, save=True, amax_out=am, stream=s)  # by argument
    dx, dw, db = mx.norm_bwd(f.y, f.saved, f.rstd, f.mean, w, stream=s)
    with torch.cuda.stream(s):  # and as the current stream
        got = _all(mx, *args)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(f.y, want[0]) and torch.equal(am, want[2])
    ref_dx = mx.norm_bwd(f.y, f.saved, f.rstd, f.mean, w)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), ref_dx))
    assert all(torch.equal(p, q) for p, q in zip(want, got))

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = _all(mx, *args)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, held))
    for p, q in zip(args, _args(7)):
        p.copy_(q)
    g.replay()
    want = _all(mx, *args)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, held))


def test_calls_count_launches_and_leave_the_status_clear(mx):
    before = mx.launch_count()
    _all(mx, *_args())
    assert mx.launch_count() >= before + 6 and mx.last_device_status() == mx.MX_OK


@pytest.mark.parametrize("cols", [256, 250])
def test_offsets_past_2_to_31_elements(mx, cols):
    """Four rows 2^30 + 8 elements apart."""
    ld, rows = 2 ** 30 + 8, 4
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    far = lambda: torch.empty(rows * ld, dtype=BF, device="cuda").as_strided((rows, cols), (ld, 1))  # noqa: E731
    x = far()
    near = workloads.draw("student_t3", (rows, cols), 600, device="cuda")
    x.copy_(near)
    y = far()
    f, n = mx.norm_fwd(x, out=y, save=True), mx.norm_fwd(near, save=True)
    assert torch.equal(f.y, n.y) and torch.equal(f.saved.codes, n.saved.codes)
    p, q = mx.norm_bwd(y, x, f.rstd, f.mean, dx=y), mx.norm_bwd(n.y, near, f.rstd, f.mean)
    assert all(torch.equal(i, j) for i, j in zip(p, q))
    a, c = mx.act_fwd(x, out=y, save=True), mx.act_fwd(near, save=True)
    assert torch.equal(a.h, c.h) and torch.equal(a.gate.codes, c.gate.codes)
    d, e = mx.act_bwd(x, y, dgate=y)[0], mx.act_bwd(near, c.h)[0]
    assert torch.equal(d, e)
    assert torch.equal(mx.act8_restore(a.gate, out=y), mx.act8_restore(c.gate))


def test_more_than_2_to_31_elements(mx):
    """A dense activation of 2^31 + 4096 elements against the same rows on their own."""
    cols, rows = 4096, 2 ** 19 + 1
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    x.view(-1)[:1 << 24].normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    block = x[:4096].clone()
    for i in range(4096, rows - 1, 4096):
        x[i:i + 4096] = block[:min(4096, rows - i)]
    x[rows - 1] = block[7]
    tail = x[rows - 3:]
    a, t = mx.act_fwd(x, save=True), mx.act_fwd(tail, save=True)
    assert torch.equal(a.h[rows - 3:], t.h) and torch.equal(a.gate.codes[rows - 3:], t.gate.codes)
    assert torch.equal(a.h[:4096], a.h[4096:8192])
    del a
    f, t = mx.norm_fwd(x, save=True), mx.norm_fwd(tail, save=True)
    assert torch.equal(f.y[rows - 3:], t.y) and torch.equal(f.saved.sf[rows - 3:], t.saved.sf)
    dx, _, db = mx.norm_bwd(x, f.saved, f.rstd, f.mean, dx=f.y)
    tx, _, _ = mx.norm_bwd(tail, t.saved, t.rstd, t.mean)
    assert torch.equal(dx[rows - 3:], tx)
    want = block.double().sum(0) * ((rows - 1) // 4096) + block[7].double()
    assert ((db.double() - want).abs() <= (rows / 128 + 128) * ref.U * (block.double().abs().sum(0) * rows / 4096)).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "moss"])
def test_maxima_feed_the_quantization_that_follows(mx, fmt):
    x = workloads.draw("student_t3", (512, 1024), 610, device="cuda")
    am = torch.empty(1, device="cuda")
    y = mx.norm_fwd(x, amax_out=am).y
    own, fed = mx.quantize(y, fmt), mx.quantize(y, fmt, amax_in=am)
    assert torch.equal(own.codes, fed.codes) and torch.equal(own.scalars, fed.scalars)
    h = mx.act_fwd(x[:, :512], x[:, 512:], amax_out=am).h
    own, fed = mx.quantize(h, fmt), mx.quantize(h, fmt, amax_in=am)
    assert torch.equal(own.codes, fed.codes) and torch.equal(own.scalars, fed.scalars)
