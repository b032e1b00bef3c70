"""Several host threads in the norm calls at once, and calls of several widths in
one graph: one kernel serves many widths, each with shared memory of its own size,
and no call may depend on what another one asked for."""
import ctypes as C
import threading

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


class Norm:
    """Inputs and buffers of a forward (residual, checkpoint) and a backward call (from the
    checkpoint, residual's gradient) of one width; run() allocates nothing."""

    def __init__(self, mx, rows, cols, seed):
        self.mx = mx
        d = lambda k, i: workloads.draw(k, (rows, cols), seed + i, device="cuda")  # noqa: E731
        self.x, self.r, self.dy, self.ds = d("student_t3", 0), d("normal", 1), d("student_t3", 2), d("normal", 3)
        self.w = workloads.draw("normal", (1, cols), seed + 4, device="cuda").float()[0]
        e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
        self.y, self.s, self.dx = (torch.empty_like(self.x) for _ in range(3))
        self.mean, self.rstd, self.dw, self.db = e(rows), e(rows), e(cols), e(cols)
        self.saved = mx.Act8.empty(rows, cols, self.x.device)
        self.ws = torch.empty(mx.norm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")

    def run(self):
        self.mx.norm_fwd(self.x, self.w, residual=self.r, sum_out=self.s, save=self.saved, out=self.y, mean=self.mean,
                         rstd=self.rstd)
        self.mx.norm_bwd(self.dy, self.saved, self.rstd, self.mean, self.w, dres=self.ds, dx=self.dx, dw=self.dw,
                         db=self.db, workspace=self.ws)

    def many(self, n, stream):
        """The two calls n times through the C interface, with nothing between them that holds
        the interpreter: the threads' calls then overlap most of the time."""
        L, (rows, cols) = self.mx.lib(), self.x.shape
        p = [t.data_ptr() for t in (self.x, self.r, self.w, self.s, self.y, self.mean, self.rstd, self.dy, self.ds,
                                    self.dx, self.dw, self.db, self.ws)]
        x, r, w, s, y, mean, rstd, dy, ds, dx, dw, db, ws = (C.c_void_p(v) for v in p)
        saved, bf, f32 = C.byref(self.saved._c(self.x.device)), self.mx.OUT[BF], self.mx.OUT[torch.float32]
        at, size = C.c_void_p(stream.cuda_stream), self.ws.numel()
        for _ in range(n):
            rc = L.mx_norm_fwd(x, cols, r, cols, bf, rows, cols, 0, w, None, f32, 1e-5, s, cols, y, cols, bf, mean, rstd,
                               saved, None, at)
            rc = rc or L.mx_norm_bwd(dy, cols, bf, None, 0, saved, mean, rstd, w, f32, rows, cols, 0, ds, cols, dx, cols,
                                     bf, dw, db, None, ws, size, at)
            if rc != 0:
                raise self.mx.MXError(rc, f"{rows}x{cols}")

    def outputs(self):
        return [t.clone() for t in (self.y, self.s, self.saved.codes, self.dx, self.dw, self.db)]


# one kernel each: aligned rows of two octs a thread; rows at any address; narrow rows; four octs a thread
@pytest.mark.parametrize("widths", [(2048, 4096), (1531, 4097), (256, 200), (8200, 12288)])
def test_two_threads_at_two_widths(mx, widths):
    cases = [Norm(mx, 96, c, 900 + 10 * i) for i, c in enumerate(widths)]
    want = []
    for c in cases:
        c.run()
        want.append(c.outputs())
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(2)

    def work(case):
        try:
            stream = torch.cuda.Stream()
            start.wait(30)
            case.many(10000, stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for c, w in zip(cases, want):
        assert all(torch.equal(p, q) for p, q in zip(c.outputs(), w))
    assert mx.last_device_status() == mx.MX_OK


@pytest.mark.parametrize("widths", [(4096, 2048), (4097, 1531), (512, 64), (16384, 8200)])
def test_one_graph_of_two_widths(mx, widths):
    """The wider call first, so that the narrower one is the last to have been launched."""
    cases = [Norm(mx, 96, c, 950 + 10 * i) for i, c in enumerate(widths)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in cases:
            c.run()
    g.replay()
    torch.cuda.synchronize()
    got = [c.outputs() for c in cases]
    for c, w in zip(cases, got):
        c.run()
        assert all(torch.equal(p, q) for p, q in zip(c.outputs(), w))
