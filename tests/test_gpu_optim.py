"""The AdamW step and the gradient norm against plain implementations: 64-bit ones with
error bounds counted from the operations, and for 8-bit moments and stochastic rounding
one in single fp32 operations on the CPU, which must give the same codes.

Bounds, in u = 2^-24 (half a step of fp32).  A constant (beta, 1 - beta) is off by u, each
product and sum by u.  m: 3 u on each of its two terms but 4 with the scale, and u for the
sum: 6 u of |b1 m| + |c1 g|.  v, whose terms have one sign: 2 u on the first, 5 u on the
second (the scaled gradient's u counts twice), u for the sum: 7 u v.  The step lr m / d: d
from v by half of 7 u, the root's 2 u (approximation), its constant 1 u, sum u, so 8 u; the
reciprocal 2 u, the products 2 u, the constant lr / (1 - beta1^t) u: 14 u of the step, and
m's own error times lr / d.  The weight: decay's constant u, its product u, the sum u."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
B1, B2, EPS = 0.9, 0.999, 1e-8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def values(seed, n, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g) * scale * torch.exp(torch.randn(n, generator=g))


def placed(x, dtype, shift):
    """x on the GPU, `shift` elements past an aligned address."""
    room = torch.full((x.numel() + shift + 16,), 7.0, dtype=dtype, device="cuda")
    view = room[shift:shift + x.numel()]
    view.copy_(x)
    return view, room


# ------------------------------------------------------------------ plain forms
def ceil_exponent(b):
    m, e = torch.frexp(b)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(b == 0, torch.zeros_like(e), e).clamp(min=-127)


def philox16(seed, n, t, word):
    count = -(-n // 8)
    x = np.zeros((4, count), dtype=np.uint64)
    x[0], x[2], x[3] = np.arange(count), t, word
    low = np.uint64(0xFFFFFFFF)
    for r in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        k0, k1 = np.uint64((seed + r * 0x9E3779B9) % 2 ** 32), np.uint64(((seed >> 32) + r * 0xBB67AE85) % 2 ** 32)
        x = np.stack([(b >> np.uint64(32)) ^ x[1] ^ k0, b & low, (a >> np.uint64(32)) ^ x[3] ^ k1, a & low])
    return torch.from_numpy(x.T.astype(np.uint32).copy().view(np.uint16).reshape(-1)[:n].astype(np.int64))


def encode(x, root, u16=None):
    """(codes [1, 32 G], bytes [1, G]) of fp32 x on the CPU."""
    n = x.numel()
    G = -(-n // 32)
    pad = lambda v: torch.nn.functional.pad(v, (0, 32 * G - n)).view(G, 32)  # noqa: E731
    x = pad(x)
    finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    e = ceil_exponent(finite.abs().amax(1))
    y = x * torch.ldexp(torch.ones(G), -e)[:, None]
    if root:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
    if u16 is None:
        v = y.to(torch.float8_e4m3fn)
    else:
        a = torch.where(torch.isfinite(y), y, torch.zeros_like(y)).abs()
        step = torch.ldexp(torch.ones_like(a), (torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
        low = torch.floor(a / step)
        v = torch.copysign((low + (pad(u16) < (a / step - low) * 65536.0)) * step, y).to(torch.float8_e4m3fn)
    codes = v.view(torch.uint8)
    codes = torch.where(torch.isfinite(x), codes, (codes & 128) | 127)
    return codes.reshape(1, -1), (e + 127).to(torch.uint8).view(1, -1)


def decode(a):
    n = a.cols
    v = a.codes.cpu().view(torch.float8_e4m3fn).float().view(-1, 32)
    return (v * torch.ldexp(torch.ones(v.shape[0]), a.sf.cpu().view(-1).int() - 127)[:, None]).view(-1)[:n]


def moments32(g, m, v, s):
    """m' and v' by single fp32 operations."""
    f = lambda c: torch.tensor(c, dtype=torch.float32)  # noqa: E731
    x = g.float() * s
    return m * f(B1) + x * f(1.0 - B1), v * f(B2) + (x * x) * f(1.0 - B2)


def weights64(p, m, v, lr, wd, t):
    """(new weight, |step|) in 64 bits."""
    p, m, v = p.double(), m.double(), v.double()
    step = lr / (1 - B1 ** t) * m / (torch.sqrt(v / (1 - B2 ** t)) + EPS)
    return p * (1 - lr * wd) - step, step.abs()


SIZES = ([1], [7], [8, 40], [31, 32, 33], [2047, 2048, 2049, 5, 4096], [70001], [16 * 2048 * 40 + 24])


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("pt,gt", [(F32, F32), (F32, BF), (BF, BF), (BF, F32)], ids=str)
@pytest.mark.parametrize("shift", [0, 1])
def test_fp32_moments(mx, sizes, pt, gt, shift):
    lr, t, s = 3e-3, 7, 0.37
    p0 = [values(i, n).to(pt) for i, n in enumerate(sizes)]
    g0 = [values(50 + i, n, 1e-2).to(gt) for i, n in enumerate(sizes)]
    m0 = [values(100 + i, n, 1e-2) for i, n in enumerate(sizes)]
    v0 = [values(150 + i, n, 1e-2) ** 2 for i, n in enumerate(sizes)]
    wd = [0.1 * (i % 3) for i in range(len(sizes))]
    placed_p = [placed(p, pt, shift) for p in p0]
    params = [v for v, _ in placed_p]
    grads = [placed(g, gt, 3 * shift)[0] for g in g0]
    copies = [placed(torch.zeros(n), BF, shift)[0] for n in sizes] if pt is F32 else None
    opt = mx.AdamW(params, lr=lr, betas=(B1, B2), eps=EPS, weight_decay=wd, copies=copies)
    for a, b in zip(opt.m + opt.v, m0 + v0):
        a.copy_(b)
    top = torch.empty(len(sizes), device="cuda")
    opt.step(grads, grad_scale=torch.tensor([s], device="cuda"), amax_out=top, t=t)
    s = float(torch.tensor(s))
    for i, n in enumerate(sizes):
        p, g, m, v = p0[i].double(), g0[i].double() * s, m0[i].double(), v0[i].double()
        mm, vv = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
        em = 6 * U * ((B1 * m).abs() + ((1 - B1) * g).abs())
        assert ((opt.m[i].cpu().double() - mm).abs() <= em).all()
        assert ((opt.v[i].cpu().double() - vv).abs() <= 7 * U * vv + 2.0 ** -149).all()
        new, step = weights64(p, mm, vv, lr, wd[i], t)
        d = torch.sqrt(vv / (1 - B2 ** t)) + EPS
        bound = 14 * U * step + lr / (1 - B1 ** t) * em / d + 3 * U * (p.abs() + step)
        got = params[i].cpu().double()
        assert ((got - new).abs() <= bound + (HALF[BF] * (new.abs() + bound) if pt is BF else 0)).all()
        read = params[i]
        if copies is not None:
            assert torch.equal(copies[i], params[i].to(BF))
            read = copies[i]
        assert float(top[i]) == float(read.abs().max())
    for (view, room), n in zip(placed_p, sizes):  # nothing beside the tensors is written
        assert (room[:shift] == 7.0).all() and (room[shift + n:] == 7.0).all()


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("pt,gt", [(F32, BF), (BF, F32)], ids=str)
@pytest.mark.parametrize("rounding", ["rne", "sr"])
@pytest.mark.parametrize("shift", [0, 1])
def test_8bit_moments(mx, sizes, pt, gt, rounding, shift):
    """The codes follow from the formula alone; the weights take the moments as computed."""
    lr, t, s, seed = 3e-3, 5, 0.5, 0x123456789ABC
    p0 = [values(i, n).to(pt) for i, n in enumerate(sizes)]
    g0 = [values(50 + i, n, 1e-2).to(gt) for i, n in enumerate(sizes)]
    params = [placed(p, pt, shift)[0] for p in p0]
    grads = [placed(g, gt, shift)[0] for g in g0]
    opt = mx.AdamW(params, lr=lr, betas=(B1, B2), eps=EPS, weight_decay=0.1, state="8bit", rounding=rounding, seed=seed)
    for i, n in enumerate(sizes):
        for a, x, root in ((opt.m[i], values(100 + i, n, 1e-2), False), (opt.v[i], values(150 + i, n, 1e-2).abs(), True)):
            codes, sf = encode(x, root)
            a.codes.copy_(codes)
            a.sf.copy_(sf)
    before = [(decode(opt.m[i]), decode(opt.v[i])) for i in range(len(sizes))]
    opt.step(grads, grad_scale=torch.tensor([s], device="cuda"), t=t)
    for i, n in enumerate(sizes):
        m, r = before[i]
        mm, vv = moments32(g0[i], m, r * r, s)
        u = [philox16(seed, n, t, 4 * i + k) if rounding == "sr" else None for k in range(3)]
        for got, want in ((opt.m[i], encode(mm, False, u[0])), (opt.v[i], encode(torch.sqrt(vv), True, u[1]))):
            assert torch.equal(got.codes.cpu(), want[0])
            assert torch.equal(got.sf.cpu(), want[1])
        new, step = weights64(p0[i], mm, vv, lr, 0.1, t)  # mm and vv are the kernel's own
        bound = 14 * U * step + 3 * U * (p0[i].double().abs() + step)
        if pt is BF:  # to nearest half a step, stochastically a whole one
            bound = bound + (2 if rounding == "sr" else 1) * HALF[BF] * (new.abs() + bound)
        assert ((params[i].cpu().double() - new).abs() <= bound).all()


def test_stochastic_rounding_keeps_small_steps(mx):
    """Over many seeds the mean of a root that a step moves by a fifteenth of a code's distance is right: 256
    values x 64 seeds, p = 1/15, so the mean's standard deviation is below 0.002 of the distance; 5 of them."""
    n, start, g = 256, 1.0, 1.1 ** 0.5
    first = [values(3, n)]
    total = 0.0
    for seed in range(64):
        p = [first[0].cuda()]
        opt = mx.AdamW(p, state="8bit", rounding="sr", seed=seed, betas=(0.9, 0.9))
        codes, sf = encode(torch.full((n,), start), True)
        opt.v[0].codes.copy_(codes)
        opt.v[0].sf.copy_(sf)
        opt.step([torch.full((n,), g, device="cuda")])
        total += decode(opt.v[0]).double().mean().item()
    r = (0.9 + 0.1 * 1.1) ** 0.5
    assert abs(total / 64 - r) < 5 * 0.002 * 0.125


def test_bf16_weights_stochastic(mx):
    """A bf16 weight goes up where the number is below the bits that go: the codes' rule on the fp32 weight."""
    n, seed, t = 4099, 99, 3
    p0, g0 = values(1, n).to(BF), values(2, n, 1e-2)
    out = []
    for rounding in ("rne", "sr"):
        p = [p0.cuda()]
        opt = mx.AdamW(p, lr=1e-2, betas=(B1, B2), weight_decay=0.0, rounding=rounding, seed=seed)
        opt.step([g0.cuda()], t=t)
        out.append(p[0].cpu())
    q = [p0.float().cuda()]  # the same step on fp32 weights
    opt = mx.AdamW(q, lr=1e-2, betas=(B1, B2), weight_decay=0.0)
    opt.step([g0.cuda()], t=t)
    q = q[0].cpu()
    assert torch.equal(out[0], q.to(BF))
    bits = q.view(torch.int32)
    up = philox16(seed, n, t, 2) < (bits & 0xFFFF)
    assert torch.equal(out[1].float(), ((bits & -65536) + (up.int() << 16)).view(torch.float32))


def test_many_tensors_and_kinds(mx):
    """300 tensors of every kind in one call equal one call for each."""
    sizes = [1 + (37 * i) % 500 for i in range(300)]
    kinds = [(F32, BF), (F32, F32), (BF, BF), (BF, F32)]

    def make():
        params = [placed(values(i, n), kinds[i % 4][0], i % 3)[0] for i, n in enumerate(sizes)]
        grads = [placed(values(400 + i, n), kinds[i % 4][1], i % 2)[0] for i, n in enumerate(sizes)]
        return params, grads

    params, grads = make()
    top = torch.empty(300, device="cuda")
    opt = mx.AdamW(params, weight_decay=0.0, state="8bit")
    opt.step(grads, amax_out=top)
    alone, _ = make()
    for i in range(300):
        one = mx.AdamW([alone[i]], weight_decay=0.0, state="8bit")
        one.step([grads[i]])
        assert torch.equal(one.m[0].codes, opt.m[i].codes) and torch.equal(one.v[0].sf, opt.v[i].sf)
        assert torch.equal(alone[i], params[i])
        assert float(top[i]) == float(params[i].abs().max())


@pytest.mark.parametrize("state", ["fp32", "8bit"])
@pytest.mark.parametrize("pt,gt,rounding", [(F32, F32, "rne"), (F32, BF, "sr"), (BF, BF, "sr"), (BF, F32, "rne")], ids=str)
@pytest.mark.parametrize("n", [20000, 20003])
def test_each_array_at_its_own_address(mx, state, pt, gt, rounding, n):
    """Parameter, gradient and copy each at its own distance from an aligned address (16 bytes past one of 32, too):
    the values that aligned ones get."""
    p0, g0 = values(1, n).to(pt), values(2, n, 1e-2).to(gt)

    def run(sp, sg, sc):
        (p, room), (g, _) = placed(p0, pt, sp), placed(g0, gt, sg)
        c, croom = placed(torch.zeros(n), BF, sc) if pt is F32 else (None, None)
        top = torch.empty(1, device="cuda")
        opt = mx.AdamW([p], state=state, rounding=rounding, seed=3, copies=[c])
        for _ in range(2):
            opt.step([g], amax_out=top)
        for r, k in ((room, sp), (croom, sc)):
            assert r is None or ((r[:k] == 7.0).all() and (r[k + n:] == 7.0).all())
        m, v = (opt.m[0].codes, opt.v[0].codes) if state == "8bit" else (opt.m[0], opt.v[0])
        norm = mx.grad_norm([g, p])[:1]
        return [x.clone() for x in (p, m, v, top, p if c is None else c)], norm

    want, norm = run(0, 0, 0)
    for shifts in ((4, 0, 0), (0, 4, 8), (2, 12, 1), (8, 1, 4), (0, 0, 3), (5, 2, 0)):
        got, other = run(*shifts)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert abs(float(other) / float(norm) - 1) <= 19 * U  # sums of other orders: 9.5 u on either side


@pytest.mark.parametrize("state", ["fp32", "8bit"])
def test_no_gradient_and_nan_scale_leave_tensors(mx, state):
    p0 = [values(i, 100 + i) for i in range(3)]
    for case in ("none", "nan"):
        p = [x.cuda() for x in p0]
        copies = [torch.zeros_like(x, dtype=BF) for x in p]
        opt = mx.AdamW(p, state=state, copies=copies)
        first = [values(9, x.numel()).cuda() for x in p]
        opt.step(first)
        now = [x.clone() for x in p]
        kept = opt.m_all.codes.clone() if state == "8bit" else opt.m_all.clone()
        for c in copies:
            c.zero_()
        top = torch.empty(3, device="cuda")
        scale = torch.tensor([float("nan")], device="cuda") if case == "nan" else None
        opt.step([None] * 3 if case == "none" else first, grad_scale=scale, amax_out=top)
        assert all(torch.equal(a, b) for a, b in zip(p, now))
        assert torch.equal(kept, opt.m_all.codes if state == "8bit" else opt.m_all)
        assert all(torch.equal(c, x.to(BF)) for c, x in zip(copies, p))
        assert [float(x) for x in top] == [float(c.abs().max()) for c in copies]


@pytest.mark.parametrize("rounding", ["rne", "sr"])
def test_non_finite_gradients(mx, rounding):
    """Inf and NaN become the NaN code of their value alone; their group's other codes stay what they are."""
    n = 96
    g = values(1, n)
    g[5], g[40], g[70] = float("inf"), float("nan"), float("-inf")
    p = [values(2, n).cuda()]
    opt = mx.AdamW(p, state="8bit", rounding=rounding, seed=4, betas=(B1, B2), weight_decay=0.0)
    opt.step([g.cuda()], t=2)
    mm, vv = moments32(g, torch.zeros(n), torch.zeros(n), 1.0)
    for k, (got, x, root) in enumerate(((opt.m[0], mm, False), (opt.v[0], torch.sqrt(vv), True))):
        codes, sf = encode(x, root, philox16(4, n, 2, k) if rounding == "sr" else None)
        assert torch.equal(got.codes.cpu() & 127, codes & 127) and torch.equal(got.sf.cpu(), sf)
    bad = torch.tensor([5, 40, 70])
    assert torch.isnan(p[0].cpu()[bad]).all() and torch.isfinite(p[0].cpu()).sum() == n - 3


def test_smallest_root_stays_above_zero(mx):
    """Beside a gradient 2^30 times its own a value's root keeps the smallest code, so its step stays bounded."""
    g = torch.full((32,), 2.0 ** -15)
    g[0] = 2.0 ** 15
    p = [torch.zeros(32, device="cuda")]
    opt = mx.AdamW(p, lr=1.0, state="8bit", betas=(B1, B2), weight_decay=0.0)
    opt.step([g.cuda()])
    codes = opt.v[0].codes.cpu()[0]
    assert (codes[1:] == 1).all() and codes[0] > 1
    assert (p[0].abs() <= 1.001).all()
    opt.step([g.cuda()])
    assert torch.isfinite(p[0]).all() and (p[0].abs() <= 10).all()


def test_zero_moments_and_zero_gradient(mx):
    for state in ("fp32", "8bit"):
        p = [values(1, 40).cuda()]
        q = p[0].clone()
        opt = mx.AdamW(p, state=state, weight_decay=0.0)
        opt.step([torch.zeros(40, device="cuda")])
        assert torch.equal(p[0], q)


@pytest.mark.parametrize("state", ["fp32", "8bit"])
def test_captured_steps_count(mx, state):
    """Two graphs of two optimizers, replayed in turn, against eager steps with the number and the rate on the device."""
    n, lr = 5000, torch.full((1,), 2e-3, device="cuda")
    grads = [values(7, n).cuda()]

    def make(capturable):
        return mx.AdamW([values(1, n).cuda()], state=state, rounding="sr" if state == "8bit" else "rne", seed=5,
                        betas=(B1, B2), capturable=capturable)

    graphs = []
    for _ in range(2):
        opt = make(True)
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                opt.step(grads, lr=lr)
        torch.cuda.current_stream().wait_stream(side)
        graphs.append((opt, g))
    eager, host = make(True), make(False)
    for k in range(3):
        lr.fill_(2e-3 * (k + 1))
        for _, g in graphs:
            g.replay()
        eager.step(grads, lr=lr)
        host.step(grads, lr=float(lr))
        for opt, _ in graphs:
            assert torch.equal(opt.params[0], eager.params[0])
        # the number's powers in fp32 instead of fp64 (2^-21 of a step of at most 10 lr), the rate's product
        assert (host.params[0] - eager.params[0]).abs().max() <= 2.0 ** -20 * 10 * 6e-3 + 3 * U * 60
        assert torch.equal(host.m_all.codes if state == "8bit" else host.m_all,
                           eager.m_all.codes if state == "8bit" else eager.m_all)


def test_other_stream_and_order(mx):
    p, g = [values(1, 1 << 20).cuda()], [values(2, 1 << 20).cuda()]
    q = [p[0].clone()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = mx.AdamW(p), mx.AdamW(q)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.step(g, stream=s)
        b.step(g)
    torch.cuda.synchronize()
    assert torch.equal(p[0], q[0])


def test_two_optimizers_at_once(mx):
    """Steps of two optimizers with 8-bit moments on two streams, against the same steps one after another."""
    sizes = [40000 + 37 * i for i in range(20)]

    def make(seed):
        return mx.AdamW([values(seed + i, n).cuda() for i, n in enumerate(sizes)], state="8bit", rounding="sr", seed=seed)

    grads = [values(500 + i, n).cuda() for i, n in enumerate(sizes)]
    a, b, c, d = make(1), make(2), make(1), make(2)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        na = mx.grad_norm(grads, max_norm=1.0, stream=s)
        a.step(grads, grad_scale=na[1:], stream=s)
        nb = mx.grad_norm(grads, max_norm=2.0, stream=t)
        b.step(grads, grad_scale=nb[1:], stream=t)
        torch.cuda.synchronize()  # na and nb are read on their streams until here
    for _ in range(5):
        c.step(grads, grad_scale=mx.grad_norm(grads, max_norm=1.0)[1:])
        d.step(grads, grad_scale=mx.grad_norm(grads, max_norm=2.0)[1:])
    for x, y in ((a, c), (b, d)):
        assert all(torch.equal(p, q) for p, q in zip(x.params, y.params))
        assert torch.equal(x.v_all.codes, y.v_all.codes) and torch.equal(x.m_all.sf, y.m_all.sf)


def test_past_2g_values(mx):
    """The last values of a tensor of more than 2^31 are what the same step makes of them alone."""
    n, tail = (1 << 31) + 64 * 1024 + 8, 1024 + 8
    p = torch.zeros(n, dtype=BF, device="cuda")
    g = torch.zeros(n, dtype=BF, device="cuda")
    p[-tail:] = values(1, tail).to(BF).cuda()
    g[-tail:] = values(2, tail).to(BF).cuda()
    q, h = p[-tail:].clone(), g[-tail:].clone()
    big, small = mx.AdamW([p], state="8bit"), mx.AdamW([q], state="8bit")
    top = torch.empty(1, device="cuda")
    big.step([g], amax_out=top)
    small.step([h])
    assert torch.equal(p[-tail:], q) and float(top) == float(q.abs().max())
    assert not p[:-tail].any()
    both = mx.grad_norm([g, h])
    assert abs(float(both[0]) / (2 ** 0.5 * float(h.double().norm())) - 1) < 2e-7


# ------------------------------------------------------------------ gradient norm
@pytest.mark.parametrize("sizes", [[1], [8], [9, 8191, 8192, 8193, 0, 3], [1 << 20], [5000003], [100] * 1100], ids=lambda s: str(s[:6]))
@pytest.mark.parametrize("dtype", [F32, BF], ids=str)
@pytest.mark.parametrize("shift", [0, 1])
def test_grad_norm(mx, sizes, dtype, shift):
    """Squares u, sums of 32 (two chains of 16) 16 u of the sum of squares, half of it in the root, one rounding."""
    grads = [placed(values(i, n, 1e-3).to(dtype), dtype, shift)[0] for i, n in enumerate(sizes)]
    total = sum(float((g.double() ** 2).sum()) for g in grads)
    norm = total ** 0.5
    out = mx.grad_norm(grads, max_norm=0.5 * norm)
    assert abs(float(out[0]) / norm - 1) <= (17 / 2 + 1) * U
    assert abs(float(out[1]) / (0.5 * norm / (norm + 1e-6)) - 1) <= (17 / 2 + 2) * U
    assert float(mx.grad_norm(grads, max_norm=2 * norm)[1]) == 1.0
    assert float(mx.grad_norm(grads)[1]) == 1.0
    again = mx.grad_norm(grads, max_norm=0.5 * norm)
    assert torch.equal(out, again)


def test_grad_norm_mixed_none_and_empty(mx):
    a, b = values(1, 1000).cuda(), values(2, 77).to(BF).cuda()
    want = float((a.double() ** 2).sum() + (b.double() ** 2).sum()) ** 0.5
    got = mx.grad_norm([a, None, b, torch.empty(0, device="cuda")], max_norm=1.0)
    assert abs(float(got[0]) / want - 1) < 10 * U
    out = torch.full((2,), 9.0, device="cuda")
    mx.grad_norm([], max_norm=1.0, out=out)
    assert out.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 3e19])
def test_grad_norm_not_finite_skips_the_step(mx, bad):
    g = values(1, 3000)
    g[1234] = bad
    g = g.cuda()
    out = mx.grad_norm([g], max_norm=1.0)
    assert not torch.isfinite(out[0]) and torch.isnan(out[1])
    p = [values(2, 3000).cuda()]
    q = p[0].clone()
    mx.AdamW(p).step([g], grad_scale=out[1:])
    assert torch.equal(p[0], q)


def test_grad_norm_then_step_captured(mx):
    """Clipping and the step in one graph, replayed over new gradients."""
    n = 10000
    p, g = [values(1, n).cuda()], [values(2, n).cuda()]
    opt = mx.AdamW(p, capturable=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(g, grad_scale=mx.grad_norm(g, max_norm=1.0)[1:])
    q = [values(1, n).cuda()]
    other = mx.AdamW(q, capturable=True)
    for k in range(3):
        g[0].copy_(values(10 + k, n))
        graph.replay()
        other.step(g, grad_scale=mx.grad_norm(g, max_norm=1.0)[1:])
        assert torch.equal(p[0], q[0])
