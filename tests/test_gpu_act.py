"""The MLP's activation, forward and backward, against its plain form in 64 bits
within first-order rounding bounds; gradients also against differences."""
import pytest
import torch

import ops_ref as ref
import workloads

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ACTS = ["silu", "gelu", "gelu_tanh"]
SHAPES = [(1, 1), (3, 7), (2, 32), (5, 33), (9, 100), (130, 64), (3, 1000), (17, 1531), (64, 4096), (1, 14336),
          (5, 11009), (3, 20000)]


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def _inputs(rows, cols, dtype, seed):
    return [workloads.draw(k, (rows, cols), seed + i, sc, device="cuda").to(dtype)
            for i, (k, sc) in enumerate((("student_t3", 1.5), ("normal", 1.0), ("student_t3", 1e-3)))]


def _check_fwd(r, gate, up, act, dtype):
    a, _, _, _ = ref.activation(gate, act)
    ba, _ = ref.activation_bounds(gate, act)
    u = up.double() if up is not None else torch.ones_like(a)
    h = a * u
    ref.assert_within(r.h, h, ba * u.abs() + 2 * ref.U * h.abs() + ref.out_rounding(h, dtype), "h")


def _check_bwd(got, dh, gate, up, act, dtype):
    a, s, _, _ = ref.activation(gate, act)
    ba, bs = ref.activation_bounds(gate, act)
    d = dh.double()
    u = up.double() if up is not None else torch.ones_like(a)
    dg = d * u * s
    ref.assert_within(got[0], dg, (d * u).abs() * bs + 3 * ref.U * dg.abs() + ref.out_rounding(dg, dtype), "dgate")
    if up is None:
        assert got[1] is None
        return
    du = d * a
    ref.assert_within(got[1], du, d.abs() * ba + 2 * ref.U * du.abs() + ref.out_rounding(du, dtype), "dup")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(mx, shape, gated, act, dtype):
    gate, up, _ = _inputs(*shape, dtype, 50)
    up = up if gated else None
    amax = torch.full((1,), 9e9, device="cuda")
    r = mx.act_fwd(gate, up, act=act, save=True, amax_out=amax)
    _check_fwd(r, gate, up, act, dtype)
    assert amax.item() == r.h.float().abs().max().item()
    for got, src in ((r.gate, gate), (r.up, up)):
        if src is None:
            assert got is None
            continue
        alone = mx.act8_save(src)
        assert torch.equal(got.codes, alone.codes) and torch.equal(got.sf, alone.sf)
    plain = mx.act_fwd(gate, up, act=act)
    assert torch.equal(plain.h, r.h) and plain.gate is None and plain.up is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("source", ["kept", "act8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(mx, shape, source, gated, act, dtype):
    gate, up, dh = _inputs(*shape, dtype, 60)
    up = up if gated else None
    amax = torch.full((1,), 9e9, device="cuda")
    if source == "act8":
        g8, u8 = mx.act8_save(gate), mx.act8_save(up) if gated else None
        got = mx.act_bwd(dh, g8, u8, act=act, amax_out=amax)
        gate = ref.decode(g8.codes, g8.sf, shape[1])
        up = ref.decode(u8.codes, u8.sf, shape[1]) if gated else None
    else:
        got = mx.act_bwd(dh, gate, up, act=act, amax_out=amax)
    _check_bwd(got, dh, gate, up, act, dtype)
    assert amax.item() == max(t.float().abs().max().item() for t in got if t is not None)


@pytest.mark.parametrize("how", ["dense", "wide", "odd", "halves"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [31, 64, 200, 4096])
def test_layouts(mx, cols, dtype, how):
    """Strided and misaligned operands, the halves of one projection, outputs
    inside wider rows."""
    rows = 11
    gate, up, dh = _inputs(rows, cols, dtype, 70)
    if how == "halves":
        both = torch.cat([gate, up], 1)
        g, u, d = both[:, :cols], both[:, cols:], dh
    else:
        g, u, d = (ref.layout(t, how) for t in (gate, up, dh))
    at = 8 if how in ("wide", "dense") else 3
    wide = torch.full((rows, cols + 24), 5.0, dtype=dtype, device="cuda")
    r = mx.act_fwd(g, u, out=wide[:, at:at + cols], save=True)
    _check_fwd(r, gate, up, "silu", dtype)
    assert (wide[:, :at] == 5).all() and (wide[:, at + cols:] == 5).all()
    w2 = torch.full((rows, 2 * cols + 48), 5.0, dtype=dtype, device="cuda")
    o1, o2 = w2[:, at:at + cols], w2[:, cols + 24 + at:2 * cols + 24 + at]
    _check_bwd(mx.act_bwd(d, g, u, dgate=o1, dup=o2), dh, gate, up, "silu", dtype)
    first = w2.clone()
    assert (w2[:, :at] == 5).all() and (w2[:, at + cols:cols + 24 + at] == 5).all()
    from8 = mx.act_bwd(d, r.gate, r.up)
    assert from8[0].data_ptr() + cols * dtype.itemsize == from8[1].data_ptr()  # one [rows, 2 cols] tensor
    # in place: dgate over gate, dup over up
    got = mx.act_bwd(d, g, u, dgate=g, dup=u)
    assert torch.equal(got[0], first[:, at:at + cols]) and torch.equal(got[1], first[:, cols + 24 + at:2 * cols + 24 + at])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ACTS)
def test_extremes(mx, act, dtype):
    """Large, small and zero arguments: the limits of each function, no NaN from
    an overflowing exponential."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 20.0, -20.0, 87.0, -87.0, 90.0, -90.0, 1e4, -1e4, 1e18, -1e18,
                      3e38, -3e38], device="cuda").to(dtype).view(1, -1)
    one = torch.ones_like(z)
    h = mx.act_fwd(z, act=act).h
    _check_fwd(mx.act_fwd(z[:, :14].contiguous(), act=act), z[:, :14], None, act, dtype)
    dz, _ = mx.act_bwd(one, z, act=act)
    assert torch.isfinite(h).all() and torch.isfinite(dz).all()
    big = z.float() > 60
    assert torch.equal(h[big], z[big]) and (dz[big] == 1).all()
    low = z.float() < -1000
    assert (h[low] == 0).all() and (dz[low] == 0).all()


@pytest.mark.parametrize("cols", [32, 45, 256])
def test_non_finite_elements_stay_where_they_are(mx, cols):
    gate, up, dh = _inputs(4, cols, BF, 80)
    gate[1, 3], up[2, 4] = float("nan"), float("inf")
    r = mx.act_fwd(gate, up, save=True)
    bad = torch.zeros(4, cols, dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[2, 4] = True
    assert torch.equal(~torch.isfinite(r.h), bad)
    dg, du = mx.act_bwd(dh, r.gate, r.up)
    bad_g, bad_u = torch.zeros_like(bad), torch.zeros_like(bad)
    bad_g[1, 3] = bad_g[2, 4] = bad_u[1, 3] = True
    assert torch.equal(~torch.isfinite(dg), bad_g) and torch.equal(~torch.isfinite(du), bad_u)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(mx, act):
    """Central differences of h in 64 bits, step 1e-5: off by about 1e-10."""
    gate, up, dh = _inputs(4, 50, F32, 90)
    dg, du = mx.act_bwd(dh, gate, up, act=act)
    e = 1e-5
    f = lambda g, u: ref.activation(g, act)[0] * u  # noqa: E731
    G, Up, D = gate.double(), up.double(), dh.double()
    ng = D * (f(G + e, Up) - f(G - e, Up)) / (2 * e)
    nu = D * (f(G, Up + e) - f(G, Up - e)) / (2 * e)
    assert (dg.double() - ng).abs().max() <= 1e-5 * ng.abs().max()
    assert (du.double() - nu).abs().max() <= 1e-5 * nu.abs().max()


@pytest.mark.parametrize("shape", [(0, 64), (5, 0)])
def test_empty(mx, shape):
    x = torch.empty(shape, dtype=BF, device="cuda")
    amax = torch.full((1,), 3.0, device="cuda")
    assert mx.act_fwd(x, x, save=True, amax_out=amax).h.shape == shape and amax.item() == 0
    dg, du = mx.act_bwd(x, x, x)
    assert dg.shape == shape and du.shape == shape
