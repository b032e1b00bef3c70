"""The activation's arithmetic where a coarser one shows: the far negative side,
where the value is small but a normal number, and the slopes' zeros, where two
terms cancel.

Bounds: u = 2^-24.  CUDA's expf is within 1 last place (2 u), __expf within 2 +
1.173 |x| of them, an fp32 division within u, the approximate one within 2 last
places (4 u); each sum and product adds u, each subnormal intermediate 2^-149 at
most."""
import pytest
import torch

import ops_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = ref.U


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def _half_place(v, dtype):
    """Half a last place of v in dtype."""
    bits = 8 if dtype is BF else 24
    _, ex = torch.frexp(v.abs())
    return torch.exp2((ex - bits - 1).double()).clamp_min(2.0 ** (-134 if dtype is BF else -150))


def _both(mx, z, act):
    dz, _ = mx.act_bwd(torch.ones_like(z), z, act=act)
    return mx.act_fwd(z, act=act).h, dz


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_where_the_exponential_leaves_the_normal_numbers(mx, act, dtype):
    """p = e / (1 + e), e = exp(-t), t to beyond the last subnormal e (t = 104): e's own
    error and that of t (up to 6 u t: five operations of tanh GELU's argument, none of
    SiLU's), 4 u after it."""
    lo, hi = (-106.0, -80.0) if act == "silu" else (-10.9, -9.3)
    z = torch.linspace(lo, hi, 4096, device="cuda").to(dtype).view(1, -1)
    h, dz = _both(mx, z, act)
    a, s, p, t = ref.activation(z, act)
    t = t.abs()
    e = 2 * (2 + 1.173 * t) * U if dtype is BF else 2 * U + 0 * t
    rel = torch.expm1(e + (6 * t * U if act == "gelu_tanh" else 0) + 8 * U)
    zd, tiny = z.double().abs(), 2.0 ** -147
    ref.assert_within(h, a, a.abs() * rel + zd * tiny + _half_place(a, dtype), "value")
    inner = zd * (2 * ref.K_TANH * (1 + 3 * ref.C_TANH * zd ** 2) if act == "gelu_tanh" else 1.0)
    ref.assert_within(dz, s, (p + inner * p) * (rel + 4 * U) + (1 + inner) * tiny + _half_place(s, dtype), "slope")
    normal = a.abs() > 2.0 ** -126
    assert normal.any() and (h[normal] != 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradients_in_fp32_are_as_near_as_the_plain_form(mx, act):
    """Root mean square error of the slope over normal arguments, beside that of the plain
    form's single operations: no more than 1.1 times."""
    g = torch.Generator(device="cuda").manual_seed(3)
    z = 1.5 * torch.randn(64, 4096, generator=g, device="cuda")
    _, dz = _both(mx, z, act)
    _, s, _, _ = ref.activation(z, act)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        plain = p + z * p * (1 - p)
    elif act == "gelu":
        plain = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * (torch.exp(-0.5 * z * z) * 0.3989422804014327)
    else:
        th = torch.tanh(ref.K_TANH * (z + ref.C_TANH * z ** 3))
        plain = 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * ref.K_TANH * (1 + 3 * ref.C_TANH * z * z)
    rms = lambda v: (v.double() - s).square().mean().sqrt().item()  # noqa: E731
    assert rms(dz) <= 1.1 * rms(plain), (rms(dz), rms(plain))


def test_silu_in_fp32_adds_few_roundings(mx):
    """z / (1 + e), e = exp(-z): e's 2 u, of which 1 - p reaches the value, the sum's u, the
    reciprocal's 2 u (a last place) and the product's u; below 0 e / (1 + e) has e's 2 u
    whole and a product more."""
    z = torch.linspace(-80, 30, 1000003, device="cuda").view(1, -1)
    h = mx.act_fwd(z, act="silu").h
    a, _, p, _ = ref.activation(z, "silu")
    ref.assert_within(h, a, a.abs() * torch.where(z >= 0, 2 * (1 - p) + 4, 7.0) * U, "value")


def _gelu_rel(dtype):
    """GELU's tail e t g(t): the exponential (fp32: 2 u and u for its argument's rest), t
    = 1 / (1 + k y) (fp32 2 u: less than the approximate division's documented 4 u, so that
    not everything may be at its worst at once; what the tail makes of it is no more), the
    polynomial's own 0.1 u and its sums, at most 6 u of g, the two products and z's: 14 u;
    bf16: t 5 u, the polynomial 5 u, its sums, the products and z's 9 u: 19 u, and beside
    them the exponential's (2 + 1.173 y^2 / 2) places and 2 u y^2 / 2 of its argument."""
    return 14 * U if dtype is F32 else 19 * U


@pytest.mark.parametrize("lo,hi", [(0.0, 1.0), (1.0, 3.0), (3.0, 5.0), (5.0, 8.0), (8.0, 12.9)])
def test_gelu_in_fp32_keeps_its_precision_on_the_negative_side(mx, lo, hi):
    z = -torch.linspace(lo, hi, 100001, device="cuda").view(1, -1)
    h, dz = _both(mx, z, "gelu")
    a, s, p, _ = ref.activation(z, "gelu")
    rel, zd = _gelu_rel(F32), z.double().abs()
    gauss = torch.exp(-zd ** 2 / 2) / (2 * torch.pi) ** 0.5
    ref.assert_within(h, a, a.abs() * rel + 2.0 ** -126, "value")
    ref.assert_within(dz, s, p * rel + zd * gauss * 6 * U + U * s.abs() + 2.0 ** -120, "slope")


@pytest.mark.parametrize("act,at", [("silu", -1.28125), ("gelu", -0.75), ("gelu_tanh", -0.75)])
def test_bf16_slopes_at_their_zero(mx, act, at):
    """dgate = dh up a'(gate) at the bf16 gate next to the slope's zero, over all fractions
    of dh and up: off by half a place and the error of the two terms that cancel."""
    f = (1 + torch.arange(128, device="cuda") / 128).to(BF)
    dh, up = f.view(-1, 1).expand(128, 128).contiguous(), f.view(1, -1).expand(128, 128).contiguous()
    gate = torch.full_like(dh, at)
    dg, _ = mx.act_bwd(dh, gate, up, act=act)
    _, s, p, t = ref.activation(gate, act)
    z = gate.double().abs()
    if act == "gelu":
        e = 2 * (2 + 1.173 * z * z / 2) * U + z * z * U
        terms = p * (_gelu_rel(BF) + z * z * U) + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5 * (e + 3 * U)
    else:
        e = 2 * (2 + 1.173 * t.abs()) * U + 6 * t.abs() * U
        inner = z * (2 * ref.K_TANH * (1 + 3 * ref.C_TANH * z ** 2) if act == "gelu_tanh" else 1.0)
        terms = p * (e + 8 * U) + inner * p * (1 - p) * (e + 14 * U)
    d = dh.double() * up.double()
    ref.assert_within(dg, d * s, d * (terms + 3 * U * s.abs()) + _half_place(d * s.abs() * (1 + 2.0 ** -9), BF), "dgate")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_infinities_and_nan(mx, act, dtype):
    """As the formulas give them: the value at Inf is Inf, at -Inf -Inf times 0, at NaN NaN;
    the slope of tanh GELU has its limits at the infinities, the others' an Inf times 0.
    What stands beside them is as it is alone."""
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[1.0, inf, -inf, nan, -2.0, 3e38, -3e38, 0.5]], device="cuda").to(dtype)
    h, dz = _both(mx, z, act)
    assert h[0, 1] == inf and torch.isnan(h[0, 2:4]).all() and torch.isnan(dz[0, 3])
    if act == "gelu_tanh":
        assert dz[0, 1] == 1 and dz[0, 2] == 0
    else:
        assert torch.isnan(dz[0, 1:3]).all()
    assert h[0, 5] == z[0, 5] and h[0, 6] == 0 and dz[0, 5] == 1 and dz[0, 6] == 0
    keep = [0, 4, 7]
    alone, dalone = _both(mx, z[:, keep].contiguous(), act)
    assert torch.equal(h[:, keep], alone) and torch.equal(dz[:, keep], dalone)
