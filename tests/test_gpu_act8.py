"""8-bit activation checkpoints: codes and exponent bytes bit for bit against a
search over the code grid in 64 bits, and what they restore to."""
import numpy as np
import pytest
import torch

import oracle as orc
import ops_ref as ref
import workloads

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def _check(mx, x, what=""):
    a = mx.act8_save(x)
    codes, sf, nan = ref.encode(x)
    got = a.codes.cpu().numpy()
    assert np.array_equal(a.sf.cpu().numpy(), sf), what
    assert np.array_equal(got[~nan], codes[~nan]), what
    assert ((got[nan] & 127) == 127).all(), what
    for dt in DTYPES:
        back = mx.act8_restore(a, out_dtype=dt)
        want = ref.decode(a.codes, a.sf, x.shape[1]).to(dt)  # Inf where a rounded value leaves the type's range
        assert torch.equal(torch.isnan(back), torch.isnan(want)), what
        keep = ~torch.isnan(want)
        assert torch.equal(back[keep], want[keep]), what
    return a


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("how", ["dense", "wide", "odd"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (5, 31), (2, 32), (7, 33), (130, 64), (9, 100), (3, 1000), (17, 1531),
                                   (64, 4096), (3, 11008), (2, 20000)])
def test_codes_and_values(mx, shape, how, dtype):
    x = workloads.draw("outliers", shape, 401, device="cuda").to(dtype)
    if dtype is torch.float32:
        x = x * 1.0009765  # values that bf16 does not have
    _check(mx, ref.layout(x, how))


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_finite_bf16_pattern(mx, dtype):
    x = workloads.all_bf16_patterns().view(-1, 32).cuda().to(dtype)
    _check(mx, x)
    perm = torch.randperm(x.numel(), generator=torch.Generator().manual_seed(5)).cuda()
    _check(mx, x.reshape(-1)[perm].view(-1, 32).contiguous())


def test_agrees_with_the_mxfp8_oracle_under_the_ceil_rule(mx):
    x = workloads.draw("student_t3", (96, 512), 402)
    q = orc.quantize(x.view(torch.int16).numpy().view(np.uint16), "mxfp8", rule="ceil")
    a = mx.act8_save(x.cuda())
    assert np.array_equal(a.codes.cpu().numpy(), q.codes)
    assert np.array_equal(a.sf.cpu().numpy(), q.sf_logical)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [32, 70, 256])
def test_infinities_nans_zeros_and_the_smallest_values(mx, cols, dtype):
    x = workloads.draw("normal", (8, cols), 403, device="cuda").to(dtype)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 5], x[2, 6], x[2, 7] = float("inf"), float("-inf"), float("nan")
    x[3] = float("nan")
    x[4] = float("inf")
    x[5] = 2.0 ** -133  # a bf16 subnormal: the exponent's lower bound
    x[6] *= 2.0 ** -126
    x[7] = torch.finfo(dtype).max
    a = _check(mx, x)
    assert torch.isfinite(mx.act8_restore(a)[2, 8:]).all()  # the neighbours of a NaN keep their values


def test_largest_value_of_a_group_never_saturates(mx):
    """Every significand of bf16 as a group's maximum: restored to within half a
    code spacing (1/16 relative), never cut to 448."""
    m = torch.arange(128, device="cuda").float() / 128 + 1
    x = torch.zeros(128, 32, device="cuda")
    x[:, 3] = m * 2.0 ** 20
    got = mx.act8_restore(mx.act8_save(x.to(torch.bfloat16)), out_dtype=torch.float32)[:, 3]
    assert ((got - x[:, 3]).abs() <= x[:, 3] / 16).all()


def test_pad_columns_hold_code_zero(mx):
    a = mx.Act8.empty(5, 70, torch.device("cuda"))
    a.codes.fill_(0xAB)
    mx.act8_save(workloads.draw("normal", (5, 70), 404, device="cuda"), out=a)
    assert (a.codes[:, 70:] == 0).all()


@pytest.mark.parametrize("shape", [(0, 64), (5, 0), (0, 0)])
def test_empty(mx, shape):
    a = mx.act8_save(torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
    assert mx.act8_restore(a).shape == shape


def test_writes_stay_inside_the_view(mx):
    x = workloads.draw("normal", (6, 50), 405, device="cuda")
    for at, ld in ((8, 72), (3, 61)):
        wide = torch.full((6, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        mx.act8_restore(mx.act8_save(x), out=wide[:, at:at + 50])
        assert (wide[:, :at] == 7).all() and (wide[:, at + 50:] == 7).all()
