"""What rounding 8-bit moments to nearest means for training, and that it is said where it was not asked for."""
import warnings

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def test_said_where_not_asked_for(mx):
    p = lambda: [torch.ones(64, device="cuda")]  # noqa: E731
    with pytest.warns(UserWarning, match="never fall"):
        opt = mx.AdamW(p(), state="8bit")
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        given = mx.AdamW(p(), state="8bit", rounding="rne")
        mx.AdamW(p(), state="8bit", rounding="sr")
        mx.AdamW(p())
    for o in (opt, given):  # the default is to nearest
        o.step([torch.full((64,), 0.37, device="cuda")])
    assert torch.equal(opt.v[0].codes, given.v[0].codes)


@pytest.mark.parametrize("rounding", ["rne", "sr"])
def test_a_root_falls(mx, rounding):
    """300 steps without a gradient: the root of the second moment falls to 0.999^150 = 0.861 of itself.  To nearest
    it stays where it is.  Stochastically a step of the chain falls by one of 2^-9 to 2^-10 of the value times 64 to
    128, with the right mean: over 32768 values whose deviations are below a code's distance (0.125) each, 5 standard
    deviations of the mean are 0.0035; u16 numbers cut each step's probability by 2^-16 of a distance at most, 300 steps
    0.0006."""
    n = 1 << 15
    opt = mx.AdamW([torch.zeros(n, device="cuda")], state="8bit", rounding=rounding, seed=9, betas=(0.9, 0.999))
    opt.v[0].codes.fill_(0x7E)  # 448
    opt.v[0].sf.fill_(127 - 8)  # 1.75
    zero = [torch.zeros(n, device="cuda")]
    for _ in range(300):
        opt.step(zero)
    mean = float(mx.act8_restore(opt.v[0], out_dtype=torch.float32).double().mean()) / 1.75
    if rounding == "rne":
        assert mean == 1.0
    else:
        assert abs(mean - 0.999 ** 150) < 0.0035 + 0.0006
