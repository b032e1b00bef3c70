"""An optimizer that goes on from a saved state: the moments copied into m_all and v_all, the number into t."""
import pytest
import torch

pytestmark = pytest.mark.gpu

N = 5000


@pytest.fixture(scope="module")
def mx():
    import fp4_precision_gemms_gb300 as m
    m.build()
    return m


def tensors(seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(N, generator=g).cuda(), torch.randn(33, generator=g).cuda()]


def make(mx, state, capturable, params):
    return mx.AdamW(params, lr=1e-2, state=state, rounding="sr" if state == "8bit" else "rne", seed=5, capturable=capturable)


def parts(opt, state):
    return [a for x in (opt.m_all, opt.v_all) for a in ((x.codes, x.sf) if state == "8bit" else (x,))]


def resumed(mx, opt, state, capturable):
    """A new optimizer with the parameters, moments and number of opt."""
    other = make(mx, state, capturable, [p.clone() for p in opt.params])
    for mine, given in zip(parts(other, state), parts(opt, state)):
        mine.copy_(given)
    other.t = opt.t
    return other


def equal(a, b, state):
    return all(torch.equal(x, y) for x, y in zip([*a.params, *parts(a, state)], [*b.params, *parts(b, state)]))


@pytest.mark.parametrize("state", ["fp32", "8bit"])
@pytest.mark.parametrize("capturable", [False, True])
def test_goes_on(mx, state, capturable):
    grads = [tensors(10 + k) for k in range(6)]
    first = make(mx, state, capturable, tensors(1))
    for g in grads[:3]:
        first.step(g)
    assert first.t == 3
    second = resumed(mx, first, state, capturable)
    assert second.t == 3
    for g in grads[3:]:
        first.step(g)
        second.step(g)
        assert equal(first, second, state)
    assert first.t == second.t == 6


@pytest.mark.parametrize("state", ["fp32", "8bit"])
def test_goes_on_after_replays(mx, state):
    """The number counts the replays of a captured step, not its capture."""
    grads = tensors(10)
    opt = make(mx, state, True, tensors(1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(grads)
    assert opt.t == 0
    for _ in range(4):
        graph.replay()
    assert opt.t == 4
    eager = make(mx, state, True, tensors(1))
    for _ in range(4):
        eager.step(grads)
    second = resumed(mx, opt, state, True)
    assert equal(opt, eager, state) and second.t == 4
    graph.replay()
    eager.step(grads)
    second.step(grads)
    assert opt.t == eager.t == second.t == 5
    assert equal(opt, eager, state) and equal(opt, second, state)
    opt.t = 100  # the captured step goes on from it too
    second.t = 100
    graph.replay()
    second.step(grads)
    assert opt.t == 101 and equal(opt, second, state)


def test_a_captured_step_has_no_fixed_number(mx):
    """A number that the graph would write at every replay, or that cannot be read yet, is refused."""
    grads = tensors(10)
    opt = make(mx, "fp32", True, tensors(1))
    opt.step(grads, t=7)
    assert opt.t == 7
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(mx.MXError):
            opt.step(grads, t=7)
        with pytest.raises(mx.MXError):
            opt.t
        with pytest.raises(mx.MXError):
            opt.t = 3
        opt.step(grads)
    graph.replay()
    assert opt.t == 8


@pytest.mark.parametrize("capturable", [False, True])
def test_a_refused_step_is_not_counted(mx, capturable):
    grads = tensors(10)
    opt = make(mx, "fp32", capturable, tensors(1))
    opt.step(grads)
    for kw in (dict(lr=float("nan")), dict(lr=float("nan"), t=50)):
        with pytest.raises(mx.MXError):
            opt.step(grads, **kw)
        assert opt.t == 1
    for bad in (-1, -7):
        with pytest.raises(mx.MXError):
            opt.t = bad
    assert opt.t == 1
