"""Which calls of the gated block for few tokens are cut along K, seen by the room that they ask for: partial
sums where they are, nothing beside the tokens' operand where they are not."""
import pytest

import fp4_precision_gemms_gb300 as mx

FP8 = ("mxfp8", "moss")


@pytest.fixture(scope="module", autouse=True)
def built():
    mx.build()


def room(T, K, F, fmt):
    """Bytes beyond the tokens' operand."""
    n = mx.FORMATS[fmt]
    up = lambda b: -(-b // 256) * 256  # noqa: E731
    operand = up(mx.lib().mx_codes_bytes(n, T, K)) + up(mx.lib().mx_sf_bytes(n, T, K))
    return mx.gated_workspace_bytes(T, K, F, fmt, "fwd_quantized") - operand


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4", "moss"])
@pytest.mark.parametrize("T,K,tiles", [(1, 4096, 112), (48, 4096, 112), (48, 4096, 80), (48, 4096, 86), (64, 1024, 86), (1, 1024, 32),
                                       (64, 8192, 92), (1, 4096, 152), (64, 1024, 8)])
def test_whole(fmt, T, K, tiles):
    assert room(T, K, 128 * tiles, fmt) < 4096


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("K,tiles", [(1024, 8), (4096, 32), (4096, 64), (4096, 160), (8192, 8), (8192, 64), (768, 320), (4096, 304)])
@pytest.mark.parametrize("pass_", ["fwd", "fwd_quantized"])
def test_serves_fewer_tokens(fmt, K, tiles, pass_):
    """Cut with few tokens and whole with more: the room for more holds what fewer need."""
    sizes = [mx.gated_workspace_bytes(T, K, 128 * tiles, fmt, pass_) for T in range(1, 65)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4", "moss"])
@pytest.mark.parametrize("T,K,tiles", [(1, 4096, 160), (16, 8192, 176), (1, 8192, 32), (1, 8192, 8), (16, 8192, 32), (48, 8192, 160),
                                       (1, 4096, 320)])
def test_cut(fmt, T, K, tiles):
    """Two slots of sums a CTA at most, for the tokens in fours."""
    most = 152 * 2 * 2 * 128 * -(-T // 4) * 16
    assert 4096 < room(T, K, 128 * tiles, fmt) <= most + 4 * tiles + 1024


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4", "nvfp4_local"])
def test_many_tokens(fmt):
    assert room(65, 8192, 1024, fmt) < 8192
