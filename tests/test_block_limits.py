"""Launches of the convolution's, the norms' and the scan's gradients: what no grid can hold is turned away on the host before
anything is launched.  On the CPU; the data pointers are never dereferenced, and a workspace that is too small ends
the calls that are allowed."""
import pytest

from tests.test_block_boundary import F32, at, gated_args, gated_bwd, lib  # noqa: F401
from tests.test_gpu_block_runs import conv_split
from tests.test_ssm_boundary import bwd, good


@pytest.mark.parametrize("H,D,err", [(1 << 16, 8192, "UNSUPPORTED"), (1 << 16, 8184, "WORKSPACE"), ((1 << 16) - 1, 8192, "WORKSPACE")])
def test_weight_gradients_of_a_norm(lib, H, D, err):  # noqa: F811
    """Sums of 32 weights a work-group of 256 threads, fewer than 2^32 threads in all."""
    a = gated_args(T_=1, H=H, D=D, heads=True)
    assert gated_bwd(lib, a, size=1) == err
    if err == "UNSUPPORTED":   # one weight for all heads, or no weights' gradients to form
        assert gated_bwd(lib, {**a, "w": at(3, [D], F32), "dw": at(8, [D], F32)}, size=1) == "WORKSPACE"


@pytest.mark.parametrize("T,H,err", [(1 << 28, 1, "UNSUPPORTED"), ((1 << 28) - 64, 1, "WORKSPACE"), (1 << 27, 2, "WORKSPACE")])
def test_numbers_of_the_scans_gradients(lib, T, H, err):  # noqa: F811
    """1024 threads for 16 heads of a chunk, fewer than 2^32 in all."""
    assert bwd(lib, good(T_=T, H=H, G=1, S=64), size=1) == err


@pytest.mark.parametrize("tokens,channels,rounds", [(4096, 4352, 1), (8192, 4352, 1), (8192, 4096, 1), (32768, 1096, 1), (16384, 4352, 2)])
def test_convolution_gradients_fill_whole_rounds(lib, tokens, channels, rounds):  # noqa: F811
    """The device holds 512 of their work-groups at once."""
    k = conv_split(tokens, channels, True)
    assert 512 * (rounds - 1) < k.tiles * k.cols <= 512 * rounds and 8 <= k.run <= 40
    assert k.tiles * k.run * (256 // k.lanes) >= tokens and 8 * k.cols * k.lanes >= channels
