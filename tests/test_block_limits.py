"""The largest launches of the norms' and the scan's gradients: what no grid can hold is turned away on the host before
anything is launched.  On the CPU; the data pointers are never dereferenced, and a workspace that is too small ends
the calls that are allowed."""
import pytest

from tests.test_block_boundary import F32, at, gated_args, gated_bwd, lib  # noqa: F401
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
