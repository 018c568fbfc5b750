"""GPU checks against 64 bits of the convolution and the scan at sizes that take their longer loops: runs of several
batches of tokens, segments of wide heads, sets of several heads."""
import ctypes

import pytest
import torch

from gated_delta_rule_35_amd import kda_conv, load_library
from tests import block_ref, ssm_ref as ref
from tests.block_ref import TYPES
from tests.test_gpu_ssm import check_forward, check_gradients, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    load_library()
    yield


class Split(ctypes.Structure):
    _fields_ = [("run", ctypes.c_int32), ("lanes", ctypes.c_int32), ("tiles", ctypes.c_int64), ("cols", ctypes.c_int64)]


def conv_split(tokens, channels, bwd):
    """The library's own split of a convolution (kda::conv_split)."""
    f = load_library()._ZN3kda10conv_splitEllb
    f.argtypes, f.restype = [ctypes.c_int64, ctypes.c_int64, ctypes.c_bool], Split
    return f(tokens, channels, bwd)


@pytest.mark.parametrize("B,T,C,W,kind,act,cu", [
    (1, 16384, 4096, 4, "bf16", "silu", [0, 1000, 1031, 1031, 5003, 5004, 16379]), (3, 5555, 4104, 3, "f16", None, None),
    (1, 16400, 4096, 2, "f32", "silu", [0, 7, 16400])])
def test_forward_in_runs_of_four_batches(B, T, C, W, kind, act, cu):
    """A run of 32 tokens asks for its rows eight at a time: the window goes on from batch to batch, sequences end inside."""
    say(f"conv runs of 32 B={B} T={T} C={C} W={W} {kind}")
    assert conv_split(B * T, C, False).run == 32
    gen = torch.Generator("cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    n = B if cu is None else len(cu) - 1
    x, w, bias, state = rnd(B, T, C).to(TYPES[kind]), rnd(C, W) / W ** 0.5, 0.3 * rnd(C), rnd(n, W - 1, C).to(TYPES[kind])
    y, last = kda_conv(x, w, bias, activation=act, cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"),
                       initial_state=state, final_state=True, out=torch.full_like(x, 7.0))
    torch.cuda.synchronize()
    for c in (0, C - 24):   # channels do not mix, so that some of them are a case of their own
        some = slice(c, c + 24)
        want, mag, wl = block_ref.conv_batch(x[..., some].cpu(), w[some].cpu(), bias[some].cpu(), act, cu, state[..., some].cpu())
        got, real = y[..., some].cpu(), ~torch.isnan(want)
        block_ref.close(got[real], want[real], 2.0 ** -20 * mag[real], "y")
        assert (got[~real] == 7).all() and torch.equal(last[..., some].cpu().double(), wl)


@pytest.mark.parametrize("H,P,S,G,cu", [(4, 128, 128, 2, [0, 650, 651, 700]), (4, 128, 128, 2, None), (2, 64, 128, 1, [0, 30, 700]),
                                        (3, 128, 64, 1, None), (6, 64, 128, 1, None)])
def test_segments(H, P, S, G, cu):
    """Segments side by side, chained, of heads and states of 128."""
    say(f"ssm segments H={H} P={P} S={S} G={G} {cu}")
    c = ref.make(1, 700, H, P, S, G, N=1 if cu is None else len(cu) - 1, h0=True, seed=H + P, fast=2.0)
    c["bias"] = c["bias"] - 2   # slow decays, so that states of far segments count
    check_forward(c, cu)
    check_gradients(c, cu)


@pytest.mark.parametrize("H,P,S,G", [(5, 64, 128, 1), (3, 128, 128, 1), (4, 128, 64, 1), (6, 64, 64, 2)])
def test_one_set_of_several_heads(H, P, S, G):
    """So many chunks that a group's heads are taken one after the other, dB and dC kept in registers over them."""
    say(f"ssm one set H={H} P={P} S={S} G={G}")
    cu = [0]
    for n in [70, 130] + [1 + i % 2 for i in range(510 // G)]:
        cu.append(cu[-1] + n)
    c = ref.make(1, cu[-1], H, P, S, G, N=len(cu) - 1, h0=True, seed=P + S)
    assert (cu[-1] // 64 + len(cu)) * G >= 512   # chunk slots and groups, two for each compute unit
    check_gradients(c, cu)
