"""GPU checks of the selective state space scan where a result's terms cancel: its bf16 results are far smaller than what
they are summed from, so that what a product's operands leave out would show.

Tolerance.  Decays and steps are exact here (A = -1e-30: e^{d A} is 1 in 32 and in 64 bits; the steps are given).  A
result has two large terms, each a product of a bf16 number and one of 24 bits that is the sum of at most three exact
products, formed with at most two roundings; in the parts that a matrix product takes it is at most three products,
so that six additions follow, each off by at most 2^-23 of the terms, in whichever way they round: 2 2 + 6 2 units of
2^-24, and 24 with the parts' own remainders of 2^-27 and the zeros between them, beside the rounding of the result
itself.  16 bits of an operand would be off by up to 2^-18 = 64 units of its term."""
import pytest
import torch

from gated_delta_rule_35_amd import load_library
from tests import ssm_ref as ref
from tests.test_gpu_ssm import bwd, fwd, say

pytestmark = pytest.mark.gpu
OFF = 24 * 2.0 ** -24
SHAPES = [(64, 128), (64, 64), (128, 128), (128, 64)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    load_library()
    yield


def zeros(B, T, H, P, S):
    """A case whose inputs are all zero but for the steps, which are 1."""
    z = lambda *s: torch.zeros(*s)  # noqa: E731
    return dict(x=z(B, T, H, P).bfloat16(), dt=z(B, T, H) + 1, A=z(H) - 1e-30, B=z(B, T, 1, S).bfloat16(), C=z(B, T, 1, S).bfloat16(),
                D=None, bias=None, h0=None, dy=z(B, T, H, P).bfloat16(), dlast=None, softplus=False)


def rand(gen, *s):
    """Numbers of 1 to 2 with 24 random bits."""
    return 1 + torch.rand(*s, generator=gen)


def pairs(gen, B, T):
    """Two tokens for each row, the first ones in one chunk, others in different ones."""
    i = torch.randint(0, T - 1, (B,), generator=gen)
    i[:B // 2] %= 62
    j = torch.minimum(i + 1 + torch.randint(0, 40, (B,), generator=gen), torch.full((B,), T - 1))
    j[:B // 2] = torch.minimum(j[:B // 2], torch.full((B // 2,), 63))
    return i, j


def near(v, gen):
    """v but for its last bits: off by up to 2^-13 of itself."""
    return v * (1 + 2.0 ** -13 * torch.rand(v.shape, generator=gen))


def check_y(c, least):
    y, _ = fwd(ref.cuda(c))
    torch.cuda.synchronize()
    want, mag, _, _ = ref.run(c)
    assert float(((want.abs() < 2.0 ** -10 * mag) & (mag > 0)).sum()) >= least   # they do cancel
    ref.close(y, want, OFF * mag, "y")


def check(c, name, least):
    g = bwd(ref.cuda(c), d_initial_state=False)
    torch.cuda.synchronize()
    want, mag = ref.gradients(c)
    assert float(((want[name].abs() < 2.0 ** -10 * mag[name]) & (mag[name] > 0)).sum()) >= least
    ref.close(g[name], want[name], OFF * mag[name], name)


@pytest.mark.parametrize("P,S", SHAPES)
def test_tokens_against_each_other(P, S):
    """y = d_i x_i - d_j x_i: the pair matrix, and the state where the two are in different chunks."""
    say(f"ssm cancel pairs P={P} S={S}")
    gen = torch.Generator().manual_seed(P + S)
    B, T, H = 24, 100, 2
    c = zeros(B, T, H, P, S)
    c["B"][..., 5], c["C"][..., 5] = 1, 1
    for b, (i, j) in enumerate(zip(*pairs(gen, B, T))):
        v = rand(gen, H, P).bfloat16()
        c["x"][b, i], c["x"][b, j] = v, -v
        c["dt"][b, i] = rand(gen, H)
        c["dt"][b, j] = near(c["dt"][b, i], gen)
    check_y(c, B * H * P)


@pytest.mark.parametrize("P,S", SHAPES)
def test_channels_of_a_state_against_each_other(P, S):
    """y = S_a - S_b for an initial state."""
    say(f"ssm cancel state P={P} S={S}")
    gen = torch.Generator().manual_seed(P + S + 1)
    c = zeros(2, 70, 2, P, S)
    c["h0"] = torch.zeros(2, 2, S, P)
    c["h0"][:, :, 3] = rand(gen, 2, 2, P)
    c["h0"][:, :, S - 6] = near(c["h0"][:, :, 3], gen)
    c["C"][..., 3], c["C"][..., S - 6] = 1, -1
    check_y(c, 2 * 70 * 2 * P)


@pytest.mark.parametrize("P,S", SHAPES)
def test_a_state_against_the_token_itself(P, S):
    """y = S_a + D x with D x near -S_a."""
    say(f"ssm cancel D P={P} S={S}")
    gen = torch.Generator().manual_seed(P + S + 2)
    H = 64
    c = zeros(1, 70, H, P, S)
    c["D"] = rand(gen, H)
    c["h0"] = near(c["D"], gen)[None, :, None, None] * torch.ones(1, H, S, P)
    c["C"][..., 3] = -1
    c["x"] = c["x"] + 1
    check_y(c, 70 * H * P)


def fine(gen, n):
    """n triples of bf16 numbers whose sum has 24 bits, all but its last seven or eight the same."""
    r = (1 + torch.rand(1, generator=gen)).bfloat16().float() * 2.0 ** -8
    s = (1 + torch.rand(n, generator=gen)).bfloat16().float() * 2.0 ** -16
    return torch.stack([torch.ones(n), r.expand(n), s], dim=1)


@pytest.mark.parametrize("P,S", SHAPES)
def test_dC_of_tokens_against_each_other(P, S):
    """dC_i = d_j B_j - d_k B_k."""
    say(f"ssm cancel dC P={P} S={S}")
    gen = torch.Generator().manual_seed(P + S + 3)
    B, T = 24, 100
    c = zeros(B, T, 1, P, S)
    c["dy"][..., 7] = 1
    for b, (i, j) in enumerate(zip(*pairs(gen, B, T))):
        v = rand(gen, S).bfloat16()
        c["B"][b, i, 0], c["B"][b, j, 0] = v, -v
        c["x"][b, [i, j], 0, 7] = 1
        c["dt"][b, i] = rand(gen, 1)
        c["dt"][b, j] = near(c["dt"][b, i], gen)
    check(c, "dC", B * S)


@pytest.mark.parametrize("P,S", SHAPES)
def test_dB_of_tokens_against_each_other(P, S):
    """dB_k = <dy_i, x_k> C_i - <dy_j, x_k> C_j."""
    say(f"ssm cancel dB P={P} S={S}")
    gen = torch.Generator().manual_seed(P + S + 4)
    B, T = 24, 100
    c = zeros(B, T, 1, P, S)
    c["x"][..., 0, [3, 20, P - 1]] = 1
    for b, (i, j) in enumerate(zip(*pairs(gen, B, T))):
        v = rand(gen, S).bfloat16()
        c["C"][b, i, 0], c["C"][b, j, 0] = v, -v
        for t, f in zip((i, j), fine(gen, 2)):
            c["dy"][b, t, 0, [3, 20, P - 1]] = f.bfloat16()
    check(c, "dB", B * S)


@pytest.mark.parametrize("P,S", SHAPES)
def test_dx_of_tokens_against_each_other(P, S):
    """dx_k = <C_i, B_k> dy_i - <C_j, B_k> dy_j."""
    say(f"ssm cancel dx P={P} S={S}")
    gen = torch.Generator().manual_seed(P + S + 5)
    B, T, H = 24, 100, 2
    c = zeros(B, T, H, P, S)
    c["B"][..., 0, [3, 20, S - 1]] = 1
    for b, (i, j) in enumerate(zip(*pairs(gen, B, T))):
        v = rand(gen, H, P).bfloat16()
        c["dy"][b, i], c["dy"][b, j] = v, -v
        for t, f in zip((i, j), fine(gen, 2)):
            c["C"][b, t, 0, [3, 20, S - 1]] = f.bfloat16()
    check(c, "dx", B * H * P)


@pytest.mark.parametrize("P,S", SHAPES)
def test_dx_of_channels_of_a_state_against_each_other(P, S):
    """dx = dS_a - dS_b for the gradient of a final state."""
    say(f"ssm cancel dS P={P} S={S}")
    gen = torch.Generator().manual_seed(P + S + 6)
    c = zeros(2, 70, 3, P, S)
    c["dlast"] = torch.zeros(2, 3, S, P)
    c["dlast"][:, :, 3] = rand(gen, 2, 3, P)
    c["dlast"][:, :, S - 6] = near(c["dlast"][:, :, 3], gen)
    c["B"][..., 3], c["B"][..., S - 6] = 1, -1
    check(c, "dx", 2 * 70 * 3 * P)


@pytest.mark.parametrize("P,S", SHAPES)
def test_dx_of_a_state_against_the_token_itself(P, S):
    """dx = dS_a + D dy with D dy near -dS_a."""
    say(f"ssm cancel dS D P={P} S={S}")
    gen = torch.Generator().manual_seed(P + S + 7)
    H = 16
    c = zeros(1, 70, H, P, S)
    c["D"] = rand(gen, H)
    c["dlast"] = near(c["D"], gen)[None, :, None, None] * torch.ones(1, H, S, P)
    c["B"][..., 3] = -1
    c["dy"] = c["dy"] + 1
    check(c, "dx", 70 * H * P)
