"""GPU checks of the per-head-decay delta rule over the whole range that its contract
names (beta |k|^2 <= 2), against the 64-bit token recurrence: updates that reflect the
state, repeated keys, keys of very different sizes beside each other."""
import pytest
import torch

from gated_delta_rule_35_amd import kda_gdr_fwd, load_library
from tests import gdr_ref as ref
from tests.test_gpu_gdr import SCALE, args, say

pytestmark = pytest.mark.gpu
# o = scale (e^G q . S + sum_j A_j u_j) before its rounding, relative to scale |q| Sabs, which holds
# all of its terms: fp32 sums of at most 128 terms 128 2^-24 = 7.6e-6, S, A and u in two bf16 parts
# 2^-18 each (each part's rounding is 2^-9 of what it rounds), S and u themselves 1.2e-5 of
# the magnitudes that make them up; 3.1e-5 together, less than 2^-14.
OUTPUT_REL = 2.0 ** -14


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    load_library()
    yield


def state_magnitude(x):
    """The sum of the magnitudes of the terms that make up the final states: |S_0| and every
    |k_t| |u_t|, [N, Hv, 128, 128].  Where beta is near 2 and a key repeats, S = sum k u with
    u_t = S_t - S_{t-1} of alternating signs and twice S's size, so that 64 tokens' terms are
    128 times the state they leave; a sum of n terms in fp32, of operands with 22 bits, is
    off by 1.2e-5 (gdr_ref) of the terms' magnitudes, not of what cancels to.  An update with
    beta |k|^2 <= 2 does not expand a state, so that earlier tokens' errors add up to no more."""
    d = {n: (t.double() if t is not None else None) for n, t in x.items()}
    found = []
    for b in range(x["q"].shape[0]):
        R = x["v"].shape[2] // x["q"].shape[2]
        k = d["k"][b].repeat_interleave(R, dim=1)
        S = d["h0"][b] if d["h0"] is not None else torch.zeros(x["v"].shape[2], 128, 128, dtype=torch.float64)
        M = S.abs()
        for t in range(k.shape[0]):
            S = torch.exp(d["g"][b, t])[:, None, None] * S
            M = torch.exp(d["g"][b, t])[:, None, None] * M
            u = d["beta"][b, t][:, None] * (d["v"][b, t] - torch.einsum("hk,hkv->hv", k[t], S))
            S, M = S + k[t][:, :, None] * u[:, None, :], M + k[t].abs()[:, :, None] * u.abs()[:, None, :]
        found.append(M)
    return torch.stack(found)


def check_range(x):
    """States to the tests' bound, relative to the magnitudes that make them up; o to check_output's."""
    d = ref.cuda(x)
    out, hT = kda_gdr_fwd(*args(d), initial_state=d["h0"], final_state=True)
    torch.cuda.synchronize()
    o_ref, h_ref = ref.forward(x, SCALE)
    got, h = out.cpu().double(), hT.cpu().double()
    assert torch.isfinite(got).all() and torch.isfinite(h).all()
    err, most = (h - h_ref).flatten(2).norm(dim=-1), state_magnitude(x).flatten(2).norm(dim=-1)
    assert (err <= ref.STATE_REL * most).all(), (err / most).max()
    err, most = (got - o_ref).abs() - ref.BF16_HALF * o_ref.abs(), ref.forward_magnitude(x, SCALE)
    assert (err <= OUTPUT_REL * most).all(), float((err / most).max())


def alternating(T, size, beta, one_hot, Hv=1):
    """One unit key for every token, values that change sign from token to token, no decay:
    with beta 2 each update turns the state's part along the key over and adds 2 v, so that
    the state grows by 2 |v| a token and the corrections reach (2 T - 1) beta |v|."""
    gen = torch.Generator().manual_seed(T)
    x = ref.make(1, T, 1, Hv, seed=T)
    if one_hot:
        k = torch.zeros(128)
        k[37] = 1.0
    else:   # sixteen entries of 1/4: a unit row that bf16 holds
        k = torch.zeros(128)
        k[torch.randperm(128, generator=gen)[:16]] = 0.25
    x["k"] = k.expand(1, T, 1, 128).contiguous().bfloat16()
    sign = (1.0 - 2.0 * (torch.arange(T) % 2))[None, :, None, None]
    x["v"] = (sign * size * torch.ones(1, T, Hv, 128)).bfloat16()
    x["g"] = torch.zeros(1, T, Hv)
    x["beta"] = torch.full((1, T, Hv), beta)
    return x


@pytest.mark.parametrize("beta,size", [(2.0, 512.0), (2.0, 400.0), (2.0, 1.0), (1.5, 512.0), (1.9, 3e6)])
@pytest.mark.parametrize("one_hot", [True, False])
def test_updates_that_reflect_the_state(beta, size, one_hot):
    say(f"gdr_fwd, one key, beta={beta}, values +-{size}")
    for T in (64, 200):
        check_range(alternating(T, size, beta, one_hot))


@pytest.mark.parametrize("hi", [1.0, 2.0])
def test_random_updates_up_to_two(hi):
    """Unit keys that nearly repeat and random beta up to 2, without and with decay."""
    for lo, most in ((0.0, 0.0), (0.001, 0.5)):
        say(f"gdr_fwd, beta up to {hi}, log-decays {lo} to {most}")
        x = ref.make(2, 200, 2, 4, h0=True, seed=5, lo=max(lo, 1e-9), hi=max(most, 1e-9))
        gen = torch.Generator().manual_seed(6)
        base = torch.randn(128, generator=gen)
        k = x["k"].float() * 0.3 + base / base.norm()
        # bf16 keeps a row's length to 2^-8 of itself: 1 - 2^-7 stays below one
        x["k"] = (k / k.norm(dim=-1, keepdim=True) * (1 - 2.0 ** -7)).bfloat16()
        x["beta"] = hi * (0.5 + 0.5 * torch.rand(2, 200, 4, generator=gen))
        x["v"] = (x["v"].float() * 300).bfloat16()
        check_range(x)


@pytest.mark.parametrize("span", [3, 6, 9])
def test_keys_of_different_sizes_beside_each_other(span):
    """Keys of 2^-span to 2^span, each with beta near the most that its size allows."""
    say(f"gdr_fwd, keys of 2^-{span} to 2^{span} in one chunk")
    x = ref.make(1, 200, 1, 2, seed=span)
    gen = torch.Generator().manual_seed(span)
    size = 2.0 ** (2 * span * torch.rand(1, 200, 1, 1, generator=gen) - span)
    x["k"] = (x["k"].float() * size).bfloat16()
    n2 = x["k"].double().pow(2).sum(-1)
    x["beta"] = (1.9 * torch.rand(1, 200, 2, generator=gen) / n2).float()
    # values in proportion to what the key reads of a state of order one
    x["v"] = (x["v"].float() * size).bfloat16()
    x["h0"] = torch.randn(1, 2, 128, 128, generator=gen)
    check_range(x)


def check_output(x, cu=None):
    """o to half a bf16 step and OUTPUT_REL of what is summed for it."""
    d = ref.cuda(x)
    o, _ = kda_gdr_fwd(*args(d), initial_state=d["h0"], cu_seqlens=None if cu is None else cu.cuda())
    torch.cuda.synchronize()
    want, most = ref.forward(x, SCALE, cu)[0], ref.forward_magnitude(x, SCALE, cu)
    err = (o.cpu().double() - want).abs() - ref.BF16_HALF * want.abs()
    assert (err <= OUTPUT_REL * most).all(), float((err / most).max())


@pytest.mark.parametrize("beta,size", [(2.0, 400.0), (1.5, 512.0), (1.9, 3e6)])
@pytest.mark.parametrize("one_hot", [True, False])
def test_output_where_its_terms_cancel(beta, size, one_hot):
    """o = sum A_j u_j of alternating signs, a hundredth of its terms."""
    say(f"gdr_fwd, o of cancelling terms, beta={beta}, values +-{size}")
    check_output(alternating(200, size, beta, one_hot, Hv=2))


def test_output_of_queries_across_a_large_state():
    """A state that all keys share, read by queries nearly at right angles to it; keys of 1.4 with
    beta 1 beside keys of 8 with beta 1/32."""
    say("gdr_fwd, queries across the state")
    x = ref.make(1, 130, 1, 2, seed=3, lo=1e-4, hi=1e-3)
    long = (torch.arange(130) % 2 == 0)[None, :, None]
    base = torch.randn(128, generator=torch.Generator().manual_seed(8)).sign() * 128 ** -0.5
    x["k"] = torch.where(long[..., None], 8.0, 1.4).mul(base).expand(1, 130, 1, 128).contiguous().bfloat16()
    x["beta"] = torch.where(long, 1 / 32.0, 1.0).expand(1, 130, 2).contiguous()
    x["h0"] = 900.0 * 8 * base[None, None, :, None].expand(1, 2, 128, 128).contiguous()
    q = x["q"].float()
    x["q"] = (q - (q @ base)[..., None] * base).bfloat16()
    check_output(x)


@pytest.mark.parametrize("lens", [None, [65, 0, 1, 130], [0, 1, 200, 64, 65, 3, 130, 128] * 8])
def test_output_of_ordinary_inputs(lens):
    """Half heads, packed sequences, and whole heads (64 sequences of 16 heads)."""
    say(f"gdr_fwd, o against its terms, lengths {lens if lens is None else lens[:8]}")
    if lens is None:
        return check_output(ref.make(2, 200, 2, 4, h0=True, seed=5))
    x = ref.make(1, sum(lens), 4, 16, h0=True, N=len(lens), seed=6)
    check_output(x, torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32))


@pytest.mark.parametrize("beta", [3.0, 2.5])
def test_updates_that_expand_the_state(beta):
    """beta |k|^2 beyond 2: the state grows by beta - 1 a token, 2^60 in all at most.  Errors grow as
    it does, by no more than the terms that make it up."""
    say(f"gdr_fwd, one key, beta={beta}")
    check_range(alternating(60, 1.0, beta, True))
    x = ref.make(1, 60, 1, 2, h0=True, seed=9)
    x["beta"] = torch.full((1, 60, 2), beta)
    check_range(x)


def test_sizes_far_apart_in_one_column():
    """A large state that the gates forget within a chunk, then values 2^-40 of it: what stands
    behind the reset has fp32's accuracy of itself, as token by token."""
    say("gdr_fwd, a state 2^40 above the values after a reset")
    x = ref.make(1, 100, 1, 2, h0=True, seed=10)
    x["h0"] = x["h0"] * 2.0 ** 40
    x["g"][0, 7] = -100.0
    d = ref.cuda(x)
    out, hT = kda_gdr_fwd(*args(d), initial_state=d["h0"], final_state=True)
    torch.cuda.synchronize()
    want, state = ref.forward(x, SCALE)
    most = ref.forward_magnitude(x, SCALE)
    err = (out.cpu().double() - want).abs() - ref.BF16_HALF * want.abs()
    assert (err <= OUTPUT_REL * most).all(), float((err / most).max())
    ref.assert_states(hT, state, "final state")
