"""GPU checks of the per-head-decay delta rule's gradients token by token and head by head,
each against the magnitude of its own terms: a head, a chunk or a value channel far smaller
than the others is held as tightly as they are.

With S~ and S the state before and after token t's update, u = beta e its correction,
e = v - S~^T k, dS the gradient of S, du = dS^T k, M and N the same recurrences of magnitudes
(M = e^g M + |k| |u|, N likewise from scale |q| |do| and |k| beta |du|):

  dq = scale S do             scale M |do|
  dk = dS u - beta S~ du      N |u| + beta M~ |du|
  dv = beta du                beta N^T |k|
  dbeta = du . e              N^T |k| . |e| + |du| . (|v| + M~^T |k|)
  dg = <S~, dS>               <M~, N>
  dh0                         N

Tolerances, relative to those.  S, u, dS and du come from the walks, fp32 with 24-bit operands: 1.2e-5
(gdr_ref) of the magnitudes that make them up.  A term holds two of them: 2.4e-5; their fp16 parts
2 2^-22, P and E in two bf16 parts 2^-18, and fp32 sums of 128 terms 7.6e-6: 3.6e-5 < 2^-14 in
all.  dq, dk and dv are rounded to bf16 (2^-8 of the value) besides.  dg is a suffix sum over its
chunk of rows less columns of pairs (i, j): those with both tokens behind t cancel, having
been summed in fp32 over 64 terms in two orders, each off by 64 2^-24 = 2^-18; every pair's
magnitude is part of <M~, N> of the tokens between, so the cancelling ones leave at most 2^-17 of
the chunk's sum of <M~, N>.  What lies below fp32's normal numbers (e^-90 of something) may be
lost: 2^-100 of the largest term of any gradient is allowed besides.
"""
import pytest
import torch

from gated_delta_rule_35_amd import kda_gdr_bwd, load_library
from tests import gdr_ref as ref
from tests.test_gpu_gdr import SCALE, args, say

pytestmark = pytest.mark.gpu
TERMS, CANCELLED = 2.0 ** -14, 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    load_library()
    yield


def terms(x, do, dhT):
    """The gradients of a batch [B, T, ...] and their terms' magnitudes, in 64 bits."""
    d = {n: (t.double() if t is not None else None) for n, t in x.items()}
    B, T, Hq, _ = x["q"].shape
    Hv = x["v"].shape[2]
    R = Hv // Hq
    grad = dict(dq=torch.zeros(B, T, Hq, 128).double(), dk=torch.zeros(B, T, Hq, 128).double(),
                dv=torch.zeros(B, T, Hv, 128).double(), dg=torch.zeros(B, T, Hv).double(),
                dbeta=torch.zeros(B, T, Hv).double(), dh0=torch.zeros(B, Hv, 128, 128).double())
    most = {n: t.clone() for n, t in grad.items()}
    mv = lambda A, y: torch.matmul(A, y[..., None])[..., 0]  # noqa: E731  [h, i, j] [h, j]
    group = lambda y: y.view(Hq, R, 128).sum(1)  # noqa: E731
    for b in range(B):
        q, k = (d[n][b].repeat_interleave(R, dim=1) for n in ("q", "k"))
        v, g, beta, dO = d["v"][b], d["g"][b], d["beta"][b], do[b].double()
        S = d["h0"][b].clone() if d["h0"] is not None else torch.zeros(Hv, 128, 128).double()
        M, kept = S.abs(), []
        for t in range(T):
            S, M = torch.exp(g[t])[:, None, None] * S, torch.exp(g[t])[:, None, None] * M
            e = v[t] - mv(S.transpose(1, 2), k[t])
            u = beta[t][:, None] * e
            kept.append((S, M, e, u))
            S, M = S + k[t][:, :, None] * u[:, None], M + k[t].abs()[:, :, None] * u.abs()[:, None]
        dS = dhT[b].double().clone() if dhT is not None else torch.zeros_like(S)
        N = dS.abs()
        for t in reversed(range(T)):
            S0, M0, e, u = kept[t]
            S1, M1 = S0 + k[t][:, :, None] * u[:, None], M0 + k[t].abs()[:, :, None] * u.abs()[:, None]
            grad["dq"][b, t] = group(SCALE * mv(S1, dO[t]))
            most["dq"][b, t] = group(SCALE * mv(M1, dO[t].abs()))
            dS = dS + SCALE * q[t][:, :, None] * dO[t][:, None]
            N = N + SCALE * q[t].abs()[:, :, None] * dO[t].abs()[:, None]
            du, Du = mv(dS.transpose(1, 2), k[t]), mv(N.transpose(1, 2), k[t].abs())
            bt = beta[t][:, None]
            grad["dk"][b, t] = group(mv(dS, u) - bt * mv(S0, du))
            most["dk"][b, t] = group(mv(N, u.abs()) + bt.abs() * mv(M0, du.abs()))
            grad["dv"][b, t], most["dv"][b, t] = bt * du, bt.abs() * Du
            grad["dbeta"][b, t] = (du * e).sum(-1)
            most["dbeta"][b, t] = (Du * e.abs()).sum(-1) + (du.abs() * (v[t].abs() + mv(M0.transpose(1, 2), k[t].abs()))).sum(-1)
            dS, N = dS - k[t][:, :, None] * (bt * du)[:, None], N + k[t].abs()[:, :, None] * (bt * du).abs()[:, None]
            grad["dg"][b, t], most["dg"][b, t] = (S0 * dS).sum((1, 2)), (M0 * N).sum((1, 2))
            dS, N = torch.exp(g[t])[:, None, None] * dS, torch.exp(g[t])[:, None, None] * N
        grad["dh0"][b], most["dh0"][b] = dS, N
    return grad, most


def check(x, do=None, dhT=None, seed=0):
    gen = torch.Generator().manual_seed(seed + 5)
    do = torch.randn(x["v"].shape, generator=gen).bfloat16() if do is None else do
    d = ref.cuda(x)
    got = kda_gdr_bwd(*args(d), do.cuda(), initial_state=d["h0"], d_final_state=None if dhT is None else dhT.cuda(),
                      d_initial_state=True)
    torch.cuda.synchronize()
    want, most = terms(x, do, dhT)
    T, tiny = x["q"].shape[1], 2.0 ** -100 * max(float(m.max()) for m in most.values())
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0"):
        err = (got[n].cpu().double() - want[n]).abs()
        assert torch.isfinite(err).all(), n
        allowed = TERMS * most[n] + tiny
        if n in ("dq", "dk", "dv"):
            allowed = allowed + ref.BF16_HALF * want[n].abs()
        if n == "dg":
            chunk = torch.cat([most[n][:, a:a + 64].sum(1, keepdim=True).expand(-1, min(64, T - a), -1)
                               for a in range(0, T, 64)], dim=1)
            allowed = allowed + CANCELLED * chunk
        bad = err > allowed
        assert not bad.any(), (n, int(bad.sum()), float((err / allowed.clamp(min=1e-300)).max()),
                               bad.nonzero()[0].tolist())


def test_reference_against_autograd():
    x = ref.make(2, 70, 1, 2, h0=True, seed=1)
    gen = torch.Generator().manual_seed(2)
    do, dhT = torch.randn(x["v"].shape, generator=gen).bfloat16(), torch.randn(2, 2, 128, 128, generator=gen)
    got, most = terms(x, do, dhT)
    want = ref.gradients(x, SCALE, do, dhT)
    for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "beta"), ("dh0", "h0")):
        assert ref.rel(got[n], want[m]) <= 1e-12 and (most[n] >= got[n].abs() * (1 - 1e-9)).all()


def test_heads_of_very_different_decay():
    """Heads that keep everything beside heads that forget within a token: each decay a head's own."""
    say("gdr_bwd, log-decays of 1e-4 to 50 by head")
    x = ref.make(1, 200, 2, 8, h0=True, seed=3)
    rate = torch.tensor([1e-4, 50.0, 0.1, 5.0, 1.0, 20.0, 1e-2, 0.5])
    x["g"] = -rate * (0.5 + torch.rand(1, 200, 8, generator=torch.Generator().manual_seed(4)))
    check(x, dhT=0.1 * torch.randn(1, 8, 128, 128, generator=torch.Generator().manual_seed(5)))


@pytest.mark.parametrize("span", [10, 30])
def test_heads_of_very_different_sizes(span):
    say(f"gdr_bwd, values and output gradients of 2^-{span} to 2^{span} by head")
    x = ref.make(1, 200, 4, 4, h0=True, seed=6)
    size = 2.0 ** torch.tensor([-span, span, 0, -span // 2]).float()
    x["v"], x["h0"] = (x["v"].float() * size[:, None]).bfloat16(), x["h0"] * size[:, None, None]
    do = (torch.randn(1, 200, 4, 128, generator=torch.Generator().manual_seed(7)) * size.flip(0)[:, None]).bfloat16()
    check(x, do)


def test_value_channels_of_very_different_sizes():
    """Channels of values of 2^-20 to 2^20, and of the output's gradient the other way round, so that
    they all weigh alike in dbeta and dg; then both the same way, so that the large ones do."""
    x = ref.make(1, 150, 1, 2, h0=True, seed=8)
    size = 2.0 ** torch.linspace(-20, 20, 128).round()[torch.randperm(128, generator=torch.Generator().manual_seed(9))]
    x["v"], x["h0"] = (x["v"].float() * size).bfloat16(), x["h0"] * size
    do = torch.randn(1, 150, 2, 128, generator=torch.Generator().manual_seed(10))
    for way, s in (("against", 1 / size), ("with", size)):
        say(f"gdr_bwd, channels of 2^-20 to 2^20, output gradients {way} them")
        check(x, (do * s).bfloat16())


@pytest.mark.parametrize("kind", ["keys grow", "keys shrink", "keys start at zero", "values grow", "values shrink",
                                  "output gradients grow", "small state, large values later", "resets"])
def test_sizes_that_change_between_chunks(kind):
    say(f"gdr_bwd, {kind}")
    T = 270
    x = ref.make(1, T, 1, 2, h0=True, seed=31)
    step, do = torch.ones(T), torch.randn(1, T, 2, 128, generator=torch.Generator().manual_seed(32))
    by = lambda t, s: (t.float() * s[None, :, None, None]).bfloat16()  # noqa: E731
    if kind == "keys grow":
        step[:70] = 2.0 ** -20
        x["k"], x["h0"] = by(x["k"], step), None
    elif kind == "keys shrink":
        step[100:] = 2.0 ** -20
        x["k"] = by(x["k"], step)
        x["g"][0, 128] = -90
    elif kind == "keys start at zero":
        x["k"][0, :70] = 0
        x["k"][0, 140:210] = 0
    elif kind == "values grow":
        x["v"] = by(x["v"], 2.0 ** torch.linspace(-30, 30, T))
    elif kind == "values shrink":
        x["v"] = by(x["v"], 2.0 ** torch.linspace(30, -30, T))
        x["g"] = x["g"] * 20
    elif kind == "output gradients grow":
        do = do * 2.0 ** torch.linspace(-30, 30, T)[None, :, None, None]
        x["g"] = x["g"] * 20
    elif kind == "resets":
        x["g"][0, [0, 5, 40, 41, 64, 100, 149, 200]] = -float("inf")
    else:
        step[:200] = 2.0 ** -24
        x["v"], x["h0"] = by(x["v"], step), x["h0"] * 2.0 ** -24
    if kind == "resets":   # as the kernels count it: the factor is 0 in fp32 either way
        x["g"] = x["g"].clamp(min=-200.0)
    check(x, do.bfloat16())
    for a in (0, 64, 128, 192):   # and each chunk alone
        y = {n: (t[:, a:a + 64].contiguous() if n != "h0" and t is not None else None) for n, t in x.items()}
        check(y, do[:, a:a + 64].contiguous().bfloat16())


@pytest.mark.parametrize("hi", [1.0, 2.0])
def test_updates_up_to_two(hi):
    say(f"gdr_bwd, beta up to {hi}, keys that nearly repeat")
    x = ref.make(1, 150, 2, 4, h0=True, seed=5, lo=1e-3, hi=0.5)
    gen = torch.Generator().manual_seed(6)
    base = torch.randn(128, generator=gen)
    k = x["k"].float() * 0.3 + base / base.norm()
    x["k"] = (k / k.norm(dim=-1, keepdim=True) * (1 - 2.0 ** -7)).bfloat16()
    x["beta"] = hi * (0.5 + 0.5 * torch.rand(1, 150, 4, generator=gen))
    check(x)


def test_tokens_without_an_update():
    """beta of zero, of 2^-60 and of -2^-60: dv is exactly beta times what it multiplies, zero for a
    padded token, and nothing else sees an update that is not there."""
    say("gdr_bwd, beta of zero and near it")
    x = ref.make(1, 130, 1, 2, h0=True, seed=12)
    x["beta"][0, 20:70] = 0
    x["beta"][0, 100:110, 0], x["beta"][0, 100:110, 1] = 2.0 ** -60, -(2.0 ** -60)
    check(x)
