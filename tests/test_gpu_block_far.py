"""GPU checks of the block operators behind element 2^31 of their tensors: the same numbers as near the start."""
import pytest
import torch

from gated_delta_rule_35_amd import (kda_add_norm, kda_add_norm_bwd, kda_conv, kda_conv_bwd, kda_conv_decode, kda_gated_norm,
                                     kda_gated_norm_bwd, kda_ssm_bwd, kda_ssm_decode, kda_ssm_fwd, load_library)

pytestmark = pytest.mark.gpu
FAR = 1 << 31


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    load_library()
    yield
    torch.cuda.empty_cache()


def say(msg):
    print(f"[gpu] {msg}", flush=True)


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


def far(t, step):
    """The rows of t [1, T, ...] as a view whose rows lie `step` elements apart, the last behind element 2^31."""
    T = t.shape[1]
    assert (T - 1) * step > FAR
    big = torch.empty((T - 1) * step + t[0, 0].numel(), dtype=t.dtype, device="cuda")
    v = big.as_strided(t.shape, (0, step) + t.stride()[2:])
    v.copy_(t)
    return v


def same(a, b):
    torch.cuda.synchronize()
    a, b = (list(v.values()) if isinstance(v, dict) else v if isinstance(v, (tuple, list)) else [v] for v in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None and y is None) or torch.equal(x, y)


def test_conv():
    say("convolution, rows 2^23 apart")
    x, w, b, dy = rnd(1, 300, 520).bfloat16(), rnd(520, 4, seed=1), rnd(520, seed=2), rnd(1, 300, 520, seed=3).bfloat16()
    v = far(x, 1 << 23)
    same(kda_conv(v, w, b, final_state=True), kda_conv(x, w, b, final_state=True))
    same(kda_conv_bwd(v, w, dy, b), kda_conv_bwd(x, w, dy, b))


def test_norms():
    say("norms, rows 2^23 apart")
    x, z, dy, w = (rnd(1, 300, 2, 256, seed=i).bfloat16() for i in (0, 1, 2, 3))
    w = w[0, 0, 0].float().contiguous()
    v = far(x, 1 << 23)
    same(kda_gated_norm(v, z, w), kda_gated_norm(x, z, w))
    same(kda_gated_norm_bwd(v, z, dy, w), kda_gated_norm_bwd(x, z, dy, w))
    h, d, w = x.flatten(2), dy.flatten(2), rnd(512, seed=4)
    v = far(h, 1 << 23)
    same(kda_add_norm(v, z.flatten(2), w), kda_add_norm(h, z.flatten(2), w))
    same(kda_add_norm_bwd(v, d, w, d_sum=d), kda_add_norm_bwd(h, d, w, d_sum=d))


def test_many_rows():
    """Contiguous tensors of more than 2^31 elements: their last rows."""
    say("gated norm of 2^31 + 2^20 elements")
    n, D = FAR // 1024 + 1024, 1024
    x = torch.empty(1, n, 1, D, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    w = rnd(D, seed=2)
    y = kda_gated_norm(x, x, w)
    same(y[:, -300:], kda_gated_norm(x[:, -300:], x[:, -300:], w))
    g = kda_gated_norm_bwd(x, x, y)
    e = kda_gated_norm_bwd(x[:, -300:], x[:, -300:], y[:, -300:].contiguous())
    same([g["dx"][:, -300:], g["dgate"][:, -300:]], [e["dx"], e["dgate"]])


def test_scan_views():
    say("scan, rows 2^23 apart")
    T, H, P, S = 300, 2, 64, 128
    x, B, C = rnd(1, T, H, P).bfloat16(), rnd(1, T, 1, S, seed=1).bfloat16(), rnd(1, T, 1, S, seed=2).bfloat16()
    dt, A, dy = rnd(1, T, H, seed=3), -1 - rnd(H, seed=4).abs(), rnd(1, T, H, P, seed=5).bfloat16()
    one = dict(D=rnd(H, seed=6), dt_bias=rnd(H, seed=7) - 4)
    want = kda_ssm_fwd(x, dt, A, B, C, final_state=True, **one), kda_ssm_bwd(x, dt, A, B, C, dy, **one)
    for i in range(3):
        ins = [x, B, C]
        ins[i] = far(ins[i], 1 << 23)
        same(kda_ssm_fwd(ins[0], dt, A, ins[1], ins[2], final_state=True, **one), want[0])
        same(kda_ssm_bwd(ins[0], dt, A, ins[1], ins[2], dy, **one), want[1])
        del ins


def test_scan_states_and_rows():
    """17 rows whose kept states take 2^31 elements and more: the last row against itself alone.  Its sums are taken
    in other segments, so bf16 results may round apart where they lie between two values (one step, 2^-8, in a few of
    a thousand: 2^-11 in norm), fp32 ones by the operands' 2^-16."""
    say("scan gradients with kept states behind 2^31")
    N, T, H, P, S = 17, 16384, 64, 64, 128
    gen = torch.Generator("cuda").manual_seed(9)
    new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda").normal_(generator=gen)  # noqa: E731
    x, B, C, dt = new(N, T, H, P), new(N, T, 1, S), new(N, T, 1, S), new(N, T, H, dtype=torch.float32)
    A, bias = -1 - rnd(H, seed=4).abs(), rnd(H, seed=7) - 4
    y, hT = kda_ssm_fwd(x, dt, A, B, C, dt_bias=bias, final_state=True)
    g = kda_ssm_bwd(x, dt, A, B, C, y, dt_bias=bias)
    one = [t[-1:] for t in (x, dt, B, C, y)]
    y1, h1 = kda_ssm_fwd(one[0], one[1], A, one[2], one[3], dt_bias=bias, final_state=True)
    g1 = kda_ssm_bwd(one[0], one[1], A, one[2], one[3], one[4], dt_bias=bias)
    torch.cuda.synchronize()
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
    assert rel(y[-1:], y1) <= 2.0 ** -10 and rel(hT[-1:], h1) <= 2.0 ** -15
    for n, tol in (("dx", 2.0 ** -10), ("dB", 2.0 ** -10), ("dC", 2.0 ** -10), ("ddt", 2.0 ** -13)):
        assert rel(g[n][-1:], g1[n]) <= tol, (n, rel(g[n][-1:], g1[n]))


def test_pools():
    say("decode from pools of more than 2^31 elements")
    H, P, S, N = 64, 64, 128, 3
    slots = FAR // (H * P * S) + 2
    x, dt, A = rnd(N, H, P).bfloat16(), rnd(N, H, seed=1), -1 - rnd(H, seed=2).abs()
    B, C, first = rnd(N, 1, S, seed=3).bfloat16(), rnd(N, 1, S, seed=4).bfloat16(), rnd(N, H, S, P, seed=5)
    at = torch.tensor([slots - 1, 0, slots - 2], dtype=torch.int32, device="cuda")
    pool = torch.empty(slots, H, S, P, device="cuda")
    pool[at.long()] = first
    small = first.clone()
    want, _ = kda_ssm_decode(x, dt, A, B, C, small)
    got, _ = kda_ssm_decode(x, dt, A, B, C, pool, state_indices=at)
    same([got, pool[at.long()]], [want, small])
    del pool
    Ch = 12288
    slots = FAR // (3 * Ch) + 2
    x, w, first = rnd(N, Ch).bfloat16(), rnd(Ch, 4, seed=1), rnd(N, 3, Ch, seed=2).bfloat16()
    at = torch.tensor([slots - 1, 0, slots - 2], dtype=torch.int32, device="cuda")
    pool = torch.empty(slots, 3, Ch, dtype=torch.bfloat16, device="cuda")
    pool[at.long()] = first
    small = first.clone()
    want, _ = kda_conv_decode(x, w, small)
    got, _ = kda_conv_decode(x, w, pool, state_indices=at)
    same([got, pool[at.long()]], [want, small])
