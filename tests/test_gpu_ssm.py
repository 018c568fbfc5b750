"""GPU checks of the selective state space scan, its gradients and its single-token form against 64 bits."""
import pytest
import torch

from gated_delta_rule_35_amd import (KdaError, kda_ssm_bwd, kda_ssm_bwd_workspace_size, kda_ssm_decode, kda_ssm_fwd,
                                     kda_ssm_fwd_workspace_size, load_library)
from tests import ssm_ref as ref

pytestmark = pytest.mark.gpu
NAN = float("nan")
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    load_library()
    yield


def say(msg):
    print(f"[gpu] {msg}", flush=True)


def ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def fwd(d, cu=None, **kw):
    return kda_ssm_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], dt_bias=d["bias"], softplus=d["softplus"],
                       cu_seqlens=ints(cu), initial_state=d["h0"], final_state=kw.pop("final_state", True), **kw)


def bwd(d, cu=None, **kw):
    return kda_ssm_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], D=d["D"], dt_bias=d["bias"], softplus=d["softplus"],
                       cu_seqlens=ints(cu), initial_state=d["h0"], d_final_state=d["dlast"],
                       d_initial_state=kw.pop("d_initial_state", True), **kw)


def check_forward(c, cu=None, d=None):
    d = ref.cuda(c) if d is None else d
    out = torch.full(c["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    y, hT = fwd(d, cu, out=out)
    torch.cuda.synchronize()
    want, mag, S, Sm = ref.run(c, cu)
    ref.close(y, want, ref.BITS["y"] * mag, "y")
    ref.close(hT, S, ref.BITS["state"] * Sm, "final state")
    assert (y.cpu()[torch.isnan(want)] == 7).all(), "rows in no sequence"
    return y, hT


def check_gradients(c, cu=None, d=None):
    d = ref.cuda(c) if d is None else d
    grads = dict(dx=torch.full(c["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda"),
                 ddt=torch.full(c["dt"].shape, 7.0, device="cuda"))
    g = bwd(d, cu, grads=grads)
    torch.cuda.synchronize()
    want, mag = ref.gradients(c, cu)
    for n in GRADS:
        if g[n] is None:
            assert (n == "dD" and c["D"] is None) or (n == "ddt_bias" and c["bias"] is None)
            continue
        ref.close(g[n], want[n], ref.BITS[n] * mag[n], n)
    for n in ("dx", "ddt"):
        assert (g[n].cpu()[torch.isnan(want[n])] == 7).all(), "rows in no sequence"
    return g


SHAPES = [
    # B, T, H, P, S, G
    (1, 1, 1, 64, 128, 1), (2, 3, 2, 64, 64, 1), (1, 63, 3, 64, 128, 1), (1, 64, 2, 128, 64, 2), (2, 65, 4, 64, 128, 2),
    (1, 130, 5, 64, 64, 5), (1, 200, 3, 128, 128, 1), (3, 17, 8, 64, 128, 1), (1, 100, 6, 64, 128, 2), (1, 129, 4, 128, 128, 4),
]


@pytest.mark.parametrize("B,T,H,P,S,G", SHAPES)
@pytest.mark.parametrize("h0,dt,softplus", [(False, "bf16", True), (True, "f32", True), (True, "f32", False)])
def test_forward(B, T, H, P, S, G, h0, dt, softplus):
    say(f"ssm_fwd B={B} T={T} H={H} P={P} S={S} G={G} h0={h0} dt={dt} softplus={softplus}")
    check_forward(ref.make(B, T, H, P, S, G, dt=dt, h0=h0, D=h0, bias=softplus or h0, softplus=softplus, seed=T))


@pytest.mark.parametrize("B,T,H,P,S,G", SHAPES)
@pytest.mark.parametrize("h0,dt,softplus", [(False, "bf16", True), (True, "f32", True), (True, "f32", False)])
def test_gradients(B, T, H, P, S, G, h0, dt, softplus):
    say(f"ssm_bwd B={B} T={T} H={H} P={P} S={S} G={G} h0={h0} dt={dt} softplus={softplus}")
    check_gradients(ref.make(B, T, H, P, S, G, dt=dt, h0=h0, D=h0, bias=softplus or not h0, softplus=softplus, seed=T + 1))


PACKS = [[0, 1, 1, 3, 70, 134, 134, 200], [0, 0, 64, 128, 150, 150, 150, 200], [0, 200], [0, 5, 5, 180, 180]]


@pytest.mark.parametrize("P,S", [(64, 128), (128, 64)])
@pytest.mark.parametrize("cu", PACKS)
def test_packed(cu, P, S):
    """Empty sequences, single tokens, chunks that end at every place, rows in no sequence."""
    say(f"ssm packed {cu} P={P} S={S}")
    c = ref.make(1, 200, 2, P, S, 1, N=len(cu) - 1, h0=True, seed=cu[1])
    check_forward(c, cu)
    check_gradients(c, cu)


@pytest.mark.parametrize("P,S", [(64, 128), (128, 64)])
def test_many_sequences(P, S):
    """More walks than half the compute units: work-groups of 256 columns, of which 320 (or 640) leave the last one part."""
    say(f"ssm 130 sequences P={P} S={S}")
    cu = [0]
    for n in [100, 130] + [1 + i % 3 for i in range(128)]:
        cu.append(cu[-1] + n)
    c = ref.make(1, cu[-1], 5, P, S, 1, N=130, h0=True, seed=P)
    check_forward(c, cu)
    check_gradients(c, cu)


@pytest.mark.parametrize("cu", [None, [0, 700, 701, 1100], [0, 64, 1024, 1024, 1088]])
def test_segments(cu):
    """Long sequences on few heads: segments side by side, chained; their states from outside and to outside."""
    say(f"ssm segments {cu}")
    n = 1 if cu is None else len(cu) - 1
    c = ref.make(1, 1100, 2, 64, 64, 1, N=n, h0=True, seed=3, fast=2.0)
    c["bias"] = c["bias"] - 2   # slow decays, so that states of far segments count
    y, hT = check_forward(c, cu)
    check_gradients(c, cu)
    d = ref.cuda(c)
    state = d["h0"].clone()   # the final state in the place of the initial one
    d["h0"] = state
    y2, h2 = fwd(d, cu, final_state=state)
    torch.cuda.synchronize()
    if cu is None:
        assert torch.equal(y, y2)
    assert torch.equal(hT, h2) and h2.data_ptr() == state.data_ptr()


@pytest.mark.parametrize("fast,spread", [(300.0, 3.0), (1.0, 0.1), (5000.0, 2.0)])
def test_decays_from_none_to_all(fast, spread):
    """Heads that forget within a token beside ones that keep nearly everything; every gradient against its
    own terms."""
    say(f"ssm decays to {fast}")
    c = ref.make(1, 150, 4, 64, 64, 1, h0=True, seed=11, fast=fast, spread=spread)
    c["A"][0] = -1e-6
    check_forward(c)
    check_gradients(c)


def test_sizes_far_from_one():
    say("ssm sizes")
    c = ref.make(1, 140, 3, 64, 64, 1, h0=True, seed=12)
    c["x"] = (c["x"].float() * torch.tensor([1e-10, 1.0, 1e10])[:, None]).bfloat16()
    c["B"] = (c["B"].float() * 2.0 ** torch.linspace(-20, 20, 64)).bfloat16()
    c["h0"] = c["h0"] * torch.tensor([1e-8, 1.0, 1e12])[:, None, None]
    c["dy"] = (c["dy"].float() * torch.tensor([1e5, 1.0, 1e-9])[:, None]).bfloat16()
    check_forward(c)
    check_gradients(c)


def test_steps_of_zero_change_nothing():
    say("ssm zero steps")
    c = ref.make(1, 100, 2, 64, 64, 1, h0=True, softplus=False, bias=False, seed=13)
    c["dt"][0, 20:40] = 0
    c["dt"][0, :, 1] = 0
    y, hT = check_forward(c)
    assert torch.equal(hT[0, 1].cpu(), c["h0"][0, 1])
    check_gradients(c)


def test_views():
    """Slices of one row a token, as the convolution leaves them, and other orders."""
    say("ssm views")
    c = ref.make(2, 90, 4, 64, 128, 2, dt="bf16", h0=True, seed=14)
    base, gb = check_forward(c), check_gradients(c)
    d = ref.cuda(c)
    row = torch.full((2, 90, 256 + 512 + 64), NAN, dtype=torch.bfloat16, device="cuda")
    row[..., :256], row[..., 256:512], row[..., 512:768] = (d[n].flatten(2) for n in ("x", "B", "C"))
    wide = torch.full((2, 90, 11), NAN, dtype=torch.bfloat16, device="cuda")
    wide[..., 3:7] = d["dt"]
    v = dict(d, x=row[..., :256].unflatten(-1, (4, 64)), B=row[..., 256:512].unflatten(-1, (2, 128)),
             C=row[..., 512:768].unflatten(-1, (2, 128)), dt=wide[..., 3:7], dy=d["dy"].transpose(0, 1).contiguous().transpose(0, 1))
    y, hT = fwd(v)
    g = bwd(v)
    torch.cuda.synchronize()
    assert torch.equal(y, base[0]) and torch.equal(hT, base[1])
    for n in GRADS:
        assert torch.equal(g[n], gb[n]), n
    # one step and one row of B for all heads and tokens of a batch row
    c["dt"] = c["dt"][:, :1].expand(-1, 90, -1)
    d = ref.cuda(c)
    d["dt"] = d["dt"][:, :1].contiguous().expand(-1, 90, -1)
    check_forward(c, d=d)


def test_nothing_reaches_other_sequences_or_heads():
    say("ssm NaN")
    c = ref.make(1, 300, 2, 64, 64, 1, N=3, h0=True, seed=15)
    cu = [0, 100, 201, 280]
    base, gb = fwd(ref.cuda(c), cu), bwd(ref.cuda(c), cu)
    e = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in c.items()}
    for n in ("x", "dt", "B", "C", "dy"):
        e[n][0, 280:] = NAN        # behind the last sequence
        e[n][0, 100:201] = NAN     # the middle one
    got, gg = fwd(ref.cuda(e), cu), bwd(ref.cuda(e), cu)
    torch.cuda.synchronize()
    keep = list(range(100)) + list(range(201, 280))
    assert torch.equal(base[0][0, keep], got[0][0, keep]) and torch.isnan(got[0][0, 100:201].float()).all()
    assert torch.equal(base[1][[0, 2]], got[1][[0, 2]])
    for n in ("dx", "ddt", "dB", "dC"):
        assert torch.equal(gb[n][0, keep], gg[n][0, keep]), n
    assert torch.equal(gb["dh0"][[0, 2]], gg["dh0"][[0, 2]])
    e = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in c.items()}
    e["x"][0, 50, 0], e["dy"][0, 60, 0] = NAN, float("inf")
    got, gg = fwd(ref.cuda(e), cu), bwd(ref.cuda(e), cu)
    torch.cuda.synchronize()
    assert torch.equal(base[0][0, :280, 1], got[0][0, :280, 1]) and torch.equal(gb["dx"][0, :280, 1], gg["dx"][0, :280, 1])
    assert torch.equal(gb["ddt"][0, :280, 1], gg["ddt"][0, :280, 1])


def test_gradients_match_differences():
    say("ssm differences")
    c = ref.make(1, 70, 2, 64, 64, 1, h0=True, seed=16)
    g = bwd(ref.cuda(c))
    torch.cuda.synchronize()

    def loss(a):
        d = {n: ref.d64(t) if isinstance(t, torch.Tensor) else t for n, t in a.items()}
        y, S = ref.scan(d["x"][0], d["dt"][0], d["A"], d["B"][0], d["C"][0], d["D"], d["bias"], True, d["h0"][0])
        return float((y * d["dy"][0]).sum() + (S * d["dlast"][0]).sum())

    gen = torch.Generator().manual_seed(1)
    for name, key in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("bias", "ddt_bias"), ("h0", "dh0")):
        v = torch.randn(c[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-6
        up, down = dict(c), dict(c)
        up[name], down[name] = ref.d64(c[name]) + h * v, ref.d64(c[name]) - h * v
        diff = (loss(up) - loss(down)) / (2 * h)
        along = float((ref.d64(g[key]) * v).sum())
        # bf16 gradients are off by 2^-8 of each entry at most, independently: far below 1e-3 of the product of norms
        tol = 1e-3 if key in ("dx", "dB", "dC") else 1e-5
        assert abs(along - diff) <= tol * float(ref.d64(g[key]).norm() * v.norm()), (name, along, diff)


def test_repeatable_and_two_streams():
    say("ssm twice and side by side")
    d = ref.cuda(ref.make(2, 500, 4, 64, 128, 1, h0=True, seed=17))
    torch.cuda.synchronize()
    run = lambda s=None: [*fwd(d, stream=s), *(bwd(d, stream=s)[n] for n in GRADS)]  # noqa: E731
    a = run()
    torch.cuda.synchronize()
    more = [run()] + [run(s) for s in (torch.cuda.Stream(), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for r in more:
        assert all(torch.equal(x, y) for x, y in zip(a, r))


def test_graph():
    say("ssm in a graph")
    d = ref.cuda(ref.make(1, 600, 2, 64, 64, 1, h0=True, seed=18))
    one = ref.cuda(ref.make(3, 1, 2, 64, 64, 1, seed=19))
    pool = torch.randn(5, 2, 64, 64, device="cuda")
    idx = ints([3, -1, 0])
    out = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    sizes = (600, 1, 2, 1, 64, 64)
    w1 = torch.empty(kda_ssm_fwd_workspace_size(*sizes), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(kda_ssm_bwd_workspace_size(*sizes), dtype=torch.uint8, device="cuda")

    def step(ws=True):
        y, hT = fwd(d, workspace=w1 if ws else None)
        g = bwd(d, workspace=w2 if ws else None)
        kda_ssm_decode(one["x"][:, 0], one["dt"][:, 0], one["A"], one["B"][:, 0], one["C"][:, 0], pool, D=one["D"],
                       dt_bias=one["bias"], state_indices=idx, out=out)
        return [y, hT, *(g[n] for n in GRADS)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = step()
    for i in range(3):
        gen = torch.Generator().manual_seed(i)
        d["x"].copy_(torch.randn(d["x"].shape, generator=gen))
        d["dt"].copy_(torch.randn(d["dt"].shape, generator=gen))
        pool.copy_(torch.randn(pool.shape, generator=gen))
        start = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*inside, out, pool)]
        pool.copy_(start)
        eager = step(False)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (*eager, out, pool)))


def test_empty():
    say("ssm of nothing")
    for B, T in ((0, 5), (2, 0)):
        c = ref.make(B, T, 2, 64, 64, 1, h0=True)
        d = ref.cuda(c)
        y, hT = fwd(d)
        g = bwd(d)
        torch.cuda.synchronize()
        assert torch.equal(hT.cpu(), c["h0"]) and torch.equal(g["dh0"].cpu(), c["dlast"])
        assert all((g[n] == 0).all() for n in ("dA", "dD", "ddt_bias"))
    c = ref.make(1, 10, 2, 64, 64, 1, N=0)
    g = bwd(dict(ref.cuda(c), dlast=None), [0], d_initial_state=False)
    torch.cuda.synchronize()
    assert all((g[n] == 0).all() for n in ("dA", "dD", "ddt_bias"))
    c = ref.make(1, 0, 2, 64, 64, 1, N=2, h0=True)
    y, hT = fwd(ref.cuda(c), [0, 0, 0])
    g = bwd(ref.cuda(c), [0, 0, 0])
    torch.cuda.synchronize()
    assert torch.equal(hT.cpu(), c["h0"]) and torch.equal(g["dh0"].cpu(), c["dlast"])


@pytest.mark.parametrize("H,P,S,G,rows", [(2, 64, 128, 1, 9), (6, 128, 64, 3, 9), (64, 64, 64, 8, 9), (3, 128, 128, 1, 200)])
def test_decode(H, P, S, G, rows):
    """Slots outside the pool, one slot named by several rows, untouched slots; as many tokens of a sequence."""
    say(f"ssm_decode H={H} P={P} S={S} G={G} rows={rows}")
    c = ref.make(1, rows, H, P, S, G, dt="bf16", seed=H)
    slots = 7
    pool = torch.randn(slots, H, S, P, generator=torch.Generator().manual_seed(1))
    idx = ([4, -1, 2, 4, 7, 0, 4, 2, -5] * (rows // 9 + 1))[:rows]
    d = ref.cuda(c)
    args = (d["x"][0], d["dt"][0], d["A"], d["B"][0], d["C"][0])
    state, out = pool.cuda(), torch.full((rows, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    kda_ssm_decode(*args, state, D=d["D"], dt_bias=d["bias"], state_indices=ints(idx), out=out)
    other = torch.full_like(state, 9.0)
    out2, _ = kda_ssm_decode(*args, pool.cuda(), D=d["D"], dt_bias=d["bias"], state_indices=ints(idx), new_state=other)
    torch.cuda.synchronize()
    for slot in range(slots):
        at = [n for n, i in enumerate(idx) if i == slot]
        if not at:
            assert torch.equal(state[slot].cpu(), pool[slot]) and (other[slot] == 9).all()
            continue
        part = {n: (t[:, at] if n in ref.TOKEN else t) for n, t in c.items()}
        part.update(h0=pool[slot][None], dy=None, dlast=None)
        y, ym, S1, Sm = ref.run(part)
        ref.close(out[at], y[0], ref.BITS["y"] * ym[0], f"slot {slot}")
        ref.close(state[slot], S1[0], ref.BITS["state"] * Sm[0], f"state {slot}")
        assert torch.equal(other[slot], state[slot]) and torch.equal(out2[at], out[at])
    assert (out[[n for n, i in enumerate(idx) if not 0 <= i < slots]] == 7).all()
    y, new = kda_ssm_decode(*args, None)
    torch.cuda.synchronize()
    part = dict(c, D=None, bias=None, h0=None)
    part = {n: (t.transpose(0, 1) if n in ref.TOKEN else t) for n, t in part.items()}
    want, mag, S1, Sm = ref.run(part)
    ref.close(y, want[:, 0], ref.BITS["y"] * mag[:, 0], "from nothing")
    ref.close(new, S1, ref.BITS["state"] * Sm, "states from nothing")


def test_decode_continues_a_prompt():
    say("ssm_fwd then ssm_decode")
    c = ref.make(2, 40, 4, 64, 128, 1, h0=True, seed=20)
    d = ref.cuda(c)
    want, mag, S, Sm = ref.run(c)
    short = {n: (t[:, :37].contiguous() if n in ref.TOKEN else t) for n, t in d.items()}
    y, state = fwd(short)
    ys = [y]
    for t in range(37, 40):
        one, state = kda_ssm_decode(d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], state, D=d["D"], dt_bias=d["bias"])
        ys.append(one[:, None])
    torch.cuda.synchronize()
    ref.close(torch.cat(ys, dim=1), want, ref.BITS["y"] * mag, "y")
    ref.close(state, S, ref.BITS["state"] * Sm, "state")


def test_refused():
    c = ref.cuda(ref.make(1, 8, 2, 64, 64, 1, h0=True))
    with pytest.raises(KdaError) as e:
        fwd(c, out=c["x"])
    assert e.value.name == "KDA_ERR_LAYOUT"
    with pytest.raises(ValueError, match="on the GPU"):
        kda_ssm_fwd(c["x"], c["dt"].cpu(), c["A"], c["B"], c["C"])
