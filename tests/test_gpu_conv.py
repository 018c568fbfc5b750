"""GPU checks of the short causal convolution, its gradients and its single-token form against 64 bits."""
import pytest
import torch

from gated_delta_rule_35_amd import (KdaError, kda_conv, kda_conv_bwd, kda_conv_bwd_workspace_size, kda_conv_decode,
                                     load_library)
from tests import block_ref as ref
from tests.block_ref import TYPES

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    load_library()
    yield


def say(msg):
    print(f"[gpu] {msg}", flush=True)


def cuda(t):
    return None if t is None else t.cuda()


def make(B, T, C, W, kind, bias, state, N=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n = B if N is None else N
    t = TYPES[kind]
    return dict(x=rnd(B, T, C).to(t), w=rnd(C, W) / W ** 0.5, bias=0.3 * rnd(C) if bias else None,
                state=rnd(n, W - 1, C).to(t) if state else None, dy=rnd(B, T, C).to(t),
                dlast=rnd(n, W - 1, C).to(t) if state else None)


def check(c, act, cu=None, x=None, what=""):
    """Forward and gradients of a case; x: a view on the GPU that holds c["x"]."""
    d = {n: cuda(t) for n, t in c.items()}
    d["x"] = d["x"] if x is None else x
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = torch.full_like(d["dy"], 7.0)
    y, last = kda_conv(d["x"], d["w"], d["bias"], activation=act, cu_seqlens=cug, initial_state=d["state"], final_state=True,
                       out=out)
    grads = dict(dx=torch.full_like(d["dy"], 7.0))
    g = kda_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], activation=act, cu_seqlens=cug, initial_state=d["state"],
                     d_final_state=d["dlast"], d_initial_state=d["state"] is not None, grads=grads)
    torch.cuda.synchronize()
    want, mag, wl = ref.conv_batch(c["x"], c["w"], c["bias"], act, cu, c["state"])
    real = ~torch.isnan(want)
    ref.close(y.cpu()[real], want[real], 2.0 ** -20 * mag[real], what + " y")
    assert (y.cpu()[~real] == 7).all() and (g["dx"].cpu()[~real] == 7).all(), what + " rows in no sequence"
    assert torch.equal(last.cpu().double(), wl), what + " final state"
    wg, m = ref.conv_grads(c["x"], c["w"], c["dy"], c["bias"], act, cu, c["state"], c["dlast"])
    ref.close(g["dx"].cpu()[real], wg["dx"][real], 2.0 ** -20 * m["dx"][real], what + " dx")
    ref.close(g["dweight"], wg["dweight"], 2.0 ** -15 * m["dweight"], what + " dweight")
    if c["bias"] is None:
        assert g["dbias"] is None
    else:
        ref.close(g["dbias"], wg["dbias"], 2.0 ** -15 * m["dbias"], what + " dbias")
    if c["state"] is not None:
        ref.close(g["dstate"], wg["dstate"], 2.0 ** -20 * m["dstate"], what + " dstate")
    return y, last, g


CASES = [
    (1, 1, 8, 4, "bf16", "silu", False, False), (2, 2, 8, 4, "f32", None, True, True), (1, 3, 24, 3, "f16", "silu", True, True),
    (3, 5, 16, 2, "bf16", None, False, True), (2, 7, 520, 4, "bf16", "silu", True, False), (1, 64, 64, 4, "f32", "silu", False, True),
    (2, 100, 136, 3, "bf16", "silu", True, True), (1, 257, 1032, 4, "f16", "silu", False, True), (5, 33, 40, 2, "f32", "silu", True, True),
    (1, 1000, 8, 4, "bf16", "silu", True, True), (2, 515, 512, 4, "bf16", None, True, True),
]


@pytest.mark.parametrize("B,T,C,W,kind,act,bias,state", CASES)
def test_against_64_bits(B, T, C, W, kind, act, bias, state):
    say(f"conv B={B} T={T} C={C} W={W} {kind} {act} bias={bias} state={state}")
    check(make(B, T, C, W, kind, bias, state, seed=T), act, what=f"{B} {T} {C}")


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("cu", [[0, 1, 1, 3, 70, 70, 70, 75], [0, 0, 2, 40, 41, 42, 43, 44], [0, 75], [0, 3, 6, 9, 12, 15, 18, 21]])
def test_packed(cu, W):
    """Empty sequences, some shorter than the filter, rows in no sequence."""
    say(f"conv packed {cu} W={W}")
    check(make(1, 75, 72, W, "bf16", True, True, N=len(cu) - 1, seed=W), "silu", cu, what=f"{cu}")
    check(make(1, 75, 72, W, "f32", False, False, N=len(cu) - 1, seed=W), "silu", cu, what=f"{cu}")


def test_long_runs():
    """Enough tokens and channels for runs of 32 tokens, sequences that end inside them."""
    say("conv long runs")
    cu = [0, 1000, 1031, 1031, 5000, 8192]
    c = make(1, 8192, 4096, 4, "bf16", True, True, N=5, seed=3)
    d = {n: cuda(t) for n, t in c.items()}
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, last = kda_conv(d["x"], d["w"], d["bias"], cu_seqlens=cug, initial_state=d["state"], final_state=True)
    g = kda_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], cu_seqlens=cug, initial_state=d["state"], d_final_state=d["dlast"],
                     d_initial_state=True)
    torch.cuda.synchronize()
    some = slice(2000, 2064)   # channels mix with none, so that some of them are a case of their own
    part = {n: (None if t is None else t[some] if n in ("w", "bias") else t[..., some]) for n, t in c.items()}
    want, mag, wl = ref.conv_batch(part["x"], part["w"], part["bias"], "silu", cu, part["state"])
    ref.close(y.cpu()[..., some], want, 2.0 ** -20 * mag, "y")
    assert torch.equal(last.cpu()[..., some].double(), wl)
    wg, m = ref.conv_grads(part["x"], part["w"], part["dy"], part["bias"], "silu", cu, part["state"], part["dlast"])
    ref.close(g["dx"].cpu()[..., some], wg["dx"], 2.0 ** -20 * m["dx"], "dx")
    ref.close(g["dweight"][some], wg["dweight"], 2.0 ** -15 * m["dweight"], "dweight")
    ref.close(g["dbias"][some], wg["dbias"], 2.0 ** -15 * m["dbias"], "dbias")
    ref.close(g["dstate"].cpu()[..., some], wg["dstate"], 2.0 ** -20 * m["dstate"], "dstate")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_views(kind):
    """A slice of wider rows, rows in another order, and one row for the whole batch."""
    say(f"conv views {kind}")
    c = make(2, 50, 64, 4, kind, True, False, seed=9)
    wide = torch.full((2, 50, 200), NAN, dtype=TYPES[kind])
    wide[..., 72:136] = c["x"]
    base = check(c, "silu")[0]
    assert torch.equal(check(c, "silu", x=wide.cuda()[..., 72:136])[0], base)
    assert torch.equal(check(c, "silu", x=c["x"].transpose(0, 1).contiguous().cuda().transpose(0, 1))[0], base)
    c["x"] = c["x"][:1].expand(2, -1, -1)
    check(c, "silu", x=c["x"][:1].cuda().expand(2, -1, -1))


def test_nothing_reaches_other_sequences():
    """NaN and infinity in one sequence stay there, and behind the last sequence they are not seen."""
    say("conv NaN")
    c = make(1, 90, 16, 4, "bf16", False, True, N=3, seed=4)
    cu = [0, 30, 60, 80]
    args = lambda x, dy: (x.cuda(), c["w"].cuda(), dy.cuda())  # noqa: E731
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kw = dict(cu_seqlens=cug, initial_state=c["state"].cuda())
    x, dy = c["x"].clone(), c["dy"].clone()
    x[0, 30:60], x[0, 80:], dy[0, 80:], dy[0, 30:60] = NAN, NAN, NAN, float("inf")
    y0, last0 = kda_conv(args(c["x"], c["dy"])[0], c["w"].cuda(), final_state=True, **kw)
    y1, last1 = kda_conv(args(x, dy)[0], c["w"].cuda(), final_state=True, **kw)
    g0 = kda_conv_bwd(*args(c["x"], c["dy"]), d_initial_state=True, **kw)
    g1 = kda_conv_bwd(*args(x, dy), d_initial_state=True, **kw)
    for a, b in ((y0, y1), (g0["dx"], g1["dx"])):
        assert torch.equal(a[0, :30], b[0, :30]) and torch.equal(a[0, 60:80], b[0, 60:80])
    for a, b in ((last0, last1), (g0["dstate"], g1["dstate"])):
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    assert torch.isnan(y1[0, 30:60]).all()


def test_gradients_match_differences():
    say("conv differences")
    c = make(1, 6, 8, 3, "f32", True, True, seed=2)
    d = {n: cuda(t) for n, t in c.items()}
    g = kda_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], initial_state=d["state"], d_final_state=d["dlast"], d_initial_state=True)

    def loss(**kw):
        a = {**c, **kw}
        y, last, _ = ref.conv(ref.d64(a["x"])[0], ref.d64(a["w"]), ref.d64(a["bias"]), "silu", ref.d64(a["state"])[0])
        return float((y * ref.d64(c["dy"])[0]).sum() + (last * ref.d64(c["dlast"])[0]).sum())

    gen = torch.Generator().manual_seed(1)
    for name, key in (("x", "dx"), ("w", "dweight"), ("bias", "dbias"), ("state", "dstate")):
        v = torch.randn(c[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        diff = (loss(**{name: ref.d64(c[name]) + h * v}) - loss(**{name: ref.d64(c[name]) - h * v})) / (2 * h)
        along = float((ref.d64(g[key]) * v).sum())
        assert abs(along - diff) <= 1e-5 * float(ref.d64(g[key]).norm() * v.norm()), (name, along, diff)


def test_repeatable_and_two_streams():
    say("conv twice and side by side")
    c = {n: cuda(t) for n, t in make(2, 700, 264, 4, "bf16", True, True, seed=6).items()}
    run = lambda s=None: kda_conv_bwd(c["x"], c["w"], c["dy"], c["bias"], initial_state=c["state"],  # noqa: E731
                                      d_final_state=c["dlast"], d_initial_state=True, stream=s)
    a, b = run(), run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    more = [run(s) for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for r in (b, *more):
        for n in a:
            assert torch.equal(a[n], r[n]), n


def test_graph():
    say("conv in a graph")
    c = {n: cuda(t) for n, t in make(2, 300, 128, 4, "bf16", True, True, seed=8).items()}
    pool, idx = torch.randn(5, 3, 128, device="cuda").bfloat16(), torch.tensor([3, 0, -1], dtype=torch.int32, device="cuda")
    tok = torch.randn(3, 128, device="cuda").bfloat16()
    ws = torch.empty(kda_conv_bwd_workspace_size(600, 128, 4), dtype=torch.uint8, device="cuda")
    out, last = torch.empty_like(c["x"]), torch.empty_like(c["state"])
    grads = dict(dx=torch.empty_like(c["x"]), dweight=torch.empty_like(c["w"]), dbias=torch.empty_like(c["bias"]))
    dstate, one = torch.empty_like(c["state"]), torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")

    def step():
        kda_conv(c["x"], c["w"], c["bias"], initial_state=c["state"], out=out, final_state=last)
        kda_conv_bwd(c["x"], c["w"], c["dy"], c["bias"], initial_state=c["state"], d_final_state=c["dlast"], grads=grads,
                     d_initial_state=dstate, workspace=ws)
        kda_conv_decode(tok, c["w"], pool, c["bias"], state_indices=idx, out=one)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        gen = torch.Generator().manual_seed(i)
        c["x"].copy_(torch.randn(c["x"].shape, generator=gen))
        pool.copy_(torch.randn(pool.shape, generator=gen))
        start = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, last, *grads.values(), dstate, one, pool)]
        pool.copy_(start)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, last, *grads.values(), dstate, one, pool)):
            assert torch.equal(a, b)


def test_empty():
    say("conv of nothing")
    c = make(2, 0, 16, 4, "bf16", True, True)
    y, last, g = check(c, "silu")
    assert torch.equal(last.cpu(), c["state"]) and torch.equal(g["dstate"].cpu(), c["dlast"])
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
    none = torch.tensor([0], dtype=torch.int32, device="cuda")
    x = torch.ones(1, 5, 16, device="cuda")
    g = kda_conv_bwd(x, c["w"].cuda(), x, cu_seqlens=none)
    torch.cuda.synchronize()
    assert (g["dweight"] == 0).all()


@pytest.mark.parametrize("C,W,kind", [(8, 4, "bf16"), (1032, 3, "f32"), (2048, 2, "f16"), (1096, 4, "bf16")])
def test_decode(C, W, kind):
    """Slots outside the pool, one slot named by several rows, untouched slots; equal to the convolution of sequences."""
    say(f"conv_decode C={C} W={W} {kind}")
    t = TYPES[kind]
    c = make(1, 9, C, W, kind, True, False, seed=C)
    pool = torch.randn(7, W - 1, C, generator=torch.Generator().manual_seed(1)).to(t)
    idx = [4, -1, 2, 4, 7, 0, 4, 2, -5]
    x = c["x"][0].cuda()
    g = lambda p: torch.tensor(p, dtype=torch.int32, device="cuda")  # noqa: E731
    state, out = pool.cuda(), torch.full((9, C), 7.0, dtype=t, device="cuda")
    kda_conv_decode(x, c["w"].cuda(), state, c["bias"].cuda(), state_indices=g(idx), out=out)
    other = torch.full_like(state, 9.0)
    out2, _ = kda_conv_decode(x, c["w"].cuda(), pool.cuda(), c["bias"].cuda(), state_indices=g(idx), new_state=other)
    torch.cuda.synchronize()
    for slot in range(7):
        rows = [n for n, i in enumerate(idx) if i == slot]
        if not rows:
            assert torch.equal(state[slot].cpu(), pool[slot]) and (other[slot] == 9).all()
            continue
        y, last, mag = ref.conv(ref.d64(c["x"])[0, rows], ref.d64(c["w"]), ref.d64(c["bias"]), "silu", ref.d64(pool)[slot])
        ref.close(out[rows], y, 2.0 ** -20 * mag, f"slot {slot}")
        assert torch.equal(state[slot].cpu().double(), last) and torch.equal(other[slot], state[slot])
        assert torch.equal(out2[rows], out[rows])
    skipped = [n for n, i in enumerate(idx) if not 0 <= i < 7]
    assert (out[skipped] == 7).all()
    # without a slot map, from nothing, and of strided rows
    wide = torch.full((9, C + 24), NAN, dtype=t, device="cuda")
    wide[:, 8:8 + C] = x
    y, new = kda_conv_decode(wide[:, 8:8 + C], c["w"].cuda(), None, None, activation=None)
    torch.cuda.synchronize()
    want = ref.d64(c["x"])[0] * ref.d64(c["w"])[:, -1]
    ref.close(y, want, 2.0 ** -20 * want.abs(), "no state")
    assert (new[:, :-1] == 0).all() and torch.equal(new[:, -1], x)


def test_decode_continues_a_prompt():
    say("conv then conv_decode")
    c = make(2, 40, 64, 4, "bf16", True, False, seed=11)
    d = {n: cuda(t) for n, t in c.items()}
    whole, last = kda_conv(d["x"], d["w"], d["bias"], final_state=True)
    y, state = kda_conv(d["x"][:, :37], d["w"], d["bias"], final_state=True)
    for t in range(37, 40):
        one, state = kda_conv_decode(d["x"][:, t], d["w"], state, d["bias"])
        assert torch.equal(one, whole[:, t])
    assert torch.equal(state, last) and torch.equal(y, whole[:, :37])


def test_refused_on_the_device():
    x = torch.zeros(1, 4, 16, device="cuda")
    w = torch.zeros(16, 4, device="cuda")
    with pytest.raises(KdaError) as e:
        kda_conv(x, w, out=x)
    assert e.value.name == "KDA_ERR_LAYOUT"
    with pytest.raises(ValueError, match="on the GPU"):
        kda_conv(x, w.cpu())
    with pytest.raises(ValueError, match="activation"):
        kda_conv(x, w, activation="tanh")
