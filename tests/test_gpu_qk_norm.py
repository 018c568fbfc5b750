"""GPU checks of the per-head q/k norm and its gradients against 64 bits, and of the
norm, the gated delta rule and both backwards used together."""
import pytest
import torch

from gated_delta_rule_35_amd import KdaError, kda_fwd, kda_gdr_bwd, kda_gdr_fwd, kda_qk_norm, kda_qk_norm_bwd, load_library
from gated_delta_rule_35_amd import kda_qk_norm_bwd_workspace_size
from tests import gdr_ref as ref

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


def case(B, T, Hq, Hk, dtype=torch.bfloat16, weight=False, rot=0, positions=False, seed=0):
    gen = torch.Generator().manual_seed(seed)
    c = dict(q=torch.randn(B, T, Hq, 128, generator=gen).to(dtype), k=torch.randn(B, T, Hk, 128, generator=gen).to(dtype),
             wq=None, wk=None, cos=None, sin=None, pos=None)
    if weight:
        c["wq"], c["wk"] = (1 + 0.3 * torch.randn(128, generator=gen) for _ in range(2))
    if rot:
        P = T + 3
        ang = torch.arange(P).double()[:, None] * 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
        c["cos"], c["sin"] = ang.cos().float(), ang.sin().float()
        if positions:
            c["pos"] = torch.randint(-2, P + 2, (B, T), generator=gen, dtype=torch.int32)
    return c


def kwargs(c, mode, interleaved, dev="cuda"):
    m = lambda t: None if t is None else t.to(dev)  # noqa: E731
    return dict(q_weight=m(c["wq"]), k_weight=m(c["wk"]), mode=mode, cos=m(c["cos"]), sin=m(c["sin"]), positions=m(c["pos"]),
                interleaved=interleaved)


def ref_norm(c, x, w, mode, interleaved):
    d = lambda t: None if t is None else t.double()  # noqa: E731
    return ref.norm(x, w, mode, 1e-6, d(c["cos"]), d(c["sin"]), None if c["pos"] is None else c["pos"].long(), interleaved)


def assert_close(got, want, dtype, what):
    """One rounding to `dtype` of an fp32 result: a row's sum of 128 squares is off by at
    most 128 2^-24 of itself and the rest by a dozen roundings, 1e-5 of the row's largest
    entry in all."""
    got = got.detach().cpu().double()
    top = want.abs().amax(dim=-1, keepdim=True)
    step = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    # fp16 results below its normal range are rounded to a fixed step of 2^-24
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    off = ((got - want).abs() - step * want.abs() - 1e-5 * top - tiny).max()
    assert torch.isfinite(got).all() and off <= 0, (what, float(off))


CASES = [
    (1, 1, 1, 1, torch.bfloat16, "l2", False, 0, False, False),
    (2, 3, 2, 1, torch.bfloat16, "rms", True, 16, False, False),
    (1, 5, 3, 3, torch.float16, "l2", False, 32, True, True),
    (3, 17, 5, 2, torch.float32, "rms", True, 64, False, True),
    (1, 100, 16, 4, torch.bfloat16, "rms", True, 96, False, True),
    (2, 33, 8, 8, torch.bfloat16, "l2", True, 128, True, False),
    (1, 70, 4, 2, torch.float32, "l2", True, 128, False, True),
    (1, 257, 7, 1, torch.float16, "rms", True, 128, False, False),
]


@pytest.mark.parametrize("B,T,Hq,Hk,dtype,mode,weight,rot,interleaved,positions", CASES)
def test_norm_and_gradients(B, T, Hq, Hk, dtype, mode, weight, rot, interleaved, positions):
    say(f"qk_norm B={B} T={T} Hq={Hq} Hk={Hk} {dtype} {mode} weight={weight} rot={rot} interleaved={interleaved}")
    c = case(B, T, Hq, Hk, dtype, weight, rot, positions, seed=T)
    kw = kwargs(c, mode, interleaved)
    got = kda_qk_norm(c["q"].cuda(), c["k"].cuda(), **kw)
    for ddt in (torch.bfloat16, torch.float32):
        gen = torch.Generator().manual_seed(T + 1)
        dy = [torch.randn(c[n].shape, generator=gen).to(ddt) for n in "qk"]
        grads = kda_qk_norm_bwd(c["q"].cuda(), c["k"].cuda(), dy[0].cuda(), dy[1].cuda(), **kw)
        torch.cuda.synchronize()
        for i, n in enumerate("qk"):
            x = c[n].double().requires_grad_()
            w = None if c["w" + n] is None else c["w" + n].double().requires_grad_()
            y = ref_norm(c, x, w, mode, interleaved)
            assert got[i].dtype == torch.bfloat16 and got[i].is_contiguous()
            assert_close(got[i], y.detach(), torch.bfloat16, "out " + n)
            want = torch.autograd.grad(y, [x] + ([w] if w is not None else []), dy[i].double())
            assert grads["d" + n].dtype == dtype
            assert_close(grads["d" + n], want[0], dtype, "d" + n)
            dw = grads[f"d{n}_weight"]
            if w is None:
                assert dw is None
            else:   # fp32 sums of B T H terms of order one
                terms = B * T * (Hq if n == "q" else Hk)
                assert (dw.cpu().double() - want[1]).abs().max() <= 1e-5 * max(1.0, terms ** 0.5) * 4


def test_many_rows_share_work_groups():
    """More rows than work-groups of the weight gradients take at once, ragged at the end."""
    say("qk_norm_bwd 3 x 1001 x (9, 2) heads")
    c = case(3, 1001, 9, 2, weight=True, rot=64, seed=5)
    gen = torch.Generator().manual_seed(8)
    dy = [torch.randn(c[n].shape, generator=gen).bfloat16() for n in "qk"]
    kw = kwargs(c, "rms", False)
    runs = [kda_qk_norm_bwd(c["q"].cuda(), c["k"].cuda(), dy[0].cuda(), dy[1].cuda(), **kw) for _ in range(2)]
    torch.cuda.synchronize()
    for n in runs[0]:
        assert torch.equal(runs[0][n], runs[1][n]), n
    for i, n in enumerate("qk"):
        x, w = c[n].double().requires_grad_(), c["w" + n].double().requires_grad_()
        want = torch.autograd.grad(ref_norm(c, x, w, "rms", False), [x, w], dy[i].double())
        assert_close(runs[0]["d" + n], want[0], torch.bfloat16, "d" + n)
        rel = (runs[0][f"d{n}_weight"].cpu().double() - want[1]).norm() / want[1].norm()
        assert rel <= 1e-5, (n, float(rel))


def test_views_in_place_zero_rows_and_other_rows():
    say("qk_norm on views, in place, with rows of zeros")
    c = case(2, 40, 4, 2, weight=True, rot=64, seed=6)
    c["q"][0, 3] = 0
    kw = kwargs(c, "l2", False)
    want = kda_qk_norm(c["q"].cuda(), c["k"].cuda(), **kw)
    assert torch.equal(want[0][0, 3], torch.zeros_like(want[0][0, 3]))
    wide = torch.full((2, 40, 8 * 128), NAN, dtype=torch.bfloat16, device="cuda")
    q, k = wide[..., :512].view(2, 40, 4, 128), wide[..., 512:768].view(2, 40, 2, 128)
    q.copy_(c["q"])
    k.copy_(c["k"])
    got = kda_qk_norm(q, k, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isnan(wide[..., 768:]).all()
    a, b = c["q"].cuda(), c["k"].cuda()
    got = kda_qk_norm(a, b, out=(a, b), **kw)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and got[0] is a
    dy = [torch.randn_like(want[0]), torch.randn_like(want[1])]
    g1 = kda_qk_norm_bwd(q, k, *dy, **kw)
    g2 = kda_qk_norm_bwd(c["q"].cuda(), c["k"].cuda(), *dy, **kw)
    assert all(torch.equal(g1[n], g2[n]) for n in g1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g3 = kda_qk_norm_bwd(q, k, *dy, stream=s, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(g1[n], g3[n]) for n in g1)


def test_graph():
    say("qk_norm and its backward in one graph")
    c = case(1, 50, 4, 2, weight=True, rot=128, seed=7)
    kw = kwargs(c, "rms", True)
    q, k = c["q"].cuda(), c["k"].cuda()
    dy = [torch.randn_like(q), torch.randn_like(k)]
    ws = torch.empty(kda_qk_norm_bwd_workspace_size(), dtype=torch.uint8, device="cuda")

    def both():
        y = kda_qk_norm(q, k, **kw)
        g = kda_qk_norm_bwd(q, k, *dy, workspace=ws, **kw)
        return list(y) + [g[n] for n in sorted(g)]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for _ in range(4):
        want = [t.clone() for t in both()]
        torch.cuda.synchronize()
        for t in held:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_two_streams_at_once():
    """Calls with weight gradients on two streams, each with its own scratch, and repeats:
    the same bits."""
    say("norm and its gradients on two streams")
    c = {n: (t.cuda() if t is not None else None) for n, t in case(2, 500, 4, 2, weight=True, rot=64, seed=21).items()}
    kw = kwargs(c, "rms", False)
    dq, dk = torch.randn_like(c["q"]), torch.randn_like(c["k"])
    want = kda_qk_norm_bwd(c["q"], c["k"], dq, dk, **kw)
    y = kda_qk_norm(c["q"], c["k"], **kw)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append((kda_qk_norm_bwd(c["q"], c["k"], dq, dk, **kw), kda_qk_norm(c["q"], c["k"], **kw)))
    torch.cuda.synchronize()
    for g, z in got:
        assert all(torch.equal(g[n], want[n]) for n in want) and all(torch.equal(a, b) for a, b in zip(z, y))


def test_far_offsets():
    """As many rows as a tensor may have, 2^26 of 2^33 elements: the last tokens get the bits
    that they get alone."""
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of free device memory")
    T, last = 1 << 20, 40
    say(f"norm and its gradients, T={T}, 64 + 1 heads")
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.randn(1, T, h, 128, generator=gen, device="cuda", dtype=torch.bfloat16) for h in (64, 1))
    q1, k1 = q[:, T - last:].contiguous(), k[:, T - last:].contiguous()
    a, b = kda_qk_norm(q, k), kda_qk_norm(q1, k1)
    assert all(torch.equal(x[:, T - last:], y) for x, y in zip(a, b))
    del a
    dq = torch.randn(1, T, 64, 128, generator=gen, device="cuda", dtype=torch.bfloat16)
    a = kda_qk_norm_bwd(q, k, dq, k)
    b = kda_qk_norm_bwd(q1, k1, dq[:, T - last:].contiguous(), k1)
    assert all(torch.equal(a[n][:, T - last:], b[n]) for n in ("dq", "dk"))
    more = [torch.empty(1, T + 1, h, 128, device="cuda", dtype=torch.bfloat16) for h in (64, 1)]
    with pytest.raises(KdaError, match="UNSUPPORTED"):   # more rows than a tensor may have
        kda_qk_norm(*more)
    del a, q, dq, more
    torch.cuda.empty_cache()


def test_norm_feeds_the_per_channel_rule():
    """kda_fwd on normalised q and k: rows of unit length as its contract wants."""
    say("qk_norm into kda_fwd")
    c = case(1, 100, 2, 2, seed=11)
    q, k = kda_qk_norm(c["q"].cuda(), c["k"].cuda(), eps=1e-12)
    # each entry is off by half a bf16 step at most, so a row's norm is off by 2^-8
    assert ((q.float().norm(dim=-1) - 1).abs() <= 2.0 ** -8).all()
    v = torch.randn(1, 100, 2, 128, device="cuda").bfloat16()
    g = torch.full((1, 100, 2, 128), -0.1, device="cuda")
    beta = torch.full((1, 100, 2), 0.5, device="cuda")
    o, _ = kda_fwd(q, k, v, g, beta, 128 ** -0.5)
    o2, _ = kda_gdr_fwd(q, k, v, g[..., 0].contiguous(), beta, 128 ** -0.5)
    torch.cuda.synchronize()
    # the per-channel rule with equal channels is the per-head rule: its fp16 operands
    # (2^-11 each, a handful of them) and both bf16 roundings apart
    assert (o.float() - o2.float()).norm() / o.float().norm() <= 2 * 2.0 ** -8


@pytest.mark.parametrize("mode,rot", [("l2", 0), ("rms", 64)])
def test_layer_forward_and_backward(mode, rot):
    """Norm, delta rule, and both backwards as a training step runs them, against autograd
    of the whole in 64 bits.  The intermediates q, k, dq, dk are bf16, so the results are
    held to the spread of those roundings: each of the few products sums terms that are
    off by 2^-8 at most and of random sign; 2^-6 of the head's norm holds four of them
    adding up in full."""
    say(f"norm + gdr, forward and backward, {mode} rot={rot}")
    c = case(1, 150, 2, 2, weight=mode == "rms", rot=rot, seed=12)
    x = ref.make(1, 150, 2, 4, h0=True, seed=13)
    scale = 128 ** -0.5 if mode == "l2" else 1.0 / 128
    if mode == "rms":   # rows of length sqrt(128) would blow the rule up: weights bring them to about one
        c["wk"] = c["wk"] * 128 ** -0.5
    kw = kwargs(c, mode, False)
    d = ref.cuda(x)
    qn, kn = kda_qk_norm(c["q"].cuda(), c["k"].cuda(), **kw)
    o, hT = kda_gdr_fwd(qn, kn, d["v"], d["g"], d["beta"], scale, initial_state=d["h0"], final_state=True)
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(14)).bfloat16()
    gr = kda_gdr_bwd(qn, kn, d["v"], d["g"], d["beta"], scale, do.cuda(), initial_state=d["h0"], d_initial_state=True)
    gn = kda_qk_norm_bwd(c["q"].cuda(), c["k"].cuda(), gr["dq"], gr["dk"], **kw)
    torch.cuda.synchronize()
    leaf = {n: c[n].double().requires_grad_() for n in ("q", "k")}
    leaf.update({n: x[n].double().requires_grad_() for n in ("v", "g", "beta", "h0")})
    w = {n: (None if c["w" + n] is None else c["w" + n].double().requires_grad_()) for n in "qk"}
    y = [ref_norm(c, leaf[n], w[n], mode, False) for n in "qk"]
    o_ref, _ = ref.recurrence(y[0][0], y[1][0], leaf["v"][0], leaf["g"][0], leaf["beta"][0], scale, leaf["h0"][0])
    names = ["q", "k", "v", "g", "beta", "h0"]
    ws = [w[n] for n in "qk" if w[n] is not None]
    want = torch.autograd.grad(o_ref, [leaf[n] for n in names] + ws, do[0].double())
    got = [gn["dq"], gn["dk"], gr["dv"], gr["dg"], gr["dbeta"], gr["dh0"]]
    if ws:
        got += [gn["dq_weight"], gn["dk_weight"]]
    assert ref.rel(o[0], o_ref) <= 2.0 ** -6
    for n, a, b in zip(names + ["dq_weight", "dk_weight"], got, want):
        assert ref.rel(a, b) <= 2.0 ** -6, n
