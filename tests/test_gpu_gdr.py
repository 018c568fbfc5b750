"""GPU checks of the gated delta rule with one decay per head (kda_gdr_fwd,
kda_gdr_bwd, kda_gdr_decode) against the 64-bit token recurrence.  Each test prints
its case before it touches the GPU."""
import pytest
import torch

from gated_delta_rule_35_amd import KdaError, kda_gdr_bwd, kda_gdr_decode, kda_gdr_fwd, load_library
from gated_delta_rule_35_amd import kda_gdr_bwd_workspace_size, kda_gdr_fwd_workspace_size
from tests import gdr_ref as ref

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    load_library()
    yield


def say(msg):
    print(f"[gpu] {msg}", flush=True)


def args(d):
    return d["q"], d["k"], d["v"], d["g"], d["beta"], SCALE


def check_forward(x, cu=None):
    d = ref.cuda(x)
    cu_d = cu.cuda() if cu is not None else None
    N = x["q"].shape[0] if cu is None else len(cu) - 1
    out = torch.full(x["v"].shape, NAN, dtype=torch.bfloat16, device="cuda")
    hT = torch.full((N, x["v"].shape[2], 128, 128), NAN, device="cuda")
    kda_gdr_fwd(*args(d), cu_seqlens=cu_d, initial_state=d["h0"], out=out, final_state=hT)
    torch.cuda.synchronize()
    o_ref, h_ref = ref.forward(x, SCALE, cu)
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(o_ref))   # rows in no sequence stay as they were
    ref.assert_rows(out, o_ref, "o", half=ref.forward_magnitude(x, SCALE, cu))
    ref.assert_states(hT, h_ref, "final state")
    return out, hT


def check_backward(x, cu=None, with_state=True, seed=0):
    gen = torch.Generator().manual_seed(seed + 77)
    d = ref.cuda(x)
    cu_d = cu.cuda() if cu is not None else None
    N = x["q"].shape[0] if cu is None else len(cu) - 1
    Hv = x["v"].shape[2]
    do = torch.randn(x["v"].shape, generator=gen).bfloat16()
    dhT = 0.1 * torch.randn(N, Hv, 128, 128, generator=gen) if with_state else None
    names = (("dq", "q"), ("dk", "k"), ("dv", "v"))
    grads = {n: torch.full(x[m].shape, NAN, dtype=torch.bfloat16, device="cuda") for n, m in names}
    grads.update({n: torch.full(x["g"].shape, NAN, device="cuda") for n in ("dg", "dbeta")})
    got = kda_gdr_bwd(*args(d), do.cuda(), initial_state=d["h0"], d_final_state=dhT.cuda() if with_state else None,
                      grads=grads, d_initial_state=with_state, cu_seqlens=cu_d)
    torch.cuda.synchronize()
    want = ref.gradients(x, SCALE, do, dhT, cu)
    for n, m in names:
        assert torch.equal(torch.isnan(got[n].cpu()), torch.isnan(want[m]))
        ref.assert_rows(got[n], want[m], n)
    for n, m in (("dg", "g"), ("dbeta", "beta")):
        assert torch.equal(torch.isnan(got[n].cpu()), torch.isnan(want[m]))
        ref.assert_gates(got[n], want[m], n)
    if with_state:
        ref.assert_states(got["dh0"], want["h0"], "dh0")
    return got


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 200])
def test_forward_lengths(T):
    say(f"gdr_fwd B=2 T={T} Hq=1 Hv=2")
    check_forward(ref.make(2, T, 1, 2, h0=T % 2 == 1, seed=T))


@pytest.mark.parametrize("Hq,Hv,beta", [(1, 1, torch.bfloat16), (3, 3, torch.float32), (2, 8, torch.bfloat16),
                                        (5, 10, torch.float32), (8, 8, torch.float32)])
def test_forward_heads(Hq, Hv, beta):
    say(f"gdr_fwd B=1 T=130 Hq={Hq} Hv={Hv} beta={beta}")
    check_forward(ref.make(1, 130, Hq, Hv, beta, h0=True, seed=Hq + Hv))


PACKED = [[65, 0, 1, 130], [1], [0, 0, 3], [64, 64], [63, 2, 127, 1, 1]]


@pytest.mark.parametrize("lens", PACKED)
@pytest.mark.parametrize("tail", [0, 5])
def test_forward_packed(lens, tail):
    say(f"gdr_fwd packed {lens} + {tail} rows in no sequence")
    x = ref.make(1, sum(lens) + tail, 2, 4, h0=True, N=len(lens), seed=sum(lens))
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    check_forward(x, cu)


@pytest.mark.parametrize("packed", [False, True])
def test_forward_more_heads_than_compute_units(packed):
    """Batches whose (sequence, value head) pairs alone fill the GPU, packed ones four times: a
    work-group then walks both halves of a head."""
    lens = [0, 1, 200, 64, 65, 3, 130, 128] * 8 if packed else None
    say(f"gdr_fwd {'packed' if packed else 'B=20'}, Hv=16")
    x = ref.make(1, sum(lens) + 9, 4, 16, h0=True, N=64, seed=51) if packed else ref.make(20, 150, 4, 16, h0=True, seed=52)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32) if packed else None
    pairs = 64 * 16 // 4 if packed else 20 * 16
    assert pairs >= torch.cuda.get_device_properties(0).multi_processor_count
    check_forward(x, cu)
    if not packed:   # the same rows a few at a time, where a work-group walks half a head
        d = ref.cuda(x)
        o, h = kda_gdr_fwd(*args(d), initial_state=d["h0"], final_state=True)
        o1, h1 = kda_gdr_fwd(*(t[3:6] for t in args(d)[:5]), SCALE, initial_state=d["h0"][3:6].contiguous(),
                             final_state=True)
        assert torch.equal(o[3:6], o1) and torch.equal(h[3:6], h1)


@pytest.mark.parametrize("T", [1, 3, 16, 17, 63, 64, 65, 129, 200])
def test_backward_lengths(T):
    say(f"gdr_bwd B=2 T={T} Hq=1 Hv=2")
    check_backward(ref.make(2, T, 1, 2, h0=T % 2 == 1, seed=100 + T), with_state=T % 4 == 1, seed=T)


@pytest.mark.parametrize("Hq,Hv,beta", [(1, 1, torch.bfloat16), (2, 8, torch.bfloat16), (3, 6, torch.float32)])
def test_backward_heads(Hq, Hv, beta):
    say(f"gdr_bwd B=1 T=130 Hq={Hq} Hv={Hv} beta={beta}")
    check_backward(ref.make(1, 130, Hq, Hv, beta, h0=True, seed=Hq + Hv))


@pytest.mark.parametrize("lens", PACKED)
@pytest.mark.parametrize("tail", [0, 5])
def test_backward_packed(lens, tail):
    say(f"gdr_bwd packed {lens} + {tail} rows in no sequence")
    x = ref.make(1, sum(lens) + tail, 2, 4, h0=True, N=len(lens), seed=sum(lens))
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    check_backward(x, cu)


@pytest.mark.parametrize("kind", ["keeps", "forgets", "resets", "no update", "wide values", "small values", "long keys",
                                  "tiny keys", "tiny queries", "growing keys"])
def test_gates_and_ranges(kind):
    """Log-decays of zero, strong ones, minus infinity between tokens, beta of zero, and
    values far from one."""
    say(f"gdr fwd and bwd, {kind}")
    x = ref.make(1, 150, 1, 2, h0=True, seed=9)
    if kind == "keeps":
        x["g"].zero_()
    elif kind == "forgets":
        x["g"] = x["g"] * 150
    elif kind == "resets":
        x["g"][0, [0, 5, 40, 41, 64, 100, 149]] = -float("inf")
    elif kind == "no update":
        x["beta"][0, 10:90] = 0
    elif kind == "wide values":
        x["v"] = (x["v"].float() * 3e6).bfloat16()
    elif kind == "small values":
        x["v"], x["h0"] = (x["v"].float() * 1e-9).bfloat16(), x["h0"] * 1e-9
    elif kind == "long keys":
        x["k"] = (x["k"].float() * 1.2).bfloat16()
    elif kind == "tiny keys":
        x["k"], x["h0"] = (x["k"].float() * 1e-7).bfloat16(), x["h0"] * 1e-7
    elif kind == "tiny queries":
        x["q"] = (x["q"].float() * 1e-20).bfloat16()
    else:   # each token's key longer than the one before, 2^-8 to 1
        x["k"] = (x["k"].float() * 2.0 ** torch.linspace(-8, 0, 150)[None, :, None, None]).bfloat16()
    check_forward(x)
    check_backward(x, with_state=kind != "wide values")


@pytest.mark.parametrize("kind", ["keys grow", "keys shrink", "keys start at zero", "no update of a small state",
                                  "values grow", "small state, large values later"])
def test_sizes_that_change_between_chunks(kind):
    """Keys, values and states whose sizes change by many powers of two from one chunk to the
    next, in both directions."""
    say(f"gdr fwd and bwd, {kind}")
    x = ref.make(1, 270, 1, 2, h0=True, seed=31)
    step = torch.ones(270)
    if kind == "keys grow":
        step[:70] = 2.0 ** -20
        x["k"], x["h0"] = (x["k"].float() * step[None, :, None, None]).bfloat16(), None
    elif kind == "keys shrink":   # and the state built from the large ones is forgotten
        step[100:] = 2.0 ** -20
        x["k"] = (x["k"].float() * step[None, :, None, None]).bfloat16()
        x["g"][0, 128] = -90
    elif kind == "keys start at zero":
        x["k"][0, :70] = 0
        x["k"][0, 140:210] = 0
    elif kind == "no update of a small state":
        x["beta"][0, :130] = 0
        x["h0"] = x["h0"] * 2.0 ** -24
        x["g"] = x["g"] * 0.01
    elif kind == "values grow":
        step = 2.0 ** torch.linspace(-30, 30, 270)
        x["v"] = (x["v"].float() * step[None, :, None, None]).bfloat16()
    else:
        step[:200] = 2.0 ** -24
        x["v"], x["h0"] = (x["v"].float() * step[None, :, None, None]).bfloat16(), x["h0"] * 2.0 ** -24
    check_forward(x)
    for a, b in ((0, 64), (64, 128), (128, 192)):   # chunk by chunk, each against its own size
        if x["h0"] is None or a:
            check_forward({n: (t[:, a:b].contiguous() if n != "h0" else None) for n, t in x.items()})
    out, _ = check_forward(x)
    want, _ = ref.forward(x, SCALE)
    half = ref.forward_magnitude(x, SCALE)
    for a in range(0, 270, 64):
        ref.assert_rows(out[:, a:a + 64], want[:, a:a + 64], (kind, a), half=half[:, a:a + 64])
    check_backward(x, with_state=x["h0"] is not None)


def test_far_scales():
    """A scale and queries whose product lies below fp32's normal numbers, on large values."""
    say("gdr_fwd, scale 2^-40, queries 2^-100, values 2^60")
    x = ref.make(1, 100, 1, 1, seed=33)
    x["q"], x["v"] = (x["q"].double() * 2.0 ** -100).bfloat16(), (x["v"].double() * 2.0 ** 60).bfloat16()
    d = ref.cuda(x)
    o, _ = kda_gdr_fwd(*args(d)[:5], 2.0 ** -40)
    torch.cuda.synchronize()
    ref.assert_rows(o, ref.forward(x, 2.0 ** -40)[0], "o", half=ref.forward_magnitude(x, 2.0 ** -40))


@pytest.mark.parametrize("many", [False, True])
def test_packed_heads_of_eight_and_many_sequences(many):
    """Value heads in a multiple of eight (each XCD an eighth of them), and more sequences than
    a work-group has threads."""
    lens = [1, 2, 0, 3] * 150 if many else [70, 3, 0, 129, 64]
    Hq, Hv = (1, 1) if many else (2, 8)
    say(f"gdr fwd and bwd, {len(lens)} sequences, Hv={Hv}")
    x = ref.make(1, sum(lens), Hq, Hv, h0=True, N=len(lens), seed=35)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    check_forward(x, cu)
    check_backward(x, cu)


def test_value_channels_are_independent():
    """Value channels of sizes from 2^-60 to 2^60, changing from token to token block: every
    channel keeps the accuracy that it has alone (all products are linear in it)."""
    say("gdr_fwd with channels of all sizes")
    x = ref.make(1, 333, 1, 2, h0=True, seed=23)
    size = 2.0 ** torch.linspace(-60, 60, 128).round()[torch.randperm(128, generator=torch.Generator().manual_seed(5))]
    y = dict(x, v=(x["v"].float() * size).bfloat16(), h0=x["h0"] * size)
    d, e = ref.cuda(x), ref.cuda(y)
    o, h = kda_gdr_fwd(*args(d), initial_state=d["h0"], final_state=True)
    o2, h2 = kda_gdr_fwd(*args(e), initial_state=e["h0"], final_state=True)
    torch.cuda.synchronize()
    o_ref, h_ref = ref.forward(x, SCALE)
    ref.assert_rows(o2.cpu().double() / size.double(), o_ref, "o", half=ref.forward_magnitude(x, SCALE))
    ref.assert_states(h2.cpu().double() / size.double(), h_ref, "state")
    # blocks of tokens that are large, then small, then large again
    steps = 2.0 ** torch.tensor([0, 30, -30, 12, -20, 0]).repeat_interleave(64)[:333].double()
    z = dict(x, v=(x["v"].double() * steps[None, :, None, None]).bfloat16(), g=x["g"] * 20)
    check_forward(z)
    for c in range(0, 333, 64):   # block by block, each against its own size
        w = {n: (t[:, c:c + 64].contiguous() if n != "h0" else None) for n, t in z.items()}
        check_forward(w)


def test_correlated_keys():
    """Keys that nearly repeat: the in-chunk system is far from the identity."""
    say("gdr fwd and bwd, keys near one direction")
    x = ref.make(1, 192, 1, 1, seed=4, lo=0.001, hi=0.02)
    base = torch.randn(128, generator=torch.Generator().manual_seed(1))
    k = x["k"].float() * 0.5 + base / base.norm()
    x["k"] = (k / k.norm(dim=-1, keepdim=True)).bfloat16()
    check_forward(x)
    check_backward(x, with_state=False)


def test_strided_inputs_match_contiguous_ones():
    """q, k, v and do as slices of wider rows, and as heads-first storage."""
    say("gdr fwd, bwd and decode on views")
    x = ref.cuda(ref.make(2, 100, 2, 4, h0=True, seed=21))
    B, T = 2, 100
    do = torch.randn(B, T, 4, 128, device="cuda").bfloat16()
    wide = torch.full((B, T, (2 + 2 + 4) * 128 + 64), NAN, dtype=torch.bfloat16, device="cuda")
    y = dict(x, q=wide[..., :256].view(B, T, 2, 128), k=wide[..., 256:512].view(B, T, 2, 128),
             v=wide[..., 512:1024].view(B, T, 4, 128))
    for n in "qkv":
        y[n].copy_(x[n])
    z = dict(x, **{n: x[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "qkv"})
    do_z = do.transpose(1, 2).contiguous().transpose(1, 2)
    want = kda_gdr_fwd(*args(x), initial_state=x["h0"], final_state=True)
    gwant = kda_gdr_bwd(*args(x), do, initial_state=x["h0"])
    for v, dov in ((y, do), (z, do_z)):
        got = kda_gdr_fwd(*args(v), initial_state=x["h0"], final_state=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        g = kda_gdr_bwd(*args(v), dov, initial_state=x["h0"])
        assert all(torch.equal(g[n], gwant[n]) for n in ("dq", "dk", "dv", "dg", "dbeta"))
    one = {n: x[n][:, 3].contiguous() for n in ("q", "k", "v", "g", "beta")}
    view = dict(one, q=y["q"][:, 3], k=y["k"][:, 3], v=y["v"][:, 3])
    a, sa = kda_gdr_decode(*args(one), x["h0"].clone())
    b, sb = kda_gdr_decode(*args(view), x["h0"].clone())
    assert torch.equal(a, b) and torch.equal(sa, sb)


def test_broadcast_heads_and_batches():
    """q, k and v that are one head or one row of the batch, seen as many (strides of 0)."""
    say("gdr fwd and bwd on expanded views")
    x = ref.cuda(ref.make(1, 90, 1, 1, h0=False, seed=41))
    g, beta = -torch.rand(2, 90, 4, device="cuda"), torch.rand(2, 90, 4, device="cuda")
    q, k = (x[n].expand(2, 90, 2, 128) for n in "qk")
    v = x["v"].expand(2, 90, 4, 128)
    do = torch.randn(1, 90, 1, 128, device="cuda").bfloat16().expand(2, 90, 4, 128)
    a = kda_gdr_fwd(q, k, v, g, beta, SCALE, final_state=True)
    b = kda_gdr_fwd(*(t.contiguous() for t in (q, k, v)), g, beta, SCALE, final_state=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = kda_gdr_bwd(q, k, v, g, beta, SCALE, do)
    b = kda_gdr_bwd(*(t.contiguous() for t in (q, k, v)), g, beta, SCALE, do.contiguous())
    assert all(torch.equal(a[n], b[n]) for n in ("dq", "dk", "dv", "dg", "dbeta"))


def test_nothing_to_do():
    """No tokens, no sequences, only empty sequences, no rows: states pass through, nothing
    else is written."""
    say("gdr fwd, bwd and decode without tokens or sequences")
    h0 = torch.randn(2, 4, 128, 128, device="cuda")
    e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    x = (e(2, 0, 2, 128), e(2, 0, 2, 128), e(2, 0, 4, 128), e(2, 0, 4, t=torch.float32), e(2, 0, 4, t=torch.float32), SCALE)
    o, hT = kda_gdr_fwd(*x, initial_state=h0, final_state=True)
    assert o.shape == (2, 0, 4, 128) and torch.equal(hT, h0)
    assert torch.equal(kda_gdr_fwd(*x, final_state=True)[1], torch.zeros_like(h0))
    assert torch.equal(kda_gdr_bwd(*x, x[2], d_final_state=h0, d_initial_state=True)["dh0"], h0)
    for cu in ([0], [0, 0, 0]):   # no sequence; two empty ones
        y = ref.cuda(ref.make(1, 70, 2, 4, seed=43))
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        n = len(cu) - 1
        out, do = torch.full_like(y["v"], NAN), torch.zeros_like(y["v"])
        _, hT = kda_gdr_fwd(*args(y), cu_seqlens=cu, initial_state=h0[:n], out=out, final_state=True)
        assert torch.isnan(out).all() and torch.equal(hT, h0[:n])
        grads = {m: torch.full_like(y[s], NAN) for m, s in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"),
                                                            ("dbeta", "beta"))}
        got = kda_gdr_bwd(*args(y), do, d_final_state=h0[:n], d_initial_state=True, grads=grads, cu_seqlens=cu)
        assert all(torch.isnan(got[m]).all() for m in grads) and torch.equal(got["dh0"], h0[:n])
    o, s = kda_gdr_decode(e(0, 2, 128), e(0, 2, 128), e(0, 4, 128), e(0, 4, t=torch.float32), e(0, 4, t=torch.float32),
                          SCALE, h0.clone(), state_indices=e(0, t=torch.int32))
    assert o.shape == (0, 4, 128) and torch.equal(s, h0)


def test_rows_in_no_sequence_are_not_read():
    """NaN in every input of rows behind the last sequence reaches nothing."""
    say("gdr fwd and bwd, NaN behind the last sequence")
    x = ref.make(1, 150, 1, 2, h0=True, N=2, seed=45)
    cu = torch.tensor([0, 70, 141], dtype=torch.int32)
    for n in ("q", "k", "v", "g", "beta"):
        x[n][0, 141:] = NAN
    d = ref.cuda(x)
    out, hT = kda_gdr_fwd(*args(d), cu_seqlens=cu.cuda(), initial_state=d["h0"], out=torch.full_like(d["v"], 7.0),
                          final_state=True)
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(3)).bfloat16()
    do[0, 141:] = NAN
    got = kda_gdr_bwd(*args(d), do.cuda(), initial_state=d["h0"], d_initial_state=True, cu_seqlens=cu.cuda())
    torch.cuda.synchronize()
    assert (out[0, 141:] == 7).all() and torch.isfinite(hT).all()
    want, _ = ref.forward(x, SCALE, cu)
    ref.assert_rows(out[:, :141], want[:, :141], "o", half=ref.forward_magnitude(x, SCALE, cu)[:, :141])
    grads = ref.gradients(x, SCALE, do, None, cu)
    for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        ref.assert_rows(got[n][:, :141], grads[m][:, :141], n)
    assert torch.isfinite(got["dh0"]).all()


def test_repeats_aliases_and_streams():
    """Runs are bitwise equal: again, with the final state over the initial one, with a
    caller's workspace, on another stream; two workspaces on two streams at once."""
    say("gdr_fwd repeats")
    x = ref.cuda(ref.make(2, 333, 2, 4, h0=True, seed=31))
    o, h = kda_gdr_fwd(*args(x), initial_state=x["h0"], final_state=True)
    h2 = x["h0"].clone()
    o2, _ = kda_gdr_fwd(*args(x), initial_state=h2, final_state=h2)
    ws = torch.empty(kda_gdr_fwd_workspace_size(666, 2, 4), dtype=torch.uint8, device="cuda")
    o3, h3 = kda_gdr_fwd(*args(x), initial_state=x["h0"], final_state=True, workspace=ws)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        o4, h4 = kda_gdr_fwd(*args(x), initial_state=x["h0"], final_state=True)
    o5, h5 = kda_gdr_fwd(*args(x), initial_state=x["h0"], final_state=True, stream=s2)
    torch.cuda.synchronize()
    for a, b in ((o2, h2), (o3, h3), (o4, h4), (o5, h5)):
        assert torch.equal(o, a) and torch.equal(h, b)
    do = torch.randn_like(x["v"])
    g1 = kda_gdr_bwd(*args(x), do, initial_state=x["h0"], d_initial_state=True)
    g2 = kda_gdr_bwd(*args(x), do, initial_state=x["h0"], d_initial_state=True, stream=s1)
    torch.cuda.synchronize()
    assert all(torch.equal(g1[n], g2[n]) for n in g1)


def test_library_allocates_without_workspace():
    """The C entry points with a NULL workspace (allocated in stream order)."""
    import ctypes

    from gated_delta_rule_35_amd import binding
    say("C kda_gdr_fwd with a NULL workspace")
    x = ref.cuda(ref.make(1, 100, 1, 2, seed=32))
    want, _ = kda_gdr_fwd(*args(x))
    out = torch.empty_like(want)
    ds = [binding.describe(t) for t in (x["q"], x["k"], x["v"], x["g"], x["beta"], out)]
    r = [ctypes.addressof(t) for t in ds]
    lib = load_library()
    st = lib.kda_gdr_fwd(*r[:5], SCALE, None, None, r[5], None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def replay_and_compare(graph, eager, outs):
    """Replays with eager work between them, every replay against the eager result."""
    for _ in range(4):
        want = [t.clone() for t in eager()]
        torch.cuda.synchronize()
        for t in outs:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_graphs():
    """Forward and backward captured side by side, each with its own workspace."""
    say("gdr graphs")
    x = ref.cuda(ref.make(1, 300, 2, 4, h0=True, seed=41))
    do = torch.randn_like(x["v"])
    ws = torch.empty(kda_gdr_fwd_workspace_size(300, 1, 4), dtype=torch.uint8, device="cuda")
    wb = torch.empty(kda_gdr_bwd_workspace_size(300, 1, 4), dtype=torch.uint8, device="cuda")
    out, hT = torch.empty_like(x["v"]), torch.empty_like(x["h0"])

    def fwd(out, hT, ws):
        kda_gdr_fwd(*args(x), initial_state=x["h0"], out=out, final_state=hT, workspace=ws)
        return out, hT

    def bwd(grads, ws):
        r = kda_gdr_bwd(*args(x), do, initial_state=x["h0"], grads=grads, workspace=ws)
        return [r[n] for n in ("dq", "dk", "dv", "dg", "dbeta")]

    fwd(out, hT, ws)
    held = bwd(None, wb)
    grads = dict(zip(("dq", "dk", "dv", "dg", "dbeta"), held))
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        fwd(out, hT, ws)
    with torch.cuda.graph(g2):
        bwd(grads, wb)
    replay_and_compare(g1, lambda: fwd(torch.empty_like(out), torch.empty_like(hT), None), [out, hT])
    replay_and_compare(g2, lambda: bwd(None, None), held)


def test_gradients_against_differences():
    """The gradients along a random direction against central differences of the 64-bit
    recurrence.  The step h = 1e-4 leaves a difference error of order h^2 = 1e-8; the
    gradient's own error is the bf16 rounding of dq, dk, dv, whose signs are random over
    thousands of entries, so 2^-8 of the sum of the parts' magnitudes is never reached."""
    say("gdr_bwd against differences")
    x = ref.make(1, 70, 1, 2, h0=True, seed=51)
    gen = torch.Generator().manual_seed(3)
    do = torch.randn(x["v"].shape, generator=gen).bfloat16()
    d = ref.cuda(x)
    got = kda_gdr_bwd(*args(d), do.cuda(), initial_state=d["h0"], d_initial_state=True)
    torch.cuda.synchronize()
    x64 = {n: t.double() for n, t in x.items()}
    for n, m in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("h0", "dh0")):
        w = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-4

        def loss(sign):
            y = dict(x64)
            y[n] = y[n] + sign * h * w
            return float((ref.forward(y, SCALE)[0] * do.double()).sum())

        want = (loss(1) - loss(-1)) / (2 * h)
        parts = got[m].cpu().double() * w
        assert abs(float(parts.sum()) - want) <= 2.0 ** -8 * float(parts.abs().sum()) / 4 + 1e-6, (n, want)


# ------------------------------------------------------------------ decode


def decode_ref(x, t, S, slots):
    """One 64-bit step of every row on the pool S, rows in order; returns o (NaN: skipped)."""
    d = {n: x[n][:, t].double() for n in ("q", "k", "v", "g", "beta")}
    o = torch.full(d["v"].shape, NAN, dtype=torch.float64)
    for n, s in enumerate(slots):
        if 0 <= s < S.shape[0]:
            on, S[s] = ref.recurrence(*(d[m][n:n + 1] for m in ("q", "k", "v", "g", "beta")), SCALE, S[s])
            o[n] = on[0]
    return o


@pytest.mark.parametrize("N,Hq,Hv,beta", [(1, 1, 1, torch.float32), (3, 2, 8, torch.bfloat16), (7, 4, 4, torch.float32),
                                          (40, 16, 64, torch.bfloat16)])
@pytest.mark.parametrize("mapped", [False, True])
def test_decode(N, Hq, Hv, beta, mapped):
    say(f"gdr_decode N={N} Hq={Hq} Hv={Hv} mapped={mapped}")
    steps = 3
    x = ref.make(N, steps, Hq, Hv, beta, h0=False, seed=N + Hv)
    gen = torch.Generator().manual_seed(N)
    P = N + 5 if mapped else N
    slots = torch.randperm(P, generator=gen)[:N] if mapped else torch.arange(N)
    if mapped:
        slots[N // 2] = -1 if N % 2 else P
    pool = 0.1 * torch.randn(P, Hv, 128, 128, generator=gen)
    got, S = pool.cuda(), pool.double()
    named = [int(s) for s in slots if 0 <= s < P]
    idx = slots.to(torch.int32).cuda() if mapped else None
    for t in range(steps):
        one = {n: x[n][:, t].contiguous().cuda() for n in ("q", "k", "v", "g", "beta")}
        out = torch.full((N, Hv, 128), NAN, dtype=torch.bfloat16, device="cuda")
        o, new = kda_gdr_decode(*args(one), got, state_indices=idx, out=out)
        torch.cuda.synchronize()
        assert new is got
        want = decode_ref(x, t, S, slots.tolist())
        assert torch.equal(torch.isnan(o.cpu()), torch.isnan(want))
        ref.assert_rows(o, want, "o", dim=1)
    ref.assert_states(got[named], S[named], "pool")
    others = [s for s in range(P) if s not in named]
    assert torch.equal(got[others].cpu(), pool[others])


def test_decode_same_slot_twice():
    """Rows that name one slot are tokens of one sequence in order, for both widths of
    the kernel's column slices."""
    for N, Hv in ((9, 2), (70, 32)):
        say(f"gdr_decode with repeated slots N={N} Hv={Hv}")
        x = ref.make(N, 1, 1, Hv, seed=N)
        slots = [(n * n) % 5 for n in range(N)]
        pool = 0.1 * torch.randn(6, Hv, 128, 128, generator=torch.Generator().manual_seed(2))
        S, got = pool.double(), pool.cuda()
        one = {n: x[n][:, 0].contiguous().cuda() for n in ("q", "k", "v", "g", "beta")}
        o, _ = kda_gdr_decode(*args(one), got, state_indices=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        ref.assert_rows(o, decode_ref(x, 0, S, slots), "o", dim=1)
        ref.assert_states(got, S, "pool")


def test_decode_states_none_separate_and_reset():
    say("gdr_decode from zero, into another buffer, after a reset")
    x = ref.cuda(ref.make(3, 1, 2, 4, h0=True, seed=61))
    one = {n: x[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")}
    a, sa = kda_gdr_decode(*args(one), None)
    b, sb = kda_gdr_decode(*args(one), torch.zeros_like(x["h0"]))
    assert torch.equal(a, b) and torch.equal(sa, sb)
    kept = x["h0"].clone()
    c, sc = kda_gdr_decode(*args(one), x["h0"], new_state=torch.full_like(kept, NAN))
    d, sd = kda_gdr_decode(*args(one), kept.clone())
    assert torch.equal(x["h0"], kept) and torch.equal(c, d) and torch.equal(sc, sd)
    one["g"] = torch.full_like(one["g"], -float("inf"))
    e, se = kda_gdr_decode(*args(one), kept.clone())
    assert torch.equal(e, a) and torch.equal(se, sa)


def test_decode_graph():
    say("gdr_decode graph")
    x = ref.cuda(ref.make(5, 1, 2, 4, seed=71))
    one = {n: x[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")}
    idx = torch.tensor([3, -1, 0, 6, 1], dtype=torch.int32, device="cuda")
    pool = torch.randn(7, 4, 128, 128, device="cuda")
    out, new = torch.zeros(5, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(pool)
    kda_gdr_decode(*args(one), pool, state_indices=idx, out=out, new_state=new)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda_gdr_decode(*args(one), pool, state_indices=idx, out=out, new_state=new)

    def eager():
        o, s = torch.full_like(out, 7), torch.full_like(new, 7)
        kda_gdr_decode(*args(one), pool, state_indices=idx, out=o, new_state=s)
        return o, s

    replay_and_compare(g, eager, [out, new])


def test_decode_continues_the_forward():
    say("gdr_fwd over 70 tokens, then three decode steps")
    x = ref.make(2, 73, 2, 4, h0=True, seed=81)
    d = ref.cuda(x)
    pre = {n: d[n][:, :70].contiguous() for n in ("q", "k", "v", "g", "beta")}
    o, S = kda_gdr_fwd(*args(pre), initial_state=d["h0"], final_state=True)
    outs = [o]
    for t in range(70, 73):
        one = {n: d[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")}
        outs.append(kda_gdr_decode(*args(one), S)[0][:, None])
    torch.cuda.synchronize()
    o_ref, h_ref = ref.forward(x, SCALE)
    ref.assert_rows(torch.cat(outs, 1), o_ref, "o", half=ref.forward_magnitude(x, SCALE))
    ref.assert_states(S, h_ref, "state")


def test_far_offsets():
    """Tensors, workspaces and pools of more than 2^31 elements: the last sequence, and the last
    slot, get the bits that they get alone."""
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of free device memory")
    last, T, Hv = 100, 270000, 64
    say(f"gdr_fwd and gdr_bwd, T={T} Hv={Hv}")
    gen = torch.Generator(device="cuda").manual_seed(61)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k = (torch.nn.functional.normalize(rnd(1, T, 1, 128), dim=-1) for _ in range(2))
    v = rnd(1, T, Hv, 128)
    g, beta = -torch.rand(1, T, Hv, device="cuda", generator=gen), torch.rand(1, T, Hv, device="cuda", generator=gen)
    assert v.numel() > 1 << 31
    cu = torch.tensor([0, T - last, T], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, last], dtype=torch.int32, device="cuda")
    tail = [t[:, T - last:].contiguous() for t in (q, k, v, g, beta)]
    o, hT = kda_gdr_fwd(q, k, v, g, beta, SCALE, cu_seqlens=cu, final_state=True)
    o1, h1 = kda_gdr_fwd(*tail, SCALE, cu_seqlens=one, final_state=True)
    assert torch.equal(o[:, T - last:], o1) and torch.equal(hT[1], h1[0]) and torch.isfinite(hT).all()
    del o, hT
    first = 150000   # 2344 chunks of 64 heads: 2^31 elements of kept states are passed
    b = [t[:, T - last - first:].contiguous() for t in (q, k, v, g, beta)]
    do = rnd(1, first + last, Hv, 128)
    del q, k, v, g, beta
    cu = torch.tensor([0, first, first + last], dtype=torch.int32, device="cuda")
    got = kda_gdr_bwd(*b, SCALE, do, cu_seqlens=cu, d_initial_state=True)
    want = kda_gdr_bwd(*tail, SCALE, do[:, first:].contiguous(), cu_seqlens=one, d_initial_state=True)
    assert all(torch.equal(got[n][:, first:], want[n]) for n in ("dq", "dk", "dv", "dg", "dbeta"))
    assert torch.equal(got["dh0"][1], want["dh0"][0])
    assert all(torch.isfinite(got[n]).all() for n in ("dq", "dk", "dg", "dbeta"))
    del got, b, do
    slots = 140000
    say(f"gdr_decode, a pool of {slots} slots")
    pool = torch.empty(slots, 1, 128, 128, device="cuda")
    S = torch.randn(1, 1, 128, 128, device="cuda", generator=gen)
    pool[-1], pool[0] = S[0], 0
    row = [t[:, 0, :1].contiguous() for t in tail]
    a, new = kda_gdr_decode(*row, SCALE, S.clone())
    b, _ = kda_gdr_decode(*row, SCALE, pool, state_indices=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b) and torch.equal(pool[-1], new[0]) and not pool[0].any()
    del pool
    torch.cuda.empty_cache()


def test_refusal_on_device_tensors():
    x = ref.cuda(ref.make(1, 10, 1, 2, seed=91))
    with pytest.raises(KdaError) as e:
        kda_gdr_fwd(*args(x), out=x["v"])
    assert e.value.name == "KDA_ERR_LAYOUT"
    with pytest.raises(ValueError):
        kda_gdr_fwd(x["q"].cpu(), *args(x)[1:])
