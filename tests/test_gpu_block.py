"""GPU checks of the operators as a block runs them: each one reads, through views, what the one before it
wrote.  Every step is held to its own 64-bit form of the very tensors that it read, within that form's
tolerance, so that nothing builds up over the chain."""
import pytest
import torch

from gated_delta_rule_35_amd import (kda_add_norm, kda_add_norm_bwd, kda_conv, kda_conv_bwd, kda_conv_bwd_workspace_size,
                                     kda_conv_decode, kda_gated_norm, kda_gated_norm_bwd, kda_gdr_decode, kda_gdr_fwd,
                                     kda_qk_norm, kda_ssm_bwd, kda_ssm_bwd_workspace_size, kda_ssm_decode, kda_ssm_fwd,
                                     kda_ssm_fwd_workspace_size, load_library)
from tests import block_ref, gdr_ref, ssm_ref
from tests.block_ref import d64

pytestmark = pytest.mark.gpu
EPS = 1e-6
H, P, S, G, W, D = 8, 64, 128, 2, 4, 128   # heads, their width, states, groups, taps, width of the model
INNER, MIXED = H * P, H * P + 2 * G * S    # channels of x, and of x, B and C together


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    load_library()
    yield


def say(msg):
    print(f"[gpu] {msg}", flush=True)


def weights(seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    w = dict(n1=1 + 0.2 * rnd(D), into=(rnd(D, INNER + MIXED + H) / D ** 0.5).bfloat16(), conv=rnd(MIXED, W) / W ** 0.5, cb=0.1 * rnd(MIXED),
             A=-(1 + 7 * torch.rand(H, generator=gen)), D=1 + 0.2 * rnd(H), bias=-3 + rnd(H), gate=1 + 0.2 * rnd(H, P),
             out=(rnd(INNER, D) / INNER ** 0.5).bfloat16(), n2=1 + 0.2 * rnd(D))
    return {n: t.cuda() for n, t in w.items()}


def parts(xbc):
    """x, B and C as views of the convolution's result [.., T, MIXED]."""
    x, B, C = xbc.split([INNER, G * S, G * S], dim=-1)
    return x.unflatten(-1, (H, P)), B.unflatten(-1, (G, S)), C.unflatten(-1, (G, S))


def project(n, w):
    u = torch.matmul(n.flatten(0, -2), w["into"]).unflatten(0, n.shape[:-1])
    z, xbc, dt = u.split([INNER, MIXED, H], dim=-1)
    return z.unflatten(-1, (H, P)), xbc, dt


def forward(hid, res, w, cu=None, state=None, h0=None, scratch=None):
    """The block over whole sequences: everything that its backward pass and the checks need."""
    s = {}
    s["n"], s["res"] = kda_add_norm(hid, res, w["n1"], eps=EPS)
    s["z"], s["xbc"], s["dt"] = project(s["n"], w)
    s["mixed"], s["last"] = kda_conv(s["xbc"], w["conv"], w["cb"], cu_seqlens=cu, initial_state=state, final_state=True,
                                     out=torch.zeros_like(s["xbc"], memory_format=torch.contiguous_format))
    s["x"], s["B"], s["C"] = parts(s["mixed"])
    s["y"], s["hT"] = kda_ssm_fwd(s["x"], s["dt"], w["A"], s["B"], s["C"], D=w["D"], dt_bias=w["bias"], cu_seqlens=cu,
                                  initial_state=h0, final_state=True, workspace=scratch,
                                  out=torch.zeros(s["x"].shape, dtype=hid.dtype, device=hid.device))
    s["g"] = kda_gated_norm(s["y"], s["z"], w["gate"], gate_first=True, eps=EPS)
    s["o"] = torch.matmul(s["g"].flatten(0, 1).flatten(1), w["out"]).view(hid.shape)
    s["out"], s["sum"] = kda_add_norm(s["o"], s["res"], w["n2"], eps=EPS)
    return s


def backward(s, d_out, d_sum, w, cu=None, state=None, h0=None, dlast=None, dhT=None, scratch=None, conv_scratch=None):
    g = {}
    g["n2"] = kda_add_norm_bwd(s["sum"], d_out, w["n2"], eps=EPS, d_sum=d_sum)
    do = g["n2"]["dx"].flatten(0, 1)
    g["dg"] = torch.matmul(do, w["out"].t().contiguous()).view(s["y"].shape)
    g["gate"] = kda_gated_norm_bwd(s["y"], s["z"], g["dg"], w["gate"], gate_first=True, eps=EPS)
    zero = lambda t: torch.zeros(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
    g["ssm"] = kda_ssm_bwd(s["x"], s["dt"], w["A"], s["B"], s["C"], g["gate"]["dx"], D=w["D"], dt_bias=w["bias"], cu_seqlens=cu,
                           initial_state=h0, d_final_state=dhT, d_initial_state=h0 is not None, workspace=scratch,
                           grads=dict(dx=zero(s["x"]), dB=zero(s["B"]), dC=zero(s["C"]), ddt=torch.zeros(s["dt"].shape, device="cuda")))
    g["dmixed"] = torch.cat([g["ssm"][n].flatten(-2) for n in ("dx", "dB", "dC")], dim=-1)
    g["conv"] = kda_conv_bwd(s["xbc"], w["conv"], g["dmixed"], w["cb"], cu_seqlens=cu, initial_state=state, d_final_state=dlast,
                             d_initial_state=state is not None, grads=dict(dx=zero(s["xbc"])), workspace=conv_scratch)
    du = torch.cat([g["gate"]["dgate"].flatten(-2), g["conv"]["dx"], g["ssm"]["ddt"].to(d_out.dtype)], dim=-1)
    dn = torch.matmul(du.flatten(0, 1), w["into"].t().contiguous()).view(s["n"].shape)
    g["dn"] = dn
    g["n1"] = kda_add_norm_bwd(s["res"], dn, w["n1"], eps=EPS, d_sum=g["n2"]["dresidual"])
    return g


def inputs(B, T, N, seed, states):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = dict(hid=rnd(B, T, D).bfloat16(), res=rnd(B, T, D), d_out=rnd(B, T, D).bfloat16(), d_sum=rnd(B, T, D))
    if states:
        d.update(state=rnd(N, W - 1, MIXED).bfloat16(), h0=rnd(N, H, S, P), dlast=rnd(N, W - 1, MIXED).bfloat16(), dhT=rnd(N, H, S, P))
    d = {n: t.cuda() for n, t in d.items()}
    return {n: d.get(n) for n in ("hid", "res", "d_out", "d_sum", "state", "h0", "dlast", "dhT")}


def check_add(x, res, w, y, h):
    want = d64(res) + d64(x)
    mag = d64(res).abs() + d64(x).abs()
    block_ref.close(h, want, 2.0 ** -24 * mag, "sum")
    r = block_ref.rms(want, EPS)
    block_ref.close(y, want * r * d64(w), 2.0 ** -17 * (want * r * d64(w)).abs() + 2.0 ** -23 * r * mag * d64(w).abs(), "norm of the sum")


def check_add_grads(h, w, dy, dh, g):
    hl, wl = d64(h).requires_grad_(), d64(w).requires_grad_()
    got = torch.autograd.grad(hl * block_ref.rms(hl, EPS) * wl, [hl, wl], d64(dy))
    with torch.no_grad():
        size = 2.0 ** -16 * block_ref.norm_grad_size(hl, d64(dy) * wl, EPS) + 2.0 ** -24 * d64(dh).abs()
        per = (d64(dy) * hl * block_ref.rms(hl, EPS)).abs().sum((0, 1))
    total = got[0] + d64(dh)
    block_ref.close(g["dresidual"], total, size, "dresidual")
    block_ref.close(g["dx"], total, size + 2.0 ** -24 * total.abs(), "dx of the sum")
    block_ref.close(g["dweight"], got[1], 2.0 ** -16 * per, "dweight of the sum's norm")


def scan_case(s, w, i, dy=None):
    return dict(x=s["x"], dt=s["dt"], A=w["A"], B=s["B"], C=s["C"], D=w["D"], bias=w["bias"], h0=i["h0"], dy=dy, dlast=i["dhT"], softplus=True)


def check_forward(s, i, w, cu=None):
    check_add(i["hid"], i["res"], w["n1"], s["n"], s["res"])
    want, mag, last = block_ref.conv_batch(s["xbc"], w["conv"], w["cb"], "silu", cu, i["state"])
    real = ~torch.isnan(want)
    block_ref.close(s["mixed"].cpu()[real], want[real], 2.0 ** -20 * mag[real], "convolution")
    assert torch.equal(d64(s["last"]), last), "the convolution's last inputs"
    y, ym, hT, hm = ssm_ref.run(scan_case(s, w, i), cu)
    ssm_ref.close(s["y"], y, ssm_ref.BITS["y"] * ym, "scan")
    ssm_ref.close(s["hT"], hT, ssm_ref.BITS["state"] * hm, "final state")
    want = block_ref.gated(d64(s["y"]), d64(s["z"]), d64(w["gate"]), "silu", True, EPS)
    block_ref.close(s["g"], want, 2.0 ** -17 * want.abs(), "gated norm")
    check_add(s["o"], s["res"], w["n2"], s["out"], s["sum"])


def check_backward(s, g, i, w, cu=None):
    check_add_grads(s["sum"], w["n2"], i["d_out"], i["d_sum"], g["n2"])
    xl, zl, wl = (d64(t).requires_grad_() for t in (s["y"], s["z"], w["gate"]))
    got = torch.autograd.grad(block_ref.gated(xl, zl, wl, "silu", True, EPS), [xl, zl, wl], d64(g["dg"]))
    with torch.no_grad():
        a = block_ref.act(zl, "silu")
        v = xl * a
        size = block_ref.norm_grad_size(v, d64(g["dg"]) * wl, EPS)
        per = (d64(g["dg"]) * v * block_ref.rms(v, EPS)).abs().sum((0, 1))
        block_ref.close(g["gate"]["dx"], got[0], 2.0 ** -16 * size * a.abs(), "dx of the gated norm")
        block_ref.close(g["gate"]["dgate"], got[1], 2.0 ** -16 * 1.2 * size * xl.abs(), "dgate")
        block_ref.close(g["gate"]["dweight"], got[2], 2.0 ** -16 * per, "dweight of the gated norm")
    want, mag = ssm_ref.gradients(scan_case(s, w, i, g["gate"]["dx"]), cu)
    for n in ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias") + (("dh0",) if i["h0"] is not None else ()):
        ssm_ref.close(g["ssm"][n], want[n], ssm_ref.BITS[n] * mag[n], n)
    want, mag = block_ref.conv_grads(s["xbc"], w["conv"], g["dmixed"], w["cb"], "silu", cu, i["state"], i["dlast"])
    real = ~torch.isnan(want["dx"])
    block_ref.close(g["conv"]["dx"].cpu()[real], want["dx"][real], 2.0 ** -20 * mag["dx"][real], "dx of the convolution")
    for n, off in (("dweight", 2.0 ** -15), ("dbias", 2.0 ** -15)) + ((("dstate", 2.0 ** -20),) if i["state"] is not None else ()):
        block_ref.close(g["conv"][n], want[n], off * mag[n], n)
    check_add_grads(s["res"], w["n1"], g["dn"], g["n2"]["dresidual"], g["n1"])


@pytest.mark.parametrize("B,T,cu,states", [(2, 70, None, False), (1, 1, None, True), (1, 150, [0, 1, 66, 66, 130, 141], True)])
def test_scan_block(B, T, cu, states):
    """Sum and norm, projection, convolution, scan, gated norm, projection, sum and norm, and all of it backwards."""
    say(f"block with a scan B={B} T={T} {cu}")
    w, i = weights(1), inputs(B, T, B if cu is None else len(cu) - 1, T, states)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    s = forward(i["hid"], i["res"], w, c, i["state"], i["h0"])
    g = backward(s, i["d_out"], i["d_sum"], w, c, i["state"], i["h0"], i["dlast"], i["dhT"])
    torch.cuda.synchronize()
    check_forward(s, i, w, cu)
    check_backward(s, g, i, w, cu)


def test_scan_block_decode():
    """A prompt and five tokens after it, states in pools, two sequences of three slots: the whole as one sequence."""
    say("block with a scan: prompt, then tokens")
    w, T, more = weights(2), 67, 5
    i = inputs(2, T + more, 2, 5, True)
    s = forward(i["hid"][:, :T].contiguous(), i["res"][:, :T].contiguous(), w, None, i["state"], i["h0"])
    slots = torch.tensor([2, 0, -1], dtype=torch.int32, device="cuda")
    taps, pool = torch.full((3, W - 1, MIXED), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((3, H, S, P), 9.0, device="cuda")
    taps[[2, 0]], pool[[2, 0]] = s["last"], s["hT"]
    names = ("n", "res", "z", "xbc", "dt", "mixed", "y", "g", "o", "out", "sum")
    rows = {n: [s[n]] for n in names}
    for t in range(T, T + more):
        hid, res = (torch.cat([v[:, t], v[:1, t]]) for v in (i["hid"], i["res"]))   # a third row that pads the batch
        k = {}
        k["n"], k["res"] = (v[:, 0] for v in kda_add_norm(hid[:, None], res[:, None], w["n1"], eps=EPS))
        k["z"], k["xbc"], k["dt"] = project(k["n"], w)
        k["mixed"] = torch.zeros_like(k["xbc"], memory_format=torch.contiguous_format)
        kda_conv_decode(k["xbc"], w["conv"], taps, w["cb"], state_indices=slots, out=k["mixed"])
        x, B, C = parts(k["mixed"])
        k["y"] = torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda")
        kda_ssm_decode(x, k["dt"], w["A"], B, C, pool, D=w["D"], dt_bias=w["bias"], state_indices=slots, out=k["y"])
        k["g"] = kda_gated_norm(k["y"][:, None], k["z"][:, None], w["gate"], gate_first=True, eps=EPS)[:, 0]
        k["o"] = torch.matmul(k["g"].flatten(1), w["out"])
        k["out"], k["sum"] = (v[:, 0] for v in kda_add_norm(k["o"][:, None], k["res"][:, None], w["n2"], eps=EPS))
        for n in names:
            rows[n].append(k[n][:2, None])
    torch.cuda.synchronize()
    s = {n: torch.cat(v, dim=1) for n, v in rows.items()}
    s["x"], s["B"], s["C"] = parts(s["mixed"])
    s["last"], s["hT"] = taps[[2, 0]], pool[[2, 0]]
    check_forward(s, i, w)
    assert (taps[1] == 9).all() and (pool[1] == 9).all(), "the slot that no row names"


def test_scan_block_graph():
    """Forward and backward of the block in one graph, replayed on new inputs beside eager runs."""
    say("block with a scan in a graph")
    T = 130
    w, i = weights(3), inputs(1, T, 1, 8, True)
    sizes = (T, 1, H, G, P, S)
    scratch = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
               (kda_ssm_fwd_workspace_size(*sizes), kda_ssm_bwd_workspace_size(*sizes), kda_conv_bwd_workspace_size(T, MIXED, W))]

    def step(a=None, b=None, c=None):
        s = forward(i["hid"], i["res"], w, None, i["state"], i["h0"], a)
        g = backward(s, i["d_out"], i["d_sum"], w, None, i["state"], i["h0"], i["dlast"], i["dhT"], b, c)
        return [s["out"], s["sum"], s["last"], s["hT"]] + [t for n in ("n2", "gate", "ssm", "conv", "n1") for t in g[n].values() if t is not None]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):   # the library's products take their workspaces here
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        inside = step(*scratch)
    for r in range(3):
        for n, t in inputs(1, T, 1, 20 + r, True).items():
            i[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in inside]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, eager)), r


def test_delta_rule_block():
    """Convolution, q/k norm on its views, gated delta rule, gated norm: a packed prompt, then tokens from its states."""
    say("block with the delta rule: prompt, then tokens")
    gen = torch.Generator().manual_seed(31)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    Hq, Hv, C, lens, more = 2, 4, 2 * 2 * 128 + 4 * 128, [40, 75], 4
    full = [n + more for n in lens]
    cu, whole = [0, lens[0], sum(lens)], [0, full[0], sum(full)]
    u, gate = rnd(1, whole[-1], C).bfloat16(), rnd(1, whole[-1], Hv, 128).bfloat16()
    g, beta = -torch.rand(1, whole[-1], Hv, generator=gen), torch.sigmoid(rnd(1, whole[-1], Hv))
    w, wn = rnd(C, W) / 2, 1 + 0.2 * rnd(128)
    prompt = torch.cat([torch.arange(a, a + n) for a, n in zip(whole, lens)])
    d = [t.cuda() for t in (u, gate, g, beta, w, wn)]
    U, Z, g_, b_, w_, wn_ = d
    split = lambda t: [p.unflatten(-1, (-1, 128)) for p in t.split([Hq * 128, Hq * 128, Hv * 128], dim=-1)]  # noqa: E731
    scale = 128 ** -0.5
    got = dict(mixed=torch.zeros_like(U), q=torch.zeros(1, whole[-1], Hq, 128, dtype=torch.bfloat16, device="cuda"))
    got["k"], got["o"], got["y"] = torch.zeros_like(got["q"]), torch.zeros_like(Z), torch.zeros_like(Z)
    at = prompt.cuda()
    mixed, taps = kda_conv(U[:, at], w_, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), final_state=True)
    q, k, v = split(mixed)
    q, k = kda_qk_norm(q, k)
    o, state = kda_gdr_fwd(q, k, v, g_[:, at], b_[:, at], scale, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), final_state=True)
    y = kda_gated_norm(o, Z[:, at], wn_)
    for n, t in (("mixed", mixed), ("q", q), ("k", k), ("o", o), ("y", y)):
        got[n][:, at] = t
    for j in range(more):
        at = torch.tensor([a + n + j for a, n in zip(whole, lens)], device="cuda")
        mixed, _ = kda_conv_decode(U[0, at], w_, taps)
        q, k, v = split(mixed)
        q, k = (t[:, 0] for t in kda_qk_norm(q[:, None], k[:, None]))
        o, _ = kda_gdr_decode(q, k, v, g_[0, at], b_[0, at], scale, state)
        y = kda_gated_norm(o[:, None], Z[0, at][:, None], wn_)[:, 0]
        for n, t in (("mixed", mixed), ("q", q), ("k", k), ("o", o), ("y", y)):
            got[n][0, at] = t
    torch.cuda.synchronize()
    want, mag, last = block_ref.conv_batch(u, w, None, "silu", whole)
    block_ref.close(got["mixed"], want, 2.0 ** -20 * mag, "convolution")
    assert torch.equal(d64(taps), last)
    q, k, v = split(got["mixed"])
    for n, t in (("q", q), ("k", k)):
        want = gdr_ref.norm(d64(t))
        block_ref.close(got[n], want, 1e-5 * want.abs().amax(dim=-1, keepdim=True), n)
    x = dict(q=got["q"], k=got["k"], v=v, g=g, beta=beta, h0=None)
    want, hT = gdr_ref.forward(x, scale, whole)
    gdr_ref.assert_rows(got["o"], want, "o", half=gdr_ref.forward_magnitude(x, scale, whole))
    gdr_ref.assert_states(state, hT, "final state")
    want = block_ref.gated(d64(got["o"]), d64(gate), d64(wn), "silu", False, EPS)
    block_ref.close(got["y"], want, 2.0 ** -17 * want.abs(), "gated norm")
