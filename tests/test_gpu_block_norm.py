"""GPU checks of the norms around a block and their gradients against 64 bits."""
import pytest
import torch

from gated_delta_rule_35_amd import (KdaError, kda_add_norm, kda_add_norm_bwd, kda_gated_norm, kda_gated_norm_bwd,
                                     kda_norm_bwd_workspace_size, load_library)
from tests import block_ref as ref
from tests.block_ref import TYPES, d64

pytestmark = pytest.mark.gpu
NAN, EPS = float("nan"), 1e-6


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


def make_gated(B, T, H, D, kind, weight, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    t = TYPES[kind]
    w = None if weight is None else 1 + 0.3 * (rnd(H, D) if weight == "heads" else rnd(D))
    return dict(x=rnd(B, T, H, D).to(t), gate=(2 * rnd(B, T, H, D)).to(t), w=w, dy=rnd(B, T, H, D).to(t))


def check_gated(c, act, first, x=None, gate=None, eps=EPS):
    d = {n: cuda(t) for n, t in c.items()}
    x, gate = d["x"] if x is None else x, d["gate"] if gate is None else gate
    y = kda_gated_norm(x, gate, d["w"], activation=act, gate_first=first, eps=eps)
    g = kda_gated_norm_bwd(x, gate, d["dy"], d["w"], activation=act, gate_first=first, eps=eps)
    torch.cuda.synchronize()
    xl, zl = d64(c["x"]).requires_grad_(), d64(c["gate"]).requires_grad_()
    wl = None if c["w"] is None else d64(c["w"]).requires_grad_()
    want = ref.gated(xl, zl, wl, act, first, eps)
    assert y.dtype == c["x"].dtype and y.is_contiguous()
    ref.close(y, want.detach(), 2.0 ** -17 * want.detach().abs(), "y")
    got = torch.autograd.grad(want, [xl, zl] + ([] if wl is None else [wl]), d64(c["dy"]))
    with torch.no_grad():
        a, w, dy = ref.act(zl, act), 1.0 if wl is None else wl, d64(c["dy"])
        v = xl * a if first else xl
        dn = dy * w if first else dy * a * w
        size = ref.norm_grad_size(v, dn, eps)
        n = v * ref.rms(v, eps)
        ref.close(g["dx"], got[0], 2.0 ** -16 * size * (a.abs() if first else 1), "dx")
        ref.close(g["dgate"], got[1], 2.0 ** -16 * 1.2 * (size * xl.abs() if first else (dy * n * w).abs()), "dgate")
        if wl is None:
            assert g["dweight"] is None
        else:
            per = (dy * n * (1 if first else a)).abs().sum((0, 1) if wl.dim() == 2 else (0, 1, 2))
            ref.close(g["dweight"], got[2], 2.0 ** -16 * per, "dweight")
    return y, g


GATED = [
    (1, 1, 1, 8, "bf16", "shared", "silu", False), (2, 3, 2, 128, "f16", "heads", "sigmoid", False),
    (1, 17, 3, 64, "f32", "shared", "silu", True), (1, 33, 5, 136, "bf16", "heads", "silu", False),
    (2, 9, 1, 512, "bf16", None, "sigmoid", True), (1, 21, 2, 520, "f32", "shared", "sigmoid", False),
    (1, 5, 3, 1024, "f16", "heads", "silu", True), (2, 7, 1, 1032, "bf16", "shared", "silu", False),
    (1, 13, 1, 2048, "f32", "heads", "silu", True), (1, 6, 2, 2056, "bf16", "heads", "silu", False),
    (1, 11, 1, 4096, "f32", "shared", "sigmoid", True), (1, 3, 1, 4104, "f16", "shared", "silu", False),
    (1, 5, 1, 8192, "f32", "shared", "silu", False), (2, 3, 2, 8192, "bf16", "heads", "silu", True),
    (1, 100, 64, 128, "bf16", "shared", "silu", False), (1, 7, 9, 192, "bf16", "shared", "silu", True),
]


@pytest.mark.parametrize("B,T,H,D,kind,weight,act,first", GATED)
def test_gated(B, T, H, D, kind, weight, act, first):
    say(f"gated_norm B={B} T={T} H={H} D={D} {kind} {weight} {act} first={first}")
    check_gated(make_gated(B, T, H, D, kind, weight, seed=D + T), act, first)


ADD = [
    (1, 1, 8, "bf16", "bf16", 1.0, True), (2, 3, 64, "f16", "f16", 0.5, True), (1, 37, 128, "f32", "f32", -1.5, True),
    (3, 5, 136, "bf16", "f32", 0.25, False), (1, 9, 520, "f16", "f32", 1.0, True), (1, 5, 1032, "bf16", "bf16", 0.0, True),
    (2, 5, 2048, "bf16", "f32", 0.7, True), (1, 7, 4096, "f32", "f32", 1.0, True), (1, 3, 4104, "bf16", "bf16", 2.0, False),
    (2, 2, 8192, "f16", "f32", 1.0, True),
]


def make_add(B, T, D, kind, res, weight, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=rnd(B, T, D).to(TYPES[kind]), res=(2 * rnd(B, T, D)).to(TYPES[res]), w=1 + 0.3 * rnd(D) if weight else None,
                dy=rnd(B, T, D).to(TYPES[kind]), dh=rnd(B, T, D).to(TYPES[res]))


def check_add(c, scale, x=None, res=None):
    d = {n: cuda(t) for n, t in c.items()}
    y, h = kda_add_norm(d["x"] if x is None else x, d["res"] if res is None else res, d["w"], scale=scale, eps=EPS)
    torch.cuda.synchronize()
    s = float(torch.tensor(scale, dtype=torch.float32))
    want = d64(c["res"]) + s * d64(c["x"])
    mag = d64(c["res"]).abs() + abs(s) * d64(c["x"]).abs()
    w = 1.0 if c["w"] is None else d64(c["w"])
    assert y.dtype == c["x"].dtype and h.dtype == c["res"].dtype
    ref.close(h, want, 2.0 ** -24 * mag, "sum")
    r = ref.rms(want, EPS)
    ref.close(y, want * r * w, 2.0 ** -17 * (want * r * w).abs() + 2.0 ** -23 * (r * mag * w), "y")
    for dh in (d["dh"], None):
        g = kda_add_norm_bwd(h, d["dy"], d["w"], scale=scale, eps=EPS, d_sum=dh)
        torch.cuda.synchronize()
        hl = d64(h).requires_grad_()
        wl = None if c["w"] is None else d64(c["w"]).requires_grad_()
        yl = hl * ref.rms(hl, EPS) * (1.0 if wl is None else wl)
        got = torch.autograd.grad(yl, [hl] + ([] if wl is None else [wl]), d64(c["dy"]))
        total = got[0] + (0 if dh is None else d64(c["dh"]))
        with torch.no_grad():
            size = 2.0 ** -16 * ref.norm_grad_size(hl, d64(c["dy"]) * w, EPS) + (0 if dh is None else 2.0 ** -24 * d64(c["dh"]).abs())
        ref.close(g["dresidual"], total, size, "dresidual")
        ref.close(g["dx"], s * total, abs(s) * (size + 2.0 ** -24 * total.abs()), "dx")
        assert g["dx"].dtype == c["dy"].dtype and g["dresidual"].dtype == c["res"].dtype
        if wl is None:
            assert g["dweight"] is None
        else:
            with torch.no_grad():
                per = (d64(c["dy"]) * hl * ref.rms(hl, EPS)).abs().sum((0, 1))
            ref.close(g["dweight"], got[1], 2.0 ** -16 * per, "dweight")
    return y, h


@pytest.mark.parametrize("B,T,D,kind,res,scale,weight", ADD)
def test_add(B, T, D, kind, res, scale, weight):
    say(f"add_norm B={B} T={T} D={D} {kind} residual {res} scale={scale} weight={weight}")
    check_add(make_add(B, T, D, kind, res, weight, seed=D), scale)


@pytest.mark.parametrize("rows,H,D,weight", [(2500, 1, 128, "shared"), (1700, 3, 64, "heads"), (4200, 1, 256, "shared"),
                                             (1300, 1, 4096, "shared"), (2, 1100, 16, "heads")])
def test_many_rows_share_work_groups(rows, H, D, weight):
    """More rows than work-groups of the weights' gradients take at once, ragged at the end; repeatable."""
    say(f"gated_norm_bwd {rows} x {H} x {D} {weight}")
    c = make_gated(1, rows, H, D, "bf16", weight, seed=rows)
    _, g = check_gated(c, "silu", False)
    again = kda_gated_norm_bwd(c["x"].cuda(), c["gate"].cuda(), c["dy"].cuda(), c["w"].cuda(), eps=EPS)
    torch.cuda.synchronize()
    for n in g:
        assert torch.equal(g[n], again[n]), n


def test_rows_of_nothing_and_of_extremes():
    """Rows of zeros, gates of 0 and of both infinities' neighbourhood, rows far above and below one."""
    say("norms of extreme rows")
    c = make_gated(1, 6, 1, 128, "f32", "shared", seed=1)
    c["x"][0, 0] = 0
    c["x"][0, 1] *= 1e12
    c["x"][0, 2] *= 1e-12
    c["gate"][0, 3], c["gate"][0, 4], c["gate"][0, 5] = 0, 80.0, -80.0
    for first in (False, True):
        y, g = check_gated(c, "silu", first)
        assert (y[0, 0] == 0).all()
    y, _ = check_gated(c, "sigmoid", True)
    a = make_add(1, 3, 64, "f32", "f32", True, seed=2)
    a["x"][0, 0], a["res"][0, 0] = 0, 0
    a["res"][0, 1] *= 1e12
    check_add(a, 1.0)


def test_views_and_aliases():
    say("norm views")
    c = make_gated(2, 11, 4, 128, "bf16", "shared", seed=3)
    wide = torch.full((2, 11, 3 * 512 + 64), NAN, dtype=torch.bfloat16)
    wide[..., 64:576], wide[..., 1088:1600] = c["x"].flatten(2), c["gate"].flatten(2)
    wide = wide.cuda()
    base, gb = check_gated(c, "silu", False)
    y, g = check_gated(c, "silu", False, x=wide[..., 64:576].unflatten(-1, (4, 128)), gate=wide[..., 1088:1600].unflatten(-1, (4, 128)))
    assert torch.equal(y, base) and all(torch.equal(g[n], gb[n]) for n in g)
    # heads before tokens, and one gate for all heads
    y, _ = check_gated(c, "silu", False, x=c["x"].transpose(1, 2).contiguous().cuda().transpose(1, 2))
    assert torch.equal(y, base)
    c["gate"] = c["gate"][:, :, :1].expand(-1, -1, 4, -1)
    check_gated(c, "silu", False, gate=c["gate"][:, :, :1].contiguous().cuda().expand(-1, -1, 4, -1))
    c = make_gated(2, 11, 4, 128, "bf16", "shared", seed=3)
    x = c["x"].cuda()
    kda_gated_norm(x, c["gate"].cuda(), c["w"].cuda(), out=x)
    assert torch.equal(x, base)
    for kind, res, D in (("bf16", "f32", 136), ("f16", "f16", 4096)):
        a = make_add(2, 7, D, kind, res, True, seed=4)
        y0, h0 = check_add(a, 0.5)
        x, r = a["x"].cuda(), a["res"].cuda()
        kda_add_norm(x, r, a["w"].cuda(), scale=0.5, out=x, new_residual=r)
        assert torch.equal(x, y0) and torch.equal(r, h0)
        pad = torch.full((2, 7, D + 16), NAN, dtype=a["x"].dtype)
        pad[..., 8:8 + D] = a["x"]
        y, h = check_add(a, 0.5, x=pad.cuda()[..., 8:8 + D])
        assert torch.equal(y, y0) and torch.equal(h, h0)


def test_empty():
    for B, T in ((0, 3), (2, 0)):
        x = torch.zeros(B, T, 2, 64, device="cuda")
        w = torch.ones(64, device="cuda")
        assert kda_gated_norm(x, x, w).shape == x.shape
        g = kda_gated_norm_bwd(x, x, x, w)
        torch.cuda.synchronize()
        assert (g["dweight"] == 0).all()
        h = torch.zeros(B, T, 64, device="cuda")
        kda_add_norm(h, torch.zeros_like(h), w)
        g = kda_add_norm_bwd(h, torch.zeros_like(h), w)
        torch.cuda.synchronize()
        assert (g["dweight"] == 0).all()


def test_gradients_match_differences():
    say("norm differences")
    gen = torch.Generator().manual_seed(7)
    c = make_gated(1, 3, 2, 24, "f32", "heads", seed=6)
    d = {n: cuda(t) for n, t in c.items()}
    h = 1e-5
    for first in (False, True):
        g = kda_gated_norm_bwd(d["x"], d["gate"], d["dy"], d["w"], gate_first=first, eps=EPS)
        for name, key in (("x", "dx"), ("gate", "dgate"), ("w", "dweight")):
            v = torch.randn(c[name].shape, generator=gen, dtype=torch.float64)

            def loss(e):
                a = {n: d64(t) for n, t in c.items()}
                a[name] = a[name] + e * v
                return float((ref.gated(a["x"], a["gate"], a["w"], "silu", first, EPS) * a["dy"]).sum())

            along, diff = float((d64(g[key]) * v).sum()), (loss(h) - loss(-h)) / (2 * h)
            assert abs(along - diff) <= 1e-5 * float(d64(g[key]).norm() * v.norm()), (name, first, along, diff)


def test_two_streams_and_graph():
    say("norms side by side and in a graph")
    c = {n: cuda(t) for n, t in make_gated(2, 500, 2, 256, "bf16", "heads", seed=8).items()}
    a = {n: cuda(t) for n, t in make_add(2, 300, 1024, "bf16", "f32", True, seed=9).items()}

    def step(s=None, **kw):
        y = kda_gated_norm(c["x"], c["gate"], c["w"], stream=s)
        g = kda_gated_norm_bwd(c["x"], c["gate"], c["dy"], c["w"], stream=s, **kw)
        z, h = kda_add_norm(a["x"], a["res"], a["w"], scale=0.5, stream=s)
        f = kda_add_norm_bwd(h, a["dy"], a["w"], scale=0.5, d_sum=a["dh"], stream=s)
        return [y, *g.values(), z, h, *f.values()]

    base = step()
    torch.cuda.synchronize()
    many = [step(s) for s in (torch.cuda.Stream(), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for r in many:
        assert all(torch.equal(x, y) for x, y in zip(base, r))
    ws = torch.empty(kda_norm_bwd_workspace_size(2, 256), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = step(workspace=ws)
    for i in range(3):
        gen = torch.Generator().manual_seed(i)
        c["x"].copy_(torch.randn(c["x"].shape, generator=gen))
        a["res"].copy_(torch.randn(a["res"].shape, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in inside]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, eager))


def test_refused():
    x = torch.zeros(1, 4, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(KdaError) as e:
        kda_gated_norm(x, x, w, out=x)   # the gate would be overwritten
    assert e.value.name == "KDA_ERR_LAYOUT"
    with pytest.raises(ValueError, match="activation"):
        kda_gated_norm(x, x, w, activation=None)
    with pytest.raises(ValueError, match="on the GPU"):
        kda_gated_norm(x, x.cpu(), w)
