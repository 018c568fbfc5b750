"""Plain 64-bit forms of the gated delta rule with one decay per head and of the
per-head q/k norm, token by token on the CPU, and the tolerances of their tests.

Tolerances.  bf16 results are rounded once, by at most 2^-8 of the value
(torch.finfo(bfloat16).eps / 2).  Of the backward and of decode, what enters them carries
at least 16 bits, so sums are off by a few 2^-16 of their largest terms: together
|got - ref| <= 2^-8 |ref| + 2^-13 max|ref| of the head.  The forward's o takes S, A and u
in fp16, each entry off by at most 2^-11 (torch.finfo(float16).eps / 2) of itself: with
o = scale (q . S + sum_j A_j u_j), |A_j| <= sum_c |q_c| |k_jc| decayed, and Sabs the
recurrence of the magnitudes (|S_0| and |k| |u|, decayed), the first part is off by at
most 2^-11 scale |q| Sabs and the second by twice that at most, and since Sabs holds both
parts' sources once, together by 2^-10 scale |q| Sabs, beside the terms above.  fp32 results come from fp32 sums of at most 128 terms at a
time with 24-bit operands: a sum of n terms is off by at most n 2^-24 of the sum of
their magnitudes, so 128 2^-24 = 7.6e-6, and 1.2e-5 with the handful of roundings
around it, relative in the 2-norm of a head's state.  dg and dbeta are differences of
such sums: their errors are compared with the 2-norm of the terms' own scale, the
largest of the head's gradient norm, and held to 2e-5.
"""
import torch

BF16_HALF = 2.0 ** -8
STATE_REL = 1.2e-5
GATE_REL = 2e-5


def recurrence(q, k, v, g, beta, scale, h0=None):
    """One sequence: q, k [T, Hq, D], v [T, Hv, D], g, beta [T, Hv], h0 [Hv, D, D] or
    None, float64.  Returns o [T, Hv, D] and the final state; differentiable."""
    R = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(R, dim=1), k.repeat_interleave(R, dim=1)
    S = torch.zeros(v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if h0 is None else h0
    outs = []
    for t in range(q.shape[0]):
        S = torch.exp(g[t])[:, None, None] * S
        u = beta[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
        S = S + k[t][:, :, None] * u[:, None, :]
        outs.append(scale * torch.einsum("hk,hkv->hv", q[t], S))
    return (torch.stack(outs) if outs else v.clone()), S


def magnitude(q, k, v, g, beta, scale, h0=None):
    """scale |q| Sabs of every token and value channel (see above) of one sequence."""
    R = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(R, dim=1), k.repeat_interleave(R, dim=1)
    S = torch.zeros(v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if h0 is None else h0
    M, outs = S.abs(), []
    for t in range(q.shape[0]):
        S, M = torch.exp(g[t])[:, None, None] * S, torch.exp(g[t])[:, None, None] * M
        u = beta[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
        S, M = S + k[t][:, :, None] * u[:, None, :], M + k[t].abs()[:, :, None] * u.abs()[:, None, :]
        outs.append(scale * torch.einsum("hk,hkv->hv", q[t].abs(), M))
    return torch.stack(outs) if outs else v.clone()


def forward_magnitude(x, scale, cu=None):
    d = {n: (t.detach().cpu().double() if t is not None else None) for n, t in x.items()}
    o = torch.zeros(d["v"].shape, dtype=torch.float64)
    for n, (b, a, e) in enumerate(spans(x, cu)):
        o[b, a:e] = magnitude(*(d[m][b, a:e] for m in ("q", "k", "v", "g", "beta")), scale,
                              d["h0"][n] if d.get("h0") is not None else None)
    return o


def forward(x, scale, cu=None):
    """Batched recurrence of a dict of inputs ([B, T, ...]); cu packs row 0.  Rows in no
    sequence come back as NaN."""
    d = {n: (t.detach().cpu().double() if t is not None else None) for n, t in x.items()}
    o = torch.full(d["v"].shape, float("nan"), dtype=torch.float64)
    states = []
    for n, (b, a, e) in enumerate(spans(x, cu)):
        on, S = recurrence(*(d[m][b, a:e] for m in ("q", "k", "v", "g", "beta")), scale,
                           d["h0"][n] if d.get("h0") is not None else None)
        o[b, a:e] = on
        states.append(S)
    return o, torch.stack(states) if states else torch.zeros(0, x["v"].shape[2], 128, 128, dtype=torch.float64)


def spans(x, cu=None):
    if cu is None:
        return [(b, 0, x["q"].shape[1]) for b in range(x["q"].shape[0])]
    c = [int(i) for i in cu]
    return [(0, a, e) for a, e in zip(c, c[1:])]


def gradients(x, scale, do, dhT=None, cu=None):
    """Gradients by autograd of the recurrence; rows in no sequence NaN."""
    names = ("q", "k", "v", "g", "beta")
    d = {n: x[n].detach().cpu().double() for n in names}
    res = {n: torch.full(d[n].shape, float("nan"), dtype=torch.float64) for n in names}
    h0 = x["h0"].detach().cpu().double() if x.get("h0") is not None else None
    dh = []
    for n, (b, a, e) in enumerate(spans(x, cu)):
        leaves = [d[m][b, a:e].clone().requires_grad_() for m in names]
        S0 = (h0[n].clone() if h0 is not None else torch.zeros(d["v"].shape[2], 128, 128, dtype=torch.float64))
        S0.requires_grad_()
        o, S = recurrence(*leaves, scale, S0)
        loss = (o * do[b, a:e].detach().cpu().double()).sum()
        if dhT is not None:
            loss = loss + (S * dhT[n].detach().cpu().double()).sum()
        got = torch.autograd.grad(loss, leaves + [S0], allow_unused=True)
        for m, gr, leaf in zip(names, got, leaves):
            res[m][b, a:e] = torch.zeros_like(leaf) if gr is None else gr
        dh.append(torch.zeros_like(S0) if got[-1] is None else got[-1])
    res["h0"] = torch.stack(dh) if dh else None
    return res


def norm(x, w=None, mode="l2", eps=1e-6, cos=None, sin=None, pos=None, interleaved=False):
    """x [B, T, H, 128] float64; cos, sin [P, half] float64; pos [B, T] long."""
    n2 = x.pow(2).sum(-1, keepdim=True)
    y = x / torch.sqrt((n2 / 128 if mode == "rms" else n2) + eps)
    if w is not None:
        y = y * w
    if cos is None:
        return y
    h = cos.shape[1]
    if pos is None:
        pos = torch.arange(x.shape[1])[None].expand(x.shape[0], -1)
    pos = pos.clamp(0, cos.shape[0] - 1)
    c, s = cos[pos][:, :, None], sin[pos][:, :, None]
    if interleaved:
        a, b = y[..., 0:2 * h:2], y[..., 1:2 * h:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = y[..., :h], y[..., h:2 * h]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([turned, y[..., 2 * h:]], dim=-1)


def assert_rows(got, ref, what, dim=2, half=None):
    """bf16 rows against 64 bits, head by head (dim); rows whose reference is NaN are skipped.
    half: the magnitudes that entered in fp16.  Rounding alone leaves a 2-norm error of
    2^-8 / sqrt(3) at most over many entries (it is uniform within half a step); with what
    else is allowed here, a tenth more."""
    half = torch.zeros_like(ref) if half is None else half
    got, ref = got.detach().cpu().double(), ref.detach()
    for h in range(ref.shape[dim]):
        a, b, m = got.select(dim, h), ref.select(dim, h), half.select(dim, h)
        real = ~torch.isnan(b)
        if not real.any():
            continue
        top = b[real].abs().max()
        off = ((a - b).abs()[real] - BF16_HALF * b.abs()[real] - 2.0 ** -10 * m[real]).max()
        assert torch.isfinite(a[real]).all() and off <= 2.0 ** -13 * top, (what, h, float(off), float(top))
        if int(real.sum()) >= 4096:
            assert rel(a, b) <= 1.1 * BF16_HALF / 3 ** 0.5, (what, h, rel(a, b))


def rel(got, ref):
    got, ref = got.detach().cpu().double(), ref.detach()
    real = ~torch.isnan(ref)
    n = ref[real].norm()
    d = (got[real] - ref[real]).norm()
    return float(d / n) if n > 0 else float(d)


def assert_states(got, ref, what):
    for n in range(ref.shape[0]):
        for h in range(ref.shape[1]):
            r = rel(got[n, h], ref[n, h])
            assert r <= STATE_REL, (what, n, h, r)


def assert_gates(got, ref, what):
    """dg or dbeta [B, T, Hv] against the largest of the heads' norms."""
    got, ref = got.detach().cpu().double(), ref.detach()
    real = ~torch.isnan(ref)
    ref0 = torch.where(real, ref, torch.zeros_like(ref))
    got0 = torch.where(real, got, torch.zeros_like(ref))
    norms = ref0.flatten(0, 1).norm(dim=0)
    err = (got0 - ref0).flatten(0, 1).norm(dim=0)
    assert (err <= GATE_REL * norms.max().clamp(min=1e-30)).all(), (what, float(err.max()), float(norms.max()))


def make(B, T, Hq, Hv, beta_dtype=torch.float32, h0=False, N=None, seed=0, lo=0.001, hi=2.0, unit=True):
    """Inputs of a batch on the CPU: log-decays -lo .. -hi spread over their logarithm."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    f = (lambda t: t / t.norm(dim=-1, keepdim=True).clamp(min=1e-6)) if unit else (lambda t: t)
    x = dict(q=f(rnd(B, T, Hq, 128)).bfloat16(), k=f(rnd(B, T, Hq, 128)).bfloat16(), v=rnd(B, T, Hv, 128).bfloat16())
    x["g"] = -lo * (hi / lo) ** torch.rand(B, T, Hv, generator=gen)
    x["beta"] = torch.sigmoid(rnd(B, T, Hv)).to(beta_dtype)
    n = B if N is None else N
    x["h0"] = 0.1 * rnd(n, Hv, 128, 128) if h0 else None
    return x


def cuda(x):
    return {n: (t.cuda() if t is not None else None) for n, t in x.items()}
