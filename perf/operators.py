"""Measured cases of the gated delta rule with one decay per head and of the q/k norm before it.

Operators (`case["op"]`):

  gdr_fwd      the chunked forward: S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T, o_t = scale S_t^T q_t,
               g and beta one number per token and value head
  gdr_bwd      its gradients with respect to q, k, v, g, beta and the initial state
  gdr_decode   one token per sequence, the states in a pool that a slot map indexes
  qk_norm      per-head norm of queries and keys, with an optional weight and position rotation
  qk_norm_bwd  its gradients with respect to the inputs and the weights

`own` False: the plain forms below, in torch operations on 32 bits (log-decays summed in 64).  `own` True: the
framework's entry points on the same inputs.
"""
import math

import numpy as np
import torch

own = False

D = 128        # head dimension
CHUNK = 64     # chunk length of the plain chunked form
EPS = 1e-6
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one short prompt on few heads: the smallest prefill, where launches count
        dict(name="fwd b1 t192 h2", op="gdr_fwd", B=1, T=192, Hq=2, Hv=2, N=0, beta="f32", h0=False),
        # a training or prefill batch that fills the GPU
        dict(name="fwd b2 t8192 h64", op="gdr_fwd", B=2, T=8192, Hq=64, Hv=64, N=0, beta="f32", h0=True),
        # ragged prompts packed into one row, grouped values, as a server prefills them
        dict(name="fwd packed 16384 h16/64", op="gdr_fwd", B=1, T=16384, Hq=16, Hv=64, N=11, beta="bf16", h0=True),
        # one request being answered: latency
        dict(name="decode n1 h16/64", op="gdr_decode", n=1, Hq=16, Hv=64, slots=4, skipped=0, beta="f32"),
        # a full server batch, some rows of the captured batch unused
        dict(name="decode n256 h64", op="gdr_decode", n=256, Hq=64, Hv=64, slots=272, skipped=5, beta="bf16"),
        # a small training step with a partial last chunk and grouped values
        dict(name="bwd b1 t1000 h4/8", op="gdr_bwd", B=1, T=1000, Hq=4, Hv=8, N=0, beta="f32", h0=True),
        # a training step that fills the GPU
        dict(name="bwd b2 t8192 h64", op="gdr_bwd", B=2, T=8192, Hq=64, Hv=64, N=0, beta="f32", h0=False),
        # documents of many lengths packed into one training row
        dict(name="bwd packed 4096 h16/32", op="gdr_bwd", B=1, T=4096, Hq=16, Hv=32, N=7, beta="bf16", h0=False),
        # queries and keys of a few decoded tokens: latency
        dict(name="norm b4 t1 h16", op="qk_norm", B=4, T=1, Hq=16, Hk=16, mode="rms", weight=True, rot=64, fused=True),
        # queries and keys of the large batch
        dict(name="norm b2 t8192 h64", op="qk_norm", B=2, T=8192, Hq=64, Hk=64, mode="l2", weight=False, rot=0, fused=False),
        # its gradients on an odd short row
        dict(name="norm bwd b1 t77 h8/2", op="qk_norm_bwd", B=1, T=77, Hq=8, Hk=2, mode="l2", weight=False, rot=0, fused=False),
        # its gradients with weights and rotation, read from a fused projection
        dict(name="norm bwd b2 t4096 h64/16", op="qk_norm_bwd", B=2, T=4096, Hq=64, Hk=16, mode="rms", weight=True, rot=128, fused=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gdr_fwd", "gdr_bwd", "gdr_decode", "qk_norm", "qk_norm_bwd"])
    Hq = rng.choice([1, 2, 4, 8, 16, 32])
    if op in ("gdr_fwd", "gdr_bwd"):
        Hv = Hq * rng.choice([1, 1, 2, 4])
        Hv = min(Hv, 64)
        room = min(16384, (1 << 20) // Hv)
        packed = rng.random() < 0.4
        B = 1 if packed else rng.choice([1, 1, 2, 3, 5])
        T = _log(rng, 1 if not packed else 40, room // B)
        N = _log(rng, 1, min(24, T)) if packed else 0
        return dict(op=op, B=B, T=T, Hq=Hq, Hv=Hv, N=N, beta=rng.choice(["f32", "bf16"]), h0=rng.random() < 0.5)
    if op == "gdr_decode":
        Hv = min(64, Hq * rng.choice([1, 2, 4]))
        n = _log(rng, 1, 256)
        skipped = rng.randint(0, n // 4)
        return dict(op=op, n=n, Hq=Hq, Hv=Hv, slots=n + rng.randint(1, 16), skipped=skipped,
                    beta=rng.choice(["f32", "bf16"]))
    Hk = Hq if rng.random() < 0.5 else max(1, Hq // rng.choice([1, 2, 4]))
    B = rng.choice([1, 2, 3])
    weight = rng.random() < 0.5
    return dict(op=op, B=B, T=_log(rng, 1, 8192 // B), Hq=Hq, Hk=Hk, mode=rng.choice(["l2", "rms"]), weight=weight,
                rot=rng.choice([0, 32, 64, 128]), fused=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs


def _lengths(total, n, seed):
    """n sequence lengths that sum to total, uneven as requests are (numpy, from the seed)."""
    r = np.random.RandomState((seed * 7919 + 13) % (1 << 31))
    if n <= 0:
        return [total]
    share = r.gamma(0.7, size=n) + 1e-3
    lens = np.floor(share / share.sum() * (total - n)).astype(np.int64) + 1
    lens[int(np.argmax(lens))] += total - int(lens.sum())
    return [int(x) for x in lens]


def _delta_inputs(lead, Hq, Hv, beta, gen):
    """q, k (unit rows), v in bf16; the log-decay of a head from a rate and a softplus step; beta a sigmoid."""
    dev = "cuda"
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(BF16)  # noqa: E731
    q = unit(torch.randn(*lead, Hq, D, generator=gen, device=dev))
    k = unit(torch.randn(*lead, Hq, D, generator=gen, device=dev))
    v = torch.randn(*lead, Hv, D, generator=gen, device=dev).to(BF16)
    rate = torch.exp(torch.rand(Hv, generator=gen, device=dev) * math.log(16.0))
    step = torch.exp(torch.rand(Hv, generator=gen, device=dev) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    bias = step + torch.log(-torch.expm1(-step))
    g = -rate * torch.nn.functional.softplus(torch.randn(*lead, Hv, generator=gen, device=dev) + bias)
    b = torch.sigmoid(torch.randn(*lead, Hv, generator=gen, device=dev)).to(BF16 if beta == "bf16" else F32)
    return dict(q=q, k=k, v=v, g=g, beta=b)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    op = case["op"]
    if op in ("gdr_fwd", "gdr_bwd"):
        s = _delta_inputs((case["B"], case["T"]), case["Hq"], case["Hv"], case["beta"], gen)
        lens = _lengths(case["T"], case["N"], int(seed)) if case["N"] else [case["T"]] * case["B"]
        n = len(lens)
        s["lens"] = lens
        s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda") if case["N"] else None
        s["h0"] = torch.randn(n, case["Hv"], D, D, generator=gen, device="cuda") * 0.1 if case["h0"] else None
        if op == "gdr_bwd":
            s["do"] = torch.randn(s["v"].shape, generator=gen, device="cuda").to(BF16)
            s["dhT"] = torch.randn(n, case["Hv"], D, D, generator=gen, device="cuda") * 0.1 if case["h0"] else None
    elif op == "gdr_decode":
        n = case["n"]
        s = _delta_inputs((n,), case["Hq"], case["Hv"], case["beta"], gen)
        r = np.random.RandomState((int(seed) * 31 + 5) % (1 << 31))
        idx = 1 + r.permutation(case["slots"] - 1)[:n] if case["slots"] > n else 1 + r.permutation(n)
        idx[r.permutation(n)[:case["skipped"]]] = -1
        s["idx"] = torch.tensor(idx, dtype=torch.int32, device="cuda")
        s["pool"] = torch.randn(max(case["slots"], n + 1), case["Hv"], D, D, generator=gen, device="cuda") * 0.1
        s["out"] = torch.zeros(n, case["Hv"], D, dtype=BF16, device="cuda")
    else:
        B, T, Hq, Hk = (case[x] for x in ("B", "T", "Hq", "Hk"))
        if case["fused"]:   # rows of one projection that also holds the values
            x = torch.randn(B, T, (Hq + 2 * Hk) * D, generator=gen, device="cuda").to(BF16)
            q, k = x[..., :Hq * D].view(B, T, Hq, D), x[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D)
        else:
            q = torch.randn(B, T, Hq, D, generator=gen, device="cuda").to(BF16)
            k = torch.randn(B, T, Hk, D, generator=gen, device="cuda").to(BF16)
        s = dict(q=q, k=k, wq=None, wk=None, cos=None, sin=None, pos=None, mode=case["mode"])
        if case["weight"]:
            s["wq"] = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
            s["wk"] = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        if case["rot"]:
            P = T + 64
            inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=F64) / case["rot"])
            ang = torch.arange(P, device="cuda", dtype=F64)[:, None] * inv
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            s["pos"] = (torch.arange(T, device="cuda")[None] + torch.randint(0, 64, (B, 1), generator=gen, device="cuda")).to(torch.int32)
        if op == "qk_norm_bwd":
            s["dq"] = torch.randn(B, T, Hq, D, generator=gen, device="cuda").to(BF16)
            s["dk"] = torch.randn(B, T, Hk, D, generator=gen, device="cuda").to(BF16)
    s["op"], s["scale"] = op, D ** -0.5
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gated_delta_rule_35_amd as kda
    op = s["op"]
    if op == "gdr_fwd":
        return kda.kda_gdr_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], cu_seqlens=s["cu"],
                               initial_state=s["h0"], final_state=True)
    if op == "gdr_bwd":
        d = kda.kda_gdr_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["do"], initial_state=s["h0"],
                            d_final_state=s["dhT"], d_initial_state=s["h0"] is not None, cu_seqlens=s["cu"])
        return d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], d["dh0"]
    if op == "gdr_decode":
        return kda.kda_gdr_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["pool"],
                                  state_indices=s["idx"], out=s["out"])
    if op == "qk_norm":
        return kda.kda_qk_norm(s["q"], s["k"], q_weight=s["wq"], k_weight=s["wk"], mode=s["mode"], eps=EPS,
                               cos=s["cos"], sin=s["sin"], positions=s["pos"])
    d = kda.kda_qk_norm_bwd(s["q"], s["k"], s["dq"], s["dk"], q_weight=s["wq"], k_weight=s["wk"], mode=s["mode"],
                            eps=EPS, cos=s["cos"], sin=s["sin"], positions=s["pos"])
    return d["dq"], d["dk"], d["dq_weight"], d["dk_weight"]


def _run_plain(s):
    op = s["op"]
    if op == "gdr_fwd":
        o, hT = _chunked(s, s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["beta"].float(), s["h0"])
        return o.to(BF16), hT
    if op == "gdr_bwd":
        x = [s[n].float().detach().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
        h0 = s["h0"].detach().requires_grad_() if s["h0"] is not None else None
        o, hT = _chunked(s, *x, h0)
        outs, grads = [o], [s["do"].float()]
        if s["dhT"] is not None:
            outs, grads = outs + [hT], grads + [s["dhT"]]
        d = torch.autograd.grad(outs, x + ([h0] if h0 is not None else []), grads)
        return d[0].to(BF16), d[1].to(BF16), d[2].to(BF16), d[3], d[4], d[5] if h0 is not None else None
    if op == "gdr_decode":
        return _decode(s)
    return _norm(s) if op == "qk_norm" else _norm_bwd(s)


# ------------------------------------------------------------------ plain forms


def _chunked(s, q, k, v, g, beta, h0):
    """The chunked gated delta rule: within a chunk, with G the running sum of g and M the strictly lower part of
    beta_i (k_i . k_j) e^{G_i - G_j},
        u = (I + M)^{-1} beta (v - e^G K S),   o = scale (e^G Q S + (QK^T e^{G_i - G_j}, j <= i) u),
        S' = e^{G_last} S + K^T (e^{G_last - G} u).
    Sequences are cut into chunks from their own start; the last one is filled up with tokens that change nothing.
    The chunks of all sequences are walked side by side, longest sequences first."""
    dev, lens = q.device, s["lens"]
    Hv, R = v.shape[2], v.shape[2] // q.shape[2]
    flat = lambda x: x.reshape(-1, *x.shape[2:])  # noqa: E731
    q, k, v, g, beta = flat(q), flat(k), flat(v), flat(g), flat(beta)
    order = sorted(range(len(lens)), key=lambda n: -lens[n])
    starts = np.concatenate([[0], np.cumsum(lens)])
    count = np.array([-(-lens[n] // CHUNK) for n in order])
    steps = [int((count > c).sum()) for c in range(int(count.max()))]      # sequences that still have a chunk c
    rows = np.concatenate([(starts[order[:m]][:, None] + c * CHUNK + np.arange(CHUNK)) for c, m in enumerate(steps)])
    ends = np.concatenate([starts[1:][order[:m]] for m in steps])
    real = torch.from_numpy(rows < ends[:, None]).to(dev)                   # [slots, 64]
    rows = torch.from_numpy(np.minimum(rows, ends[:, None] - 1)).to(dev)
    take = lambda x: (x[rows] * real.view(*real.shape, *([1] * (x.dim() - 1)))).transpose(1, 2)  # noqa: E731
    q, k = take(q).repeat_interleave(R, dim=1), take(k).repeat_interleave(R, dim=1)   # [slots, Hv, 64, 128]
    v, g, beta = take(v), take(g), take(beta).unsqueeze(-1)
    G = g.to(F64).cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    decay = torch.exp((G.unsqueeze(-1) - G.unsqueeze(-2)).masked_fill(~lower, -math.inf)).float()
    eG, eR, eL = G.exp().float().unsqueeze(-1), (G[..., -1:] - G).exp().float().unsqueeze(-1), G[..., -1].exp().float()
    kT = k.transpose(-1, -2)
    M = beta * (k @ kT) * decay * (~torch.eye(CHUNK, dtype=torch.bool, device=dev))
    A = s["scale"] * (q @ kT) * decay
    Tm, P = torch.eye(CHUNK, device=dev) - M, M @ M                        # (I - M)(I + M^2)(I + M^4) ...
    for i in range(5):
        Tm = Tm + Tm @ P
        P = P @ P if i < 4 else P
    S = torch.zeros(len(lens), Hv, D, D, device=dev) if h0 is None else h0[order]
    outs, done, at = [], [], 0
    for m in steps:
        S, gone = S[:m], S[m:]
        done.append(gone)
        i = slice(at, at + m)
        at += m
        u = Tm[i] @ (beta[i] * (v[i] - eG[i] * (k[i] @ S)))
        outs.append(s["scale"] * eG[i] * (q[i] @ S) + A[i] @ u)
        S = eL[i][..., None, None] * S + kT[i] @ (eR[i] * u)
    done.append(S)
    o = torch.cat(outs).transpose(1, 2)[real]                                # tokens in slot order
    back = torch.argsort(rows[real])
    hT = torch.cat(done[::-1])[np.argsort(order)]                            # longest first, back to the given order
    return o[back].view(s["v"].shape), hT


def _decode(s):
    Hv, R = s["v"].shape[1], s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(R, dim=1) for n in ("q", "k"))
    live = s["idx"] >= 0
    at = s["idx"].clamp(min=0).long()
    S = s["pool"][at]
    Sd = torch.exp(s["g"])[..., None, None] * S
    u = s["beta"].float()[..., None] * (s["v"].float() - (k.unsqueeze(-1) * Sd).sum(-2))
    new = Sd + k.unsqueeze(-1) * u.unsqueeze(-2)
    o = s["scale"] * (q.unsqueeze(-1) * new).sum(-2)
    s["out"].copy_(torch.where(live[:, None, None], o.to(BF16), s["out"]))
    s["pool"][at] = torch.where(live[:, None, None, None], new, S)           # unused rows rewrite the spare slot 0
    return s["out"], s["pool"]


def _turn(x, s, back=False):
    """The first rot channels of x rotated by their position: pairs (i, i + rot / 2)."""
    if s["cos"] is None:
        return x
    c, n = s["cos"][s["pos"].long()].unsqueeze(2).to(x.dtype), s["sin"][s["pos"].long()].unsqueeze(2).to(x.dtype)
    n = -n if back else n
    h = c.shape[-1]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat([a * c - b * n, b * c + a * n, x[..., 2 * h:]], dim=-1)


def _inverse_norm(x, s):
    ss = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((ss / D if s["mode"] == "rms" else ss) + EPS)


def _norm(s):
    y = []
    for x, w in ((s["q"].float(), s["wq"]), (s["k"].float(), s["wk"])):
        y.append(_turn(x * _inverse_norm(x, s) * (1.0 if w is None else w), s).to(BF16))
    return y


def _norm_bwd(s):
    dx, dw = [], []
    for x, w, dy in ((s["q"].float(), s["wq"], s["dq"]), (s["k"].float(), s["wk"], s["dk"])):
        r = _inverse_norm(x, s)
        dz = _turn(dy.float(), s, back=True)
        dw.append(None if w is None else (dz * x * r).sum((0, 1, 2)))
        dz = dz if w is None else dz * w
        m = (dz * x).sum(-1, keepdim=True) * r * r / (D if s["mode"] == "rms" else 1)
        dx.append((r * (dz - x * m)).to(BF16))
    return dx[0], dx[1], dw[0], dw[1]


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op, d2 = case["op"], D * D
    if op in ("gdr_fwd", "gdr_bwd"):
        n, Hq, Hv = case["B"] * case["T"], case["Hq"], case["Hv"]
        seqs = case["N"] or case["B"]
        bt = 2 if case["beta"] == "bf16" else 4
        ins = n * (4 * Hq * D + 2 * Hv * D + 4 * Hv + bt * Hv)
        state = 4 * seqs * Hv * d2
        if op == "gdr_fwd":   # three products with the state a token: k S, k u^T, q S
            return dict(bytes=ins + 2 * n * Hv * D + state * (2 if case["h0"] else 1), flops=6.0 * d2 * n * Hv)
        # the state's two again, then do S, dS k, dS u, S du, q do^T, k du^T
        return dict(bytes=ins + 2 * n * Hv * D + n * (4 * Hq * D + 2 * Hv * D + 8 * Hv) + state * (3 if case["h0"] else 0),
                    flops=16.0 * d2 * n * Hv)
    if op == "gdr_decode":
        n, live, Hq, Hv = case["n"], case["n"] - case["skipped"], case["Hq"], case["Hv"]
        bt = 2 if case["beta"] == "bf16" else 4
        return dict(bytes=live * (8 * Hv * d2 + 4 * Hq * D + 4 * Hv * D + 4 * Hv + bt * Hv) + 4 * n, flops=6.0 * d2 * live * Hv)
    n, rows = case["B"] * case["T"], case["B"] * case["T"] * (case["Hq"] + case["Hk"])
    extra = 4 * n + 4 * n * case["rot"] if case["rot"] else 0
    return dict(bytes=rows * D * 2 * (2 if op == "qk_norm" else 3) + extra + (1024 if case["weight"] else 0),
                flops=rows * D * (8.0 if op == "qk_norm" else 16.0))


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gdr_fwd", "gdr_bwd"):
        return _exact_delta(s, op == "gdr_bwd")
    if op == "gdr_decode":
        out, pool = s["out"].to(F64), s["pool"].to(F64)
        R = s["v"].shape[1] // s["q"].shape[1]
        for n, slot in enumerate(s["idx"].tolist()):
            if slot >= 0:
                q, k = (s[x][n].to(F64).repeat_interleave(R, dim=0) for x in ("q", "k"))
                out[n] = _step(pool[slot], q, k, s["v"][n].to(F64), s["g"][n].to(F64), s["beta"][n].to(F64), s["scale"])
        return out, pool
    return _exact_norm(s, op == "qk_norm_bwd")


def _step(S, q, k, v, g, beta, scale):
    """One token of the recurrence, S [.., 128, 128] updated in place; returns o."""
    S *= torch.exp(g)[..., None, None]
    u = beta[..., None] * (v - torch.matmul(k.unsqueeze(-2), S).squeeze(-2))
    S += k.unsqueeze(-1) * u.unsqueeze(-2)
    return scale * torch.matmul(q.unsqueeze(-2), S).squeeze(-2)


def _exact_delta(s, backward):
    """Token by token.  The gradients walk back over each stretch of 64 tokens with its states recomputed."""
    R, Hv = s["v"].shape[2] // s["q"].shape[2], s["v"].shape[2]
    if s["cu"] is None:
        parts = [(slice(0, s["q"].shape[0]), slice(0, s["q"].shape[1]), slice(0, s["q"].shape[0]))]
    else:
        c = s["cu"].tolist()
        parts = [(slice(0, 1), slice(a, b), slice(n, n + 1)) for n, (a, b) in enumerate(zip(c, c[1:]))]
    new = lambda x: torch.zeros(x.shape, dtype=F64, device=x.device)  # noqa: E731
    o, hT = new(s["v"]), torch.zeros(len(s["lens"]), Hv, D, D, dtype=F64, device="cuda")
    d = dict(q=new(s["q"]), k=new(s["k"]), v=new(s["v"]), g=new(s["g"]), beta=new(s["beta"]), h=hT.clone()) if backward else None
    for rows, span, seqs in parts:
        q, k, v, g, beta = (s[n][rows, span] for n in ("q", "k", "v", "g", "beta"))
        at = lambda x, t: x[:, t].to(F64)  # noqa: E731
        wide = lambda x, t: x[:, t].to(F64).repeat_interleave(R, dim=1)  # noqa: E731
        length = q.shape[1]
        S = hT[seqs] if s["h0"] is None else s["h0"][seqs].to(F64)
        kept = []
        for t in range(length):
            if backward and t % 64 == 0:
                kept.append(S.clone())
            o[rows, span.start + t] = _step(S, wide(q, t), wide(k, t), at(v, t), at(g, t), at(beta, t), s["scale"])
        hT[seqs] = S
        if not backward:
            continue
        do = s["do"][rows, span]
        dS = torch.zeros_like(S) if s["dhT"] is None else s["dhT"][seqs].to(F64)
        for c in range(len(kept) - 1, -1, -1):
            S, states = kept.pop(), []
            ts = range(64 * c, min(64 * c + 64, length))
            for t in ts:
                states.append(S.clone())
                _step(S, wide(q, t), wide(k, t), at(v, t), at(g, t), at(beta, t), s["scale"])
            for t in reversed(ts):
                qt, kt, vt, bt, dot = wide(q, t), wide(k, t), at(v, t), at(beta, t)[..., None], at(do, t)
                eg = torch.exp(at(g, t))[..., None, None]
                Sd = states.pop() * eg
                e = vt - torch.matmul(kt.unsqueeze(-2), Sd).squeeze(-2)
                u = bt * e
                S = Sd + kt.unsqueeze(-1) * u.unsqueeze(-2)
                dS = dS + s["scale"] * qt.unsqueeze(-1) * dot.unsqueeze(-2)
                dq = s["scale"] * torch.matmul(S, dot.unsqueeze(-1)).squeeze(-1)
                du = torch.matmul(kt.unsqueeze(-2), dS).squeeze(-2)
                dk = torch.matmul(dS, u.unsqueeze(-1)).squeeze(-1) - bt * torch.matmul(Sd, du.unsqueeze(-1)).squeeze(-1)
                dS = dS - kt.unsqueeze(-1) * (bt * du).unsqueeze(-2)
                tt = span.start + t
                d["q"][rows, tt] = dq.unflatten(1, (-1, R)).sum(2)
                d["k"][rows, tt] = dk.unflatten(1, (-1, R)).sum(2)
                d["v"][rows, tt], d["beta"][rows, tt] = bt * du, (du * e).sum(-1)
                d["g"][rows, tt] = (Sd * dS).sum((-1, -2))
                dS = dS * eg
        d["h"][seqs] = dS
    if backward:
        return d["q"], d["k"], d["v"], d["g"], d["beta"], d["h"] if s["h0"] is not None else None
    return o, hT


def _exact_norm(s, backward):
    """Row by row in the definition's order; the gradients by autograd of it."""
    found, weights = [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x = x.to(F64).requires_grad_(backward)
        w = None if w is None else w.to(F64).requires_grad_(backward)
        n2 = x.pow(2).mean(-1) if s["mode"] == "rms" else x.pow(2).sum(-1)
        y = x / torch.sqrt(n2 + EPS)[..., None]
        y = y if w is None else y * w
        if s["cos"] is not None:
            ang = torch.complex(s["cos"].to(F64), s["sin"].to(F64))[s["pos"].long()][:, :, None]
            h = ang.shape[-1]
            z = torch.complex(y[..., :h], y[..., h:2 * h]) * ang
            y = torch.cat([z.real, z.imag, y[..., 2 * h:]], dim=-1)
        if not backward:
            found.append(y)
            continue
        leaves = [x] if w is None else [x, w]
        got = torch.autograd.grad(y, leaves, dy.to(F64))
        found.append(got[0])
        weights.append(got[1] if w is not None else None)
    return found + weights
