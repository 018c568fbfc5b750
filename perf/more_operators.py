"""Measured cases of the short causal convolution, the selective state space scan, and the norms around a block.

Operators (`case["op"]`):

  conv            y_t = act(bias + sum_i w_i x_{t-W+1+i}) per channel, over each sequence, the W - 1 inputs before it
                  in an initial state; the last W - 1 inputs are the final state
  conv_bwd        its gradients with respect to x, the weights, the bias and the initial state
  conv_decode     one token per row, the last inputs in a pool that a slot map indexes
  ssm             S_t = e^{d_t A} S_{t-1} + d_t B_t x_t^T, y_t = S_t^T C_t + D x_t, with d_t = softplus(dt_t + dt_bias) and
                  A one number per head, B and C shared by the heads of a group
  ssm_bwd         its gradients with respect to x, dt, A, B, C, D, dt_bias and the initial state
  ssm_decode      one token per row, the states in a pool that a slot map indexes
  gated_norm      y = norm(x) w act(gate), or norm(x act(gate)) w: the norm after a block, with the block's gate
  gated_norm_bwd  its gradients with respect to x, the gate and the weight
  add_norm        h = residual + scale x, y = norm(h) w: a block's residual and scale, and the norm before the next block
  add_norm_bwd    its gradients with respect to x, the residual and the weight

`own` False: the plain forms below, in torch operations on 32 bits (log-decays summed in 64).  `own` True: the
framework's entry points on the same inputs.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64     # chunk length of the plain scan
EPS = 1e-6
F32, F64 = torch.float32, torch.float64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # queries, keys and values of one request's next token, on the way to the delta rule: latency
        dict(name="conv decode n1 c12288", op="conv_decode", n=1, C=12288, W=4, type="bf16", act="silu", bias=False, slots=4,
             skipped=0),
        # ragged prompts packed into one row, queries, keys and values of 16 and 64 heads, continued from states
        dict(name="conv packed 16384 c12288", op="conv", B=1, T=16384, C=12288, W=4, N=11, type="bf16", act="silu",
             bias=False, state=True, fused=False),
        # a training step's x, B and C of 64 heads, read from the rows of a projection
        dict(name="conv bwd b2 t4096 c4352", op="conv_bwd", B=2, T=4096, C=4352, W=4, N=0, type="bf16", act="silu",
             bias=True, state=False, fused=True),
        # a full server batch, some rows of the captured batch unused
        dict(name="ssm decode n256 h64", op="ssm_decode", n=256, H=64, P=64, S=128, G=1, slots=272, skipped=5, dt="bf16"),
        # one short prompt on few heads: the smallest prefill, where launches count
        dict(name="ssm b1 t195 h8", op="ssm", B=1, T=195, H=8, P=64, S=128, G=1, N=0, dt="bf16", h0=False, fused=True),
        # a training or prefill batch that fills the GPU
        dict(name="ssm b2 t8192 h64", op="ssm", B=2, T=8192, H=64, P=64, S=128, G=1, N=0, dt="bf16", h0=True, fused=False),
        # documents of many lengths packed into one training row, wide heads in groups
        dict(name="ssm bwd packed 4096 h32", op="ssm_bwd", B=1, T=4096, H=32, P=128, S=128, G=8, N=7, dt="f32", h0=True,
             fused=True),
        # a training step that fills the GPU
        dict(name="ssm bwd b2 t8192 h64", op="ssm_bwd", B=2, T=8192, H=64, P=64, S=128, G=1, N=0, dt="bf16", h0=False,
             fused=True),
        # the delta rule's heads on their way out, the gate a slice of a projection
        dict(name="gated norm b2 t8192 h64", op="gated_norm", B=2, T=8192, H=64, D=128, type="bf16", act="sigmoid",
             first=False, weight="shared", fused=True),
        # the gradients of the scan's norm, all channels of a token together, on an odd row
        dict(name="gated norm bwd b1 t3001 d4096", op="gated_norm_bwd", B=1, T=3001, H=1, D=4096, type="bf16", act="silu",
             first=True, weight="shared", fused=True),
        # a few decoded tokens between two blocks: latency
        dict(name="add norm b4 t1 d4096", op="add_norm", B=4, T=1, D=4096, type="bf16", res="bf16", scale=1.0),
        # a training step's residual stream in 32 bits, blocks scaled down
        dict(name="add norm bwd b2 t8192 d4096", op="add_norm_bwd", B=2, T=8192, D=4096, type="bf16", res="f32", scale=0.25),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["conv", "conv", "ssm", "ssm", "ssm", "gated_norm", "add_norm"])
    bwd = rng.random() < 0.5
    packed = rng.random() < 0.4
    B = 1 if packed else rng.choice([1, 1, 2, 3, 5])
    kinds = ["bf16", "bf16", "f16", "f32"]
    if kind == "conv":
        if rng.random() < 0.25:
            n = _log(rng, 1, 256)
            return dict(op="conv_decode", n=n, C=8 * _log(rng, 1, 1536), W=rng.choice([2, 3, 4, 4]), type=rng.choice(kinds),
                        act=rng.choice(["silu", "none"]), bias=rng.random() < 0.5, slots=n + rng.randint(1, 16),
                        skipped=rng.randint(0, n // 4))
        C = 8 * _log(rng, 1, 1536)
        T = _log(rng, 40 if packed else 1, min(16384, (1 << 26) // C) // B)
        return dict(op="conv_bwd" if bwd else "conv", B=B, T=T, C=C, W=rng.choice([2, 3, 4, 4]),
                    N=_log(rng, 1, min(24, T)) if packed else 0, type=rng.choice(kinds), act=rng.choice(["silu", "none"]),
                    bias=rng.random() < 0.5, state=rng.random() < 0.5, fused=rng.random() < 0.5)
    if kind == "ssm":
        G = rng.choice([1, 1, 2, 4, 8])
        H = min(64, G * rng.choice([1, 2, 3, 4, 8, 16, 64]))
        H -= H % G
        P, S = rng.choice([64, 64, 128]), rng.choice([64, 128, 128])
        if rng.random() < 0.25:
            n = _log(rng, 1, 256 if P == 64 else 128)
            return dict(op="ssm_decode", n=n, H=H, P=P, S=S, G=G, slots=n + rng.randint(1, 16), skipped=rng.randint(0, n // 4),
                        dt=rng.choice(["bf16", "f32"]))
        T = _log(rng, 40 if packed else 1, min(16384, (1 << 26) // (H * P)) // B)
        return dict(op="ssm_bwd" if bwd else "ssm", B=B, T=T, H=H, P=P, S=S, G=G, N=_log(rng, 1, min(24, T)) if packed else 0,
                    dt=rng.choice(["bf16", "f32"]), h0=rng.random() < 0.5, fused=rng.random() < 0.5)
    B = rng.choice([1, 2, 3])
    if kind == "gated_norm":
        H, D = (rng.choice([1, 2, 8, 24, 64]), 8 * rng.choice([8, 16, 16, 24])) if rng.random() < 0.6 else \
            (rng.choice([1, 1, 2, 8]), 8 * _log(rng, 1, 1024))
        T = _log(rng, 1, min(8192, (1 << 26) // (H * D)) // B)
        return dict(op="gated_norm_bwd" if bwd else "gated_norm", B=B, T=T, H=H, D=D, type=rng.choice(kinds),
                    act=rng.choice(["silu", "sigmoid"]), first=rng.random() < 0.4,
                    weight=rng.choice(["shared", "heads", "none"]), fused=rng.random() < 0.5)
    D = 8 * _log(rng, 8, 1024)
    t = rng.choice(kinds)
    return dict(op="add_norm_bwd" if bwd else "add_norm", B=B, T=_log(rng, 1, min(8192, (1 << 26) // D) // B), D=D, type=t,
                res=rng.choice([t, "f32"]), scale=rng.choice([1.0, 0.5, 0.22]))


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


def _sequences(s, case, seed):
    lens = _lengths(case["T"], case["N"], int(seed)) if case["N"] else [case["T"]] * case["B"]
    s["lens"] = lens
    s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda") if case["N"] else None
    return len(lens)


def _slots(s, case, seed):
    """A slot map: rows of the batch in slots 1 .. of a pool, `skipped` of them unused (-1); slot 0 is spare."""
    n = case["n"]
    r = np.random.RandomState((int(seed) * 31 + 5) % (1 << 31))
    idx = 1 + r.permutation(case["slots"] - 1)[:n] if case["slots"] > n else 1 + r.permutation(n)
    idx[r.permutation(n)[:case["skipped"]]] = -1
    s["idx"] = torch.tensor(idx, dtype=torch.int32, device="cuda")
    return max(case["slots"], n + 1)


def _ssm_inputs(s, lead, case, rnd, uni):
    """x, B and C as a convolution leaves them (one row a token where they are fused); dt about a step between
    0.001 and 0.1 for each head, A -1 .. -16."""
    H, P, S, G, bf = case["H"], case["P"], case["S"], case["G"], torch.bfloat16
    if case.get("fused"):
        row = rnd(*lead, H * P + 2 * G * S).to(bf)
        s["x"] = row[..., :H * P].unflatten(-1, (H, P))
        s["Bm"] = row[..., H * P:H * P + G * S].unflatten(-1, (G, S))
        s["Cm"] = row[..., H * P + G * S:].unflatten(-1, (G, S))
    else:
        s["x"], s["Bm"], s["Cm"] = rnd(*lead, H, P).to(bf), rnd(*lead, G, S).to(bf), rnd(*lead, G, S).to(bf)
    s["dt"] = rnd(*lead, H).to(TYPES[case["dt"]])
    step = torch.exp(uni(H) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -(1 + 15 * uni(H))
    s["D"] = 1 + 0.1 * rnd(H)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    rnd = lambda *z: torch.randn(*z, generator=gen, device="cuda")  # noqa: E731
    uni = lambda *z: torch.rand(*z, generator=gen, device="cuda")  # noqa: E731
    op, s = case["op"], {}
    t = TYPES[case["type"]] if "type" in case else None
    if op in ("conv", "conv_bwd"):
        B, T, C, W = (case[n] for n in ("B", "T", "C", "W"))
        n = _sequences(s, case, seed)
        s["x"] = rnd(B, T, C + 64).to(t)[..., :C] if case["fused"] else rnd(B, T, C).to(t)
        s["w"] = (2 * uni(C, W) - 1) / W ** 0.5
        s["bias"] = 0.1 * rnd(C) if case["bias"] else None
        s["state"] = rnd(n, W - 1, C).to(t) if case["state"] else None
        s["act"] = None if case["act"] == "none" else case["act"]
        if op == "conv_bwd":
            s["dy"] = rnd(B, T, C).to(t)
            s["dlast"] = rnd(n, W - 1, C).to(t) if case["state"] else None
    elif op == "conv_decode":
        n, C, W = case["n"], case["C"], case["W"]
        s["x"], s["w"] = rnd(n, C).to(t), (2 * uni(C, W) - 1) / W ** 0.5
        s["bias"] = 0.1 * rnd(C) if case["bias"] else None
        s["pool"] = rnd(_slots(s, case, seed), W - 1, C).to(t)
        s["out"] = torch.zeros(n, C, dtype=t, device="cuda")
        s["act"] = None if case["act"] == "none" else case["act"]
    elif op in ("ssm", "ssm_bwd"):
        n = _sequences(s, case, seed)
        _ssm_inputs(s, (case["B"], case["T"]), case, rnd, uni)
        s["h0"] = 0.1 * rnd(n, case["H"], case["S"], case["P"]) if case["h0"] else None
        if op == "ssm_bwd":
            s["dy"] = rnd(*s["x"].shape).to(torch.bfloat16)
            s["dlast"] = 0.1 * rnd(n, case["H"], case["S"], case["P"]) if case["h0"] else None
    elif op == "ssm_decode":
        _ssm_inputs(s, (case["n"],), case, rnd, uni)
        s["pool"] = 0.1 * rnd(_slots(s, case, seed), case["H"], case["S"], case["P"])
        s["out"] = torch.zeros(case["n"], case["H"], case["P"], dtype=torch.bfloat16, device="cuda")
    elif op in ("gated_norm", "gated_norm_bwd"):
        B, T, H, D = (case[n] for n in ("B", "T", "H", "D"))
        s["x"] = rnd(B, T, H, D).to(t)
        s["gate"] = rnd(B, T, 2 * H * D).to(t)[..., H * D:].unflatten(-1, (H, D)) if case["fused"] else rnd(B, T, H, D).to(t)
        w = case["weight"]
        s["w"] = None if w == "none" else 1 + 0.1 * (rnd(H, D) if w == "heads" else rnd(D))
        s["act"], s["first"] = case["act"], case["first"]
        if op == "gated_norm_bwd":
            s["dy"] = rnd(B, T, H, D).to(t)
    else:
        B, T, D, r = case["B"], case["T"], case["D"], TYPES[case["res"]]
        s["scale"], s["w"] = case["scale"], 1 + 0.1 * rnd(D)
        s["x"], s["res"] = rnd(B, T, D).to(t), (2 * rnd(B, T, D)).to(r)
        if op == "add_norm_bwd":   # the sum as the forward left it, and what reaches it from later blocks
            s["h"] = (s["res"].float() + s["scale"] * s["x"].float()).to(r)
            s["dy"], s["dh"] = rnd(B, T, D).to(t), rnd(B, T, D).to(r)
    s["op"] = op
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gated_delta_rule_35_amd as kda
    op = s["op"]
    if op == "conv":
        return kda.kda_conv(s["x"], s["w"], s["bias"], activation=s["act"], cu_seqlens=s["cu"], initial_state=s["state"],
                            final_state=True)
    if op == "conv_bwd":
        d = kda.kda_conv_bwd(s["x"], s["w"], s["dy"], s["bias"], activation=s["act"], cu_seqlens=s["cu"],
                             initial_state=s["state"], d_final_state=s["dlast"], d_initial_state=s["state"] is not None)
        return d["dx"], d["dweight"], d["dbias"], d["dstate"]
    if op == "conv_decode":
        return kda.kda_conv_decode(s["x"], s["w"], s["pool"], s["bias"], activation=s["act"], state_indices=s["idx"],
                                   out=s["out"])
    if op == "ssm":
        return kda.kda_ssm_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], dt_bias=s["dt_bias"], cu_seqlens=s["cu"],
                               initial_state=s["h0"], final_state=True)
    if op == "ssm_bwd":
        d = kda.kda_ssm_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], D=s["D"], dt_bias=s["dt_bias"],
                            cu_seqlens=s["cu"], initial_state=s["h0"], d_final_state=s["dlast"],
                            d_initial_state=s["h0"] is not None)
        return tuple(d[n] for n in ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"))
    if op == "ssm_decode":
        return kda.kda_ssm_decode(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["pool"], D=s["D"], dt_bias=s["dt_bias"],
                                  state_indices=s["idx"], out=s["out"])
    if op == "gated_norm":
        return kda.kda_gated_norm(s["x"], s["gate"], s["w"], activation=s["act"], gate_first=s["first"], eps=EPS)
    if op == "gated_norm_bwd":
        d = kda.kda_gated_norm_bwd(s["x"], s["gate"], s["dy"], s["w"], activation=s["act"], gate_first=s["first"], eps=EPS)
        return d["dx"], d["dgate"], d["dweight"]
    if op == "add_norm":
        return kda.kda_add_norm(s["x"], s["res"], s["w"], scale=s["scale"], eps=EPS)
    d = kda.kda_add_norm_bwd(s["h"], s["dy"], s["w"], scale=s["scale"], eps=EPS, d_sum=s["dh"])
    return d["dx"], d["dresidual"], d["dweight"]


def _run_plain(s):
    op = s["op"]
    if op == "conv":
        return _conv(s)[:2]
    if op == "conv_bwd":
        return _conv_bwd(s)
    if op == "conv_decode":
        return _conv_decode(s)
    if op == "ssm":
        d, a = _steps(s["dt"].float(), s["A"], s["dt_bias"])
        y, last = _chunked(s, s["x"].float(), d, a, s["Bm"].float(), s["Cm"].float(), s["D"], s["h0"])
        return y.to(s["x"].dtype), last
    if op == "ssm_bwd":
        return _scan_bwd(s)
    if op == "ssm_decode":
        return _ssm_decode(s)
    return {"gated_norm": _gated, "gated_norm_bwd": _gated_bwd, "add_norm": _add, "add_norm_bwd": _add_bwd}[op](s)


# ------------------------------------------------------------------ plain forms: the convolution


def _taps(s):
    """x with each sequence's W - 1 earlier inputs put before it, [rows, C] in 32 bits, and for each token its row."""
    W, C = s["w"].shape[1], s["x"].shape[-1]
    flat = s["x"].reshape(-1, C).float()
    first = flat.new_zeros(len(s["lens"]), W - 1, C) if s["state"] is None else s["state"].float()
    parts, at, t = [], [], 0
    for n, m in enumerate(s["lens"]):
        parts += [first[n], flat[t:t + m]]
        at.append(np.arange(m) + t + (n + 1) * (W - 1))
        t += m
    return torch.cat(parts), torch.from_numpy(np.concatenate(at)).to(flat.device)


def _act(z, act):
    return z * torch.sigmoid(z) if act == "silu" else torch.sigmoid(z) if act == "sigmoid" else z


def _act_slope(z, act):
    g = torch.sigmoid(z)
    return g * (1 + z * (1 - g)) if act == "silu" else g * (1 - g) if act == "sigmoid" else torch.ones_like(z)


def _conv(s):
    W = s["w"].shape[1]
    rows, at = _taps(s)
    z = sum(s["w"][:, i] * rows[at - (W - 1 - i)] for i in range(W))
    z = z if s["bias"] is None else z + s["bias"]
    ends = torch.from_numpy(np.cumsum([m + W - 1 for m in s["lens"]])).to(at.device)
    last = rows[ends[:, None] + torch.arange(1 - W, 0, device=at.device)]
    return _act(z, s["act"]).to(s["x"].dtype).view(s["x"].shape), last.to(s["x"].dtype), z, rows, at, ends


def _conv_bwd(s):
    W, C = s["w"].shape[1], s["x"].shape[-1]
    _, _, z, rows, at, ends = _conv(s)
    dz = s["dy"].reshape(-1, C).float() * _act_slope(z, s["act"])
    drows = torch.zeros_like(rows)
    if s["dlast"] is not None:
        drows[ends[:, None] + torch.arange(1 - W, 0, device=at.device)] = s["dlast"].float()
    dw = []
    for i in range(W):
        drows[at - (W - 1 - i)] += s["w"][:, i] * dz
        dw.append((dz * rows[at - (W - 1 - i)]).sum(0))
    dstate = None
    if s["state"] is not None:
        starts = ends - torch.tensor(s["lens"], device=at.device) - (W - 1)
        dstate = drows[starts[:, None] + torch.arange(W - 1, device=at.device)].to(s["x"].dtype)
    return (drows[at].to(s["x"].dtype).view(s["x"].shape), torch.stack(dw, dim=1),
            None if s["bias"] is None else dz.sum(0), dstate)


def _conv_decode(s):
    W = s["w"].shape[1]
    live, at = (s["idx"] >= 0)[:, None], s["idx"].clamp(min=0).long()
    rows = torch.cat([s["pool"][at], s["x"].unsqueeze(1)], dim=1)            # [n, W, C]
    z = (rows.float() * s["w"].t()).sum(1)
    z = z if s["bias"] is None else z + s["bias"]
    s["out"].copy_(torch.where(live, _act(z, s["act"]).to(s["out"].dtype), s["out"]))
    s["pool"][at] = torch.where(live[..., None], rows[:, 1:], rows[:, :W - 1])   # unused rows rewrite the spare slot 0
    return s["out"], s["pool"]


# ------------------------------------------------------------------ plain forms: the scan


def _steps(dt, A, bias):
    """The steps d and the log-decays d A."""
    d = torch.nn.functional.softplus(dt + bias)
    return d, d * A


def _chunked(s, x, d, a, Bm, Cm, D, h0):
    """The scan by chunks: with G the running sum of the log-decays a within a chunk,
        y = e^G C S + (C B^T e^{G_i - G_j} d_j, j <= i) x + D x,   S' = e^{G_last} S + B^T (e^{G_last - G} d x).
    Sequences are cut into chunks from their own start; the last one is filled up with tokens that change nothing.
    The chunks of all sequences are walked side by side, longest sequences first."""
    dev, lens, R = x.device, s["lens"], x.shape[2] // Bm.shape[2]
    H, P, S = x.shape[2], x.shape[3], Bm.shape[3]
    order = sorted(range(len(lens)), key=lambda n: -lens[n])
    starts = np.concatenate([[0], np.cumsum(lens)])
    count = np.array([-(-lens[n] // CHUNK) for n in order])
    steps = [int((count > c).sum()) for c in range(int(count.max()))]      # sequences that still have a chunk c
    rows = np.concatenate([(starts[order[:m]][:, None] + c * CHUNK + np.arange(CHUNK)) for c, m in enumerate(steps)])
    ends = np.concatenate([starts[1:][order[:m]] for m in steps])
    real = torch.from_numpy(rows < ends[:, None]).to(dev)                   # [slots, 64]
    rows = torch.from_numpy(np.minimum(rows, ends[:, None] - 1)).to(dev)

    def take(v):
        v = v.reshape(-1, *v.shape[2:])[rows]
        return (v * real.view(*real.shape, *([1] * (v.dim() - 2)))).transpose(1, 2)
    xs, ds, Bs, Cs = take(x), take(d), take(Bm), take(Cm)                   # [slots, H or G, 64, ..]
    G = take(a).to(F64).cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    decay = torch.exp((G.unsqueeze(-1) - G.unsqueeze(-2)).masked_fill(~lower, -math.inf)).float()
    eG, eL = G.exp().float().unsqueeze(-1), G[..., -1].exp().float()
    wx = ((G[..., -1:] - G).exp().float() * ds).unsqueeze(-1) * xs
    CB = (Cs @ Bs.transpose(-1, -2)).repeat_interleave(R, dim=1)
    inner = (CB * decay * ds.unsqueeze(-2)) @ xs
    Bs, Cs = Bs.repeat_interleave(R, dim=1), Cs.repeat_interleave(R, dim=1)
    St = torch.zeros(len(lens), H, S, P, device=dev) if h0 is None else h0[order]
    outs, done, at = [], [], 0
    for m in steps:
        St, gone = St[:m], St[m:]
        done.append(gone)
        i = slice(at, at + m)
        at += m
        outs.append(eG[i] * (Cs[i] @ St))
        St = eL[i][..., None, None] * St + Bs[i].transpose(-1, -2) @ wx[i]
    done.append(St)
    y = (torch.cat(outs) + inner).transpose(1, 2)[real]                      # tokens in slot order
    y = y[torch.argsort(rows[real])].view(x.shape) + D[:, None] * x
    return y, torch.cat(done[::-1])[np.argsort(order)]                       # longest first, back to the given order


def _scan_bwd(s):
    leaf = lambda v: v.float().detach().requires_grad_()  # noqa: E731
    x, dt, A, Bm, Cm, D, bias = (leaf(s[n]) for n in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias"))
    h0 = leaf(s["h0"]) if s["h0"] is not None else None
    d, a = _steps(dt, A, bias)
    y, last = _chunked(s, x, d, a, Bm, Cm, D, h0)
    outs, grads = ([y], [s["dy"].float()]) if s["dlast"] is None else ([y, last], [s["dy"].float(), s["dlast"]])
    g = list(torch.autograd.grad(outs, [x, dt, A, Bm, Cm, D, bias] + ([h0] if h0 is not None else []), grads))
    for i in (0, 3, 4):
        g[i] = g[i].to(s["x"].dtype)
    return tuple(g) if h0 is not None else (*g, None)


def _ssm_decode(s):
    R = s["x"].shape[1] // s["Bm"].shape[1]
    live, at = s["idx"] >= 0, s["idx"].clamp(min=0).long()
    d, a = _steps(s["dt"].float(), s["A"], s["dt_bias"])
    x = s["x"].float()
    Bm, Cm = (s[n].float().repeat_interleave(R, dim=1).unsqueeze(-1) for n in ("Bm", "Cm"))
    old = s["pool"][at]
    new = torch.exp(a)[..., None, None] * old + Bm * (d.unsqueeze(-1) * x).unsqueeze(-2)
    y = (Cm * new).sum(-2) + s["D"][:, None] * x
    s["out"].copy_(torch.where(live[:, None, None], y.to(s["out"].dtype), s["out"]))
    s["pool"][at] = torch.where(live[:, None, None, None], new, old)         # unused rows rewrite the spare slot 0
    return s["out"], s["pool"]


# ------------------------------------------------------------------ plain forms: the norms


def _gated(s):
    x, g = s["x"].float(), _act(s["gate"].float(), s["act"])
    x = x * g if s["first"] else x
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    y = y if s["w"] is None else y * s["w"]
    return (y if s["first"] else y * g).to(s["x"].dtype)


def _gated_bwd(s):
    x, z, dy, w = s["x"].float(), s["gate"].float(), s["dy"].float(), s["w"]
    g = _act(z, s["act"])
    v = x * g if s["first"] else x
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    dn = dy if s["first"] else dy * g                                        # gradient of norm(v) w
    dw = None if w is None else (dn * v * r).sum((0, 1) if w.dim() == 2 else (0, 1, 2))
    dg = None if s["first"] else dy * (v * r) * (1.0 if w is None else w)
    dn = dn if w is None else dn * w
    dv = r * (dn - v * ((dn * v).mean(-1, keepdim=True) * r * r))
    dx, dg = (dv * g, dv * x) if s["first"] else (dv, dg)
    return dx.to(s["x"].dtype), (dg * _act_slope(z, s["act"])).to(s["x"].dtype), dw


def _add(s):
    h = s["res"].float() + s["scale"] * s["x"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
    return y.to(s["x"].dtype), h.to(s["res"].dtype)


def _add_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    dn = dy * s["w"]
    dh = s["dh"].float() + r * (dn - h * ((dn * h).mean(-1, keepdim=True) * r * r))
    return (s["scale"] * dh).to(s["dy"].dtype), dh.to(s["h"].dtype), (dy * h * r).sum((0, 1))


# ------------------------------------------------------------------ what a pass cannot do without


def _size(t):
    return 4 if t == "f32" else 2


def work(case):
    op = case["op"]
    if op in ("conv", "conv_bwd"):
        n, C, W, z = case["B"] * case["T"], case["C"], case["W"], _size(case["type"])
        states = (case["N"] or case["B"]) * (W - 1) * C * z
        par = 4 * C * (W + int(case["bias"]))
        if op == "conv":
            return dict(bytes=2 * n * C * z + states * (2 if case["state"] else 1) + par, flops=(2.0 * W + 6) * n * C)
        return dict(bytes=3 * n * C * z + states * (3 if case["state"] else 0) + 2 * par, flops=(6.0 * W + 12) * n * C)
    if op == "conv_decode":
        live, C, W, z = case["n"] - case["skipped"], case["C"], case["W"], _size(case["type"])
        return dict(bytes=2 * live * C * z * W + 4 * C * (W + int(case["bias"])) + 4 * case["n"], flops=(2.0 * W + 6) * live * C)
    if op in ("ssm", "ssm_bwd"):
        n, H, P, S, G = case["B"] * case["T"], case["H"], case["P"], case["S"], case["G"]
        ins = n * (2 * H * P + 4 * G * S + _size(case["dt"]) * H) + 12 * H
        state = 4 * (case["N"] or case["B"]) * H * P * S
        if op == "ssm":   # two products with the state a token: B x^T, S^T C
            return dict(bytes=ins + 2 * n * H * P + state * (2 if case["h0"] else 1), flops=4.0 * n * H * P * S)
        # the state again, then C dy^T, S dy, dS x, dS^T B
        return dict(bytes=ins + 2 * n * H * P + n * (2 * H * P + 4 * G * S + 4 * H) + 12 * H + state * (3 if case["h0"] else 0),
                    flops=10.0 * n * H * P * S)
    if op == "ssm_decode":
        live, H, P, S, G = case["n"] - case["skipped"], case["H"], case["P"], case["S"], case["G"]
        return dict(bytes=live * (8 * H * P * S + 4 * H * P + 4 * G * S + _size(case["dt"]) * H) + 12 * H + 4 * case["n"],
                    flops=5.0 * live * H * P * S)
    n, z = case["B"] * case["T"] * case.get("H", 1) * case["D"], _size(case["type"])
    if op in ("gated_norm", "gated_norm_bwd"):
        w = 0 if case["weight"] == "none" else 4 * case["D"] * (case["H"] if case["weight"] == "heads" else 1)
        if op == "gated_norm":
            return dict(bytes=3 * n * z + w, flops=12.0 * n)
        return dict(bytes=5 * n * z + 2 * w, flops=24.0 * n)
    r = _size(case["res"])
    if op == "add_norm":
        return dict(bytes=n * (2 * z + 2 * r) + 4 * case["D"], flops=6.0 * n)
    return dict(bytes=n * (2 * z + 3 * r) + 8 * case["D"], flops=12.0 * n)


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv", "conv_bwd"):
        return _exact_conv(s, op == "conv_bwd")
    if op in ("ssm", "ssm_bwd"):
        return _exact_scan(s, op == "ssm_bwd")
    if op == "conv_decode":
        out, pool = s["out"].to(F64), s["pool"].to(F64)
        for n, slot in enumerate(s["idx"].tolist()):
            if slot >= 0:
                out[n] = 0 if s["bias"] is None else s["bias"].to(F64)
                window = [*pool[slot], s["x"][n].to(F64)]
                for i, row in enumerate(window):
                    out[n] += s["w"][:, i].to(F64) * row
                out[n] *= 1 / (1 + torch.exp(-out[n])) if s["act"] else 1
                pool[slot] = torch.stack(window[1:])
        return out, pool
    if op == "ssm_decode":
        out, pool = s["out"].to(F64), s["pool"].to(F64)
        A, D, bias = (s[n].to(F64) for n in ("A", "D", "dt_bias"))
        for n, slot in enumerate(s["idx"].tolist()):
            if slot >= 0:
                x, dt = s["x"][n].to(F64), s["dt"][n].to(F64)
                out[n] = _step(pool[slot], x, torch.log1p(torch.exp(dt + bias)), A, *_wide(s, n), D)
        return out, pool
    leaf = lambda v: v.to(F64).requires_grad_()  # noqa: E731
    w = None if s["w"] is None else leaf(s["w"])
    if op in ("gated_norm", "gated_norm_bwd"):
        x, z = leaf(s["x"]), leaf(s["gate"])
        g = z / (1 + torch.exp(-z)) if s["act"] == "silu" else 1 / (1 + torch.exp(-z))
        v = x * g if s["first"] else x
        y = v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS)
        y = y if w is None else y * w
        y = y if s["first"] else y * g
        if op == "gated_norm":
            return y.detach()
        got = torch.autograd.grad(y, [x, z] + ([] if w is None else [w]), s["dy"].to(F64))
        return (*got, None) if w is None else got
    if op == "add_norm":
        h = s["res"].to(F64) + s["scale"] * s["x"].to(F64)
        return (h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + EPS) * w).detach(), h
    h = leaf(s["h"])
    y = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + EPS) * w
    dh, dw = torch.autograd.grad(y, [h, w], s["dy"].to(F64))
    dh = dh + s["dh"].to(F64)
    return s["scale"] * dh, dh, dw


def _exact_conv(s, backward):
    """Sequence by sequence: the state and the inputs as one row, a sum over shifted views; gradients by autograd."""
    C, W = s["w"].shape
    leaf = lambda v: v.to(F64).requires_grad_(backward)  # noqa: E731
    x, w = leaf(s["x"].reshape(-1, C)), leaf(s["w"])
    bias = None if s["bias"] is None else leaf(s["bias"])
    state = leaf(torch.zeros(len(s["lens"]), W - 1, C, device="cuda") if s["state"] is None else s["state"])
    ys, lasts, t = [], [], 0
    for n, m in enumerate(s["lens"]):
        row = torch.cat([state[n], x[t:t + m]])
        z = torch.zeros(m, C, dtype=F64, device="cuda") if bias is None else bias.expand(m, C)
        for i in range(W):
            z = z + row[i:i + m] * w[:, i]
        ys.append(z / (1 + torch.exp(-z)) if s["act"] else z)
        lasts.append(row[m:])
        t += m
    y, last = torch.cat(ys), torch.stack(lasts)
    if not backward:
        return y.view(s["x"].shape), last
    outs, grads = [y], [s["dy"].reshape(-1, C).to(F64)]
    if s["dlast"] is not None:
        outs, grads = outs + [last], grads + [s["dlast"].to(F64)]
    got = list(torch.autograd.grad(outs, [x, w, state] + ([] if bias is None else [bias]), grads))
    return (got[0].view(s["x"].shape), got[1], None if bias is None else got[3], None if s["state"] is None else got[2])


def _wide(s, *at):
    """B and C of some tokens for every head."""
    R = s["x"].shape[-2] // s["Bm"].shape[-2]
    return [s[n][at].to(F64).repeat_interleave(R, dim=-2) for n in ("Bm", "Cm")]


def _step(St, x, d, A, b, c, D):
    """One token of the recurrence, St [.., S, P] updated in place; returns y."""
    St *= torch.exp(d * A)[..., None, None]
    St += b.unsqueeze(-1) * (d.unsqueeze(-1) * x).unsqueeze(-2)
    return torch.matmul(c.unsqueeze(-2), St).squeeze(-2) + D[:, None] * x


def _exact_scan(s, backward):
    """Token by token.  The gradients walk back over each stretch of 64 tokens with its states recomputed."""
    H, P, S = s["x"].shape[2], s["x"].shape[3], s["Bm"].shape[3]
    R = H // s["Bm"].shape[2]
    if s["cu"] is None:
        parts = [(slice(0, s["x"].shape[0]), slice(0, s["x"].shape[1]), slice(0, s["x"].shape[0]))]
    else:
        c = s["cu"].tolist()
        parts = [(slice(0, 1), slice(a, b), slice(n, n + 1)) for n, (a, b) in enumerate(zip(c, c[1:]))]
    A, D, bias = (s[n].to(F64) for n in ("A", "D", "dt_bias"))
    raw = s["dt"].to(F64) + bias
    steps = torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0)
    new = lambda v: torch.zeros(v.shape, dtype=F64, device="cuda")  # noqa: E731
    y, last = new(s["x"]), torch.zeros(len(s["lens"]), H, S, P, dtype=F64, device="cuda")
    dx, dB, dC, dstep, dA, dh0 = new(s["x"]), new(s["Bm"]), new(s["Cm"]), new(s["dt"]), new(A), last.clone()
    for rows, span, seqs in parts:
        St = last[seqs] if s["h0"] is None else s["h0"][seqs].to(F64)
        kept = []
        for t in range(span.start, span.stop):
            if backward and (t - span.start) % 64 == 0:
                kept.append(St.clone())
            y[rows, t] = _step(St, s["x"][rows, t].to(F64), steps[rows, t], A, *_wide(s, rows, t), D)
        last[seqs] = St
        if not backward:
            continue
        dS = torch.zeros_like(St) if s["dlast"] is None else s["dlast"][seqs].to(F64)
        for k in range(len(kept) - 1, -1, -1):
            St, before = kept.pop(), []
            ts = range(span.start + 64 * k, min(span.start + 64 * k + 64, span.stop))
            for t in ts:
                before.append(St.clone())
                _step(St, s["x"][rows, t].to(F64), steps[rows, t], A, *_wide(s, rows, t), D)
            for t in reversed(ts):
                x, dy, d, (b, c) = s["x"][rows, t].to(F64), s["dy"][rows, t].to(F64), steps[rows, t], _wide(s, rows, t)
                ea = torch.exp(d * A)[..., None, None]
                decayed = before.pop() * ea
                now = decayed + b.unsqueeze(-1) * (d.unsqueeze(-1) * x).unsqueeze(-2)
                dS = dS + c.unsqueeze(-1) * dy.unsqueeze(-2)
                dC[rows, t] = torch.matmul(now, dy.unsqueeze(-1)).squeeze(-1).unflatten(1, (-1, R)).sum(2)
                Sx = torch.matmul(dS, x.unsqueeze(-1)).squeeze(-1)
                dB[rows, t] = (d.unsqueeze(-1) * Sx).unflatten(1, (-1, R)).sum(2)
                dx[rows, t] = d.unsqueeze(-1) * torch.matmul(b.unsqueeze(-2), dS).squeeze(-2) + D[:, None] * dy
                da = (decayed * dS).sum((-1, -2))
                dstep[rows, t] = (Sx * b).sum(-1) + A * da
                dA += (d * da).sum(0)
                dS = dS * ea
        dh0[seqs] = dS
    if not backward:
        return y, last
    draw = dstep * torch.sigmoid(raw)
    dD = (s["dy"].to(F64) * s["x"].to(F64)).sum((0, 1, 3))
    return dx, draw, dA, dB, dC, dD, draw.sum((0, 1)), dh0 if s["h0"] is not None else None
