"""Plain 64-bit forms of the short causal convolution and of the norms around a block, on the
CPU, and the tolerances of their tests.

Tolerances.  Every result is rounded once, by at most half a step of its type relative to itself
(torch.finfo(t).eps / 2; below fp16's normal range by at most 2^-25).  Before that everything is fp32:
  convolution: z sums at most five terms, so it is off by at most 5 2^-24 of their magnitudes mag =
    |bias| + sum |w x|; the activation's exponential, reciprocal and product are off by at most
    a unit each and its slope is at most 1.1: together 2^-20 mag.  dz = dy act'(z) is off by 2^-20 |dy| (1 + mag)
    (act' is at most 1.1, its own slope at most 0.5), dx by as much of sum |w| |dy| (1 + mag).  The weights'
    gradients are summed over a run of at most 32 tokens, at most 256 runs and an eighth of the tiles, far fewer
    than 512 additions one after the other in these tests: 2^-24 512 = 2^-15 of the sum of the magnitudes.
  norms: the sum of squares takes at most 32 additions in a lane and 12 between lanes, 2^-18 of itself with the
    rounding of each square, its inverse root half of that, the gate's activation 2^-21: together 2^-17 of
    the result, and of a sum that is normalised, 2^-23 r |w| (|residual| + |scale x|).  dv = r (dn - v m) is off by
    2^-16 r (|dn| + |v| M), M = r^2 mean |dn v|, and its products with the gate's activation and slope (at most 1.1)
    in proportion.  The weights' gradients add at most 6 rows in a lane here, 16 lanes and 64 + 8
    work-groups one after the other, 2^-16 of the sum of the magnitudes with each term's own 2^-17.
"""
import torch

F64 = torch.float64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def d64(t):
    return None if t is None else t.detach().cpu().double()


def close(got, want, off, what):
    """|got - want| <= half a step of got's type + off (a tensor or a number)."""
    half = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -149
    got = d64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), what
    over = ((got - want).abs() - half * want.abs() * (1 + 2.0 ** -12) - off - tiny)
    assert got.numel() == 0 or float(over.max()) <= 0, (what, float(over.max()))


def act(z, kind):
    return z if kind is None else z * torch.sigmoid(z) if kind == "silu" else torch.sigmoid(z)


def spans(x, cu):
    """(row, first token, end) of each sequence."""
    if cu is None:
        return [(b, 0, x.shape[1]) for b in range(x.shape[0])]
    c = [int(i) for i in cu]
    return [(0, a, e) for a, e in zip(c, c[1:])]


def conv(x, w, bias=None, kind="silu", state=None):
    """One sequence: x [T, C], state [W - 1, C], float64.  Returns y, the final state, and mag (see above)."""
    W = w.shape[1]
    rows = torch.cat([torch.zeros(W - 1, x.shape[1], dtype=F64) if state is None else state, x])
    z = torch.zeros_like(x) if bias is None else bias.expand_as(x)
    mag = z.abs()
    for i in range(W):
        z = z + w[:, i] * rows[i:i + x.shape[0]]
        mag = mag + (w[:, i] * rows[i:i + x.shape[0]]).abs()
    return act(z, kind), rows[x.shape[0]:], mag.detach()


def conv_batch(x, w, bias=None, kind="silu", cu=None, state=None):
    """y and mag [B, T, C] (NaN in no sequence) and the final states."""
    y = torch.full(x.shape, float("nan"), dtype=F64)
    mag, last = y.clone(), []
    for n, (b, a, e) in enumerate(spans(x, cu)):
        y[b, a:e], f, mag[b, a:e] = conv(d64(x)[b, a:e], d64(w), d64(bias), kind, None if state is None else d64(state)[n])
        last.append(f)
    return y, mag, torch.stack(last) if last else torch.zeros(0, w.shape[1] - 1, x.shape[2], dtype=F64)


def conv_grads(x, w, dy, bias=None, kind="silu", cu=None, state=None, dlast=None):
    """Gradients and the magnitudes that their tolerances go by: dicts with dx, dweight, dbias, dstate."""
    W = w.shape[1]
    wl, bl = d64(w).requires_grad_(), None if bias is None else d64(bias).requires_grad_()
    g = dict(dx=torch.full(x.shape, float("nan"), dtype=F64), dstate=torch.zeros(len(spans(x, cu)), W - 1, x.shape[2], dtype=F64),
             dweight=torch.zeros(w.shape, dtype=F64), dbias=torch.zeros(w.shape[0], dtype=F64))
    m = {n: torch.zeros_like(t) for n, t in g.items()}
    for n, (b, a, e) in enumerate(spans(x, cu)):
        xl = d64(x)[b, a:e].requires_grad_()
        sl = (torch.zeros(W - 1, x.shape[2], dtype=F64) if state is None else d64(state)[n]).requires_grad_()
        y, last, mag = conv(xl, wl, bl, kind, sl)
        loss = (y * d64(dy)[b, a:e]).sum()
        if dlast is not None:
            loss = loss + (last * d64(dlast)[n]).sum()
        got = torch.autograd.grad(loss, [xl, sl, wl] + ([] if bl is None else [bl]), allow_unused=True)
        got = [torch.zeros_like(v) if r is None else r for r, v in zip(got, [xl, sl, wl] + ([] if bl is None else [bl]))]
        g["dx"][b, a:e], g["dstate"][n] = got[0], got[1]
        g["dweight"] += got[2]
        if bl is not None:
            g["dbias"] += got[3]
        dz = d64(dy)[b, a:e].abs() * (1 + mag)
        rows = torch.cat([sl.detach(), xl.detach()]).abs()
        mrow = torch.zeros_like(rows)
        for i in range(W):
            mrow[i:i + e - a] += d64(w)[:, i].abs() * dz
            m["dweight"][:, i] += (dz * rows[i:i + e - a]).sum(0)
        m["dbias"] += dz.sum(0)
        m["dstate"][n], m["dx"][b, a:e] = mrow[:W - 1], mrow[W - 1:]
    return g, m


def rms(v, eps):
    return torch.rsqrt(v.pow(2).mean(-1, keepdim=True) + eps)


def gated(x, gate, w=None, kind="silu", first=False, eps=1e-6):
    g = act(gate, kind)
    v = x * g if first else x
    y = v * rms(v, eps)
    y = y if w is None else y * w
    return y if first else y * g


def norm_grad_size(v, dn, eps):
    """r (|dn| + |v| M) of dv (see above)."""
    r = rms(v, eps)
    return r * (dn.abs() + v.abs() * (r * r * (dn * v).abs().mean(-1, keepdim=True)))
