"""Plain 64-bit forms of the selective state space scan, token by token on the CPU, and the tolerances of
its tests.

Tolerances.  Each result is compared with the magnitude of the terms that make it up: with Sabs the recurrence
of |d B x| (Sabs_t = e^{d A} Sabs_{t-1} + d |B| |x|) and Dabs that of the gradients backwards,
  y      2^-8 of itself (its one rounding to bf16), and 2^-15 of |C| Sabs + |D x|: the states and the pair
         matrix enter in two bf16 parts, off by 2^-17 of themselves at most; a chunk's sums are 128 fp32 terms,
         2^-17, the decays' exponentials a few units of 2^-24
  states 2^-17 of Sabs: 24-bit operands, 64 fp32 terms a chunk and one more a chunk, and as much for the
         gradient of the initial state
  dC, dB, dx  2^-8 of themselves and 2^-15 of Sabs |dy|, Dabs d |x| (over a group's heads), d |B| Dabs + |D dy|
  ddt    the step's slope times |A| da + |B| Dabs |x|, da = e^{dA} <Sabs, Dabs>: the sums over pairs take 64 products
         of two 128-term sums, 2^-16 with their rows and columns added over 64 tokens, 2^-15 in all
  dA, dD, ddt_bias  2^-15 of the sum of their terms' magnitudes
"""
import torch

F64 = torch.float64


def d64(t):
    return None if t is None else t.detach().cpu().double()


def step(dt, bias, softplus):
    raw = dt if bias is None else dt + bias
    return torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw


def scan(x, dt, A, B, C, D=None, bias=None, softplus=True, h0=None):
    """One sequence: x [T, H, P], dt [T, H], B, C [T, G, S], h0 [H, S, P], float64.  Returns y and the final state."""
    R = x.shape[1] // B.shape[1]
    B, C = B.repeat_interleave(R, dim=1), C.repeat_interleave(R, dim=1)
    d = step(dt, bias, softplus)
    S = torch.zeros(x.shape[1], B.shape[2], x.shape[2], dtype=F64) if h0 is None else h0
    ys = []
    for t in range(x.shape[0]):
        S = torch.exp((d[t] * A).clamp(min=-200.0))[:, None, None] * S + B[t].unsqueeze(-1) * (d[t].unsqueeze(-1) * x[t]).unsqueeze(-2)
        y = torch.matmul(C[t].unsqueeze(-2), S).squeeze(-2)
        ys.append(y if D is None else y + D[:, None] * x[t])
    return (torch.stack(ys) if ys else x.clone()), S


def spans(x, cu):
    if cu is None:
        return [(b, 0, x.shape[1]) for b in range(x.shape[0])]
    c = [int(i) for i in cu]
    return [(0, a, e) for a, e in zip(c, c[1:])]


TOKEN = ("x", "dt", "B", "C")


def run(c, cu=None):
    """y and its magnitude [B, T, H, P] (NaN in no sequence), final states and theirs, of a dict of inputs."""
    d = {n: d64(t) if isinstance(t, torch.Tensor) else t for n, t in c.items()}
    y = torch.full(d["x"].shape, float("nan"), dtype=F64)
    ym, S, Sm = y.clone(), [], []
    for n, (b, a, e) in enumerate(spans(d["x"], cu)):
        part = [d[m][b, a:e] for m in TOKEN]
        h0 = None if d["h0"] is None else d["h0"][n]
        y[b, a:e], s = scan(part[0], part[1], d["A"], part[2], part[3], d["D"], d["bias"], c["softplus"], h0)
        D = None if d["D"] is None else d["D"].abs()
        # magnitudes: steps as they are, everything else by its absolute value
        st = step(part[1], d["bias"], c["softplus"])
        ym[b, a:e], sm = magnitude(part[0], st, d["A"], part[2], part[3], D, h0)
        S.append(s)
        Sm.append(sm)
    return y, ym, torch.stack(S), torch.stack(Sm)


def magnitude(x, st, A, B, C, D, h0):
    R = x.shape[1] // B.shape[1]
    B, C, x = B.abs().repeat_interleave(R, dim=1), C.abs().repeat_interleave(R, dim=1), x.abs()
    S = torch.zeros(x.shape[1], B.shape[2], x.shape[2], dtype=F64) if h0 is None else h0.abs()
    ys = []
    for t in range(x.shape[0]):
        S = torch.exp((st[t] * A).clamp(min=-200.0))[:, None, None] * S + B[t].unsqueeze(-1) * (st[t].abs().unsqueeze(-1) * x[t]).unsqueeze(-2)
        y = torch.matmul(C[t].unsqueeze(-2), S).squeeze(-2)
        ys.append(y if D is None else y + D[:, None] * x[t])
    return (torch.stack(ys) if ys else x.clone()), S


def gradients(c, cu=None):
    """Gradients by autograd of the recurrence and, under the same names, the magnitudes of their terms."""
    d = {n: d64(t) if isinstance(t, torch.Tensor) else t for n, t in c.items()}
    nan = lambda t: torch.full(t.shape, float("nan"), dtype=F64)  # noqa: E731
    g = dict(dx=nan(d["x"]), ddt=nan(d["dt"]), dB=nan(d["B"]), dC=nan(d["C"]), dA=torch.zeros_like(d["A"]),
             dD=torch.zeros_like(d["A"]), ddt_bias=torch.zeros_like(d["A"]), dh0=[])
    m = {n: (t.clone() if n != "dh0" else []) for n, t in g.items()}
    H, P, S, G = d["x"].shape[2], d["x"].shape[3], d["B"].shape[3], d["B"].shape[2]
    for n, (b, a, e) in enumerate(spans(d["x"], cu)):
        leaves = [d[k][b, a:e].clone().requires_grad_() for k in TOKEN]
        A, D = d["A"].clone().requires_grad_(), torch.zeros(H, dtype=F64).requires_grad_() if d["D"] is None else d["D"].clone().requires_grad_()
        bias = torch.zeros(H, dtype=F64).requires_grad_() if d["bias"] is None else d["bias"].clone().requires_grad_()
        h0 = (torch.zeros(H, S, P, dtype=F64) if d["h0"] is None else d["h0"][n].clone()).requires_grad_()
        y, s = scan(leaves[0], leaves[1], A, leaves[2], leaves[3], D, bias, c["softplus"], h0)
        dy = d["dy"][b, a:e]
        loss = (y * dy).sum()
        if d["dlast"] is not None:
            loss = loss + (s * d["dlast"][n]).sum()
        alls = leaves + [A, D, bias, h0]
        got = torch.autograd.grad(loss, alls, allow_unused=True) if loss.requires_grad else [None] * len(alls)
        got = [torch.zeros_like(v) if r is None else r for r, v in zip(got, alls)]
        for k, r in zip(TOKEN, got):
            g["d" + k][b, a:e] = r
        g["dA"] += got[4]
        g["dD"] += got[5]
        g["ddt_bias"] += got[6]
        g["dh0"].append(got[7])
        # magnitudes
        with torch.no_grad():
            x, dt, B, C = (v.detach() for v in leaves)
            st = step(dt, bias.detach(), c["softplus"])
            slope = torch.sigmoid(dt + bias.detach()) if c["softplus"] else torch.ones_like(dt)
            R = H // G
            Bw, Cw, xa, dya = B.abs().repeat_interleave(R, dim=1), C.abs().repeat_interleave(R, dim=1), x.abs(), dy.abs()
            Sm, states = h0.detach().abs(), []
            for t in range(e - a):
                ea = torch.exp((st[t] * A).clamp(min=-200.0))[:, None, None]
                before = ea * Sm
                Sm = before + Bw[t].unsqueeze(-1) * (st[t].abs().unsqueeze(-1) * xa[t]).unsqueeze(-2)
                states.append((before, Sm))
            Dm = torch.zeros(H, S, P, dtype=F64) if d["dlast"] is None else d["dlast"][n].abs()
            for t in range(e - a - 1, -1, -1):
                before, Sm = states[t]
                Dm = Dm + Cw[t].unsqueeze(-1) * dya[t].unsqueeze(-2)
                m["dC"][b, a + t] = torch.matmul(Sm, dya[t].unsqueeze(-1)).squeeze(-1).unflatten(0, (G, R)).sum(1)
                Vx = torch.matmul(Dm, xa[t].unsqueeze(-1)).squeeze(-1)
                m["dB"][b, a + t] = (st[t].abs().unsqueeze(-1) * Vx).unflatten(0, (G, R)).sum(1)
                m["dx"][b, a + t] = st[t].abs().unsqueeze(-1) * torch.matmul(Bw[t].unsqueeze(-2), Dm).squeeze(-2) + D.abs()[:, None] * dya[t]
                da = (before * Dm).sum((-1, -2))
                dd = slope[t] * (A.abs() * da + (Vx * Bw[t]).sum(-1))
                m["ddt"][b, a + t] = dd
                m["dA"] += st[t].abs() * da
                m["ddt_bias"] += dd
                m["dD"] += (dya[t] * xa[t]).sum(-1)
                Dm = Dm * torch.exp((st[t] * A).clamp(min=-200.0))[:, None, None]
            m["dh0"].append(Dm)
    g["dh0"], m["dh0"] = torch.stack(g["dh0"]), torch.stack(m["dh0"])
    return g, m


def make(B, T, H, P, S, G, N=None, dt="f32", h0=False, D=True, bias=True, softplus=True, seed=0, fast=16.0, spread=1.0):
    """Inputs on the CPU: steps of 0.001 to 0.1 and more, A -1 .. -fast."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n = B if N is None else N
    c = dict(x=rnd(B, T, H, P).bfloat16(), dt=(spread * rnd(B, T, H)), A=-(1 + (fast - 1) * torch.rand(H, generator=gen)),
             B=rnd(B, T, G, S).bfloat16(), C=rnd(B, T, G, S).bfloat16(), D=1 + 0.3 * rnd(H) if D else None,
             bias=-4.6 + 2.3 * torch.rand(H, generator=gen) if bias else None, h0=rnd(n, H, S, P) if h0 else None,
             dy=rnd(B, T, H, P).bfloat16(), dlast=rnd(n, H, S, P) if h0 else None, softplus=softplus)
    if not softplus:
        c["dt"] = 0.01 * torch.exp(c["dt"])
        c["bias"] = 0.002 * torch.rand(H, generator=gen) if bias else None
    if dt == "bf16":
        c["dt"] = c["dt"].bfloat16()
    return c


def cuda(c):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in c.items()}


def close(got, want, off, what):
    """|got - want| <= half a step of got's type + off; entries whose reference is NaN are skipped."""
    half = torch.finfo(got.dtype).eps / 2 * (1 + 2.0 ** -12)
    got = d64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    real = ~torch.isnan(want)
    got, want, off = got[real], want[real], off[real]
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - half * want.abs() - off
    if got.numel():
        worst = ((got - want).abs() - half * want.abs()) / off.clamp(min=1e-300)
        assert float(over.max()) <= 2.0 ** -140, (what, "times the tolerance", float(worst.max()))


BITS = dict(y=2.0 ** -15, state=2.0 ** -17, dx=2.0 ** -15, ddt=2.0 ** -15, dB=2.0 ** -15, dC=2.0 ** -15, dA=2.0 ** -15, dD=2.0 ** -15,
            ddt_bias=2.0 ** -15, dh0=2.0 ** -17)
