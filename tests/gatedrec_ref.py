"""64-bit reference of the gated linear recurrence and RMS norm on the CPU, with bounds on
what fp32 may be off, in u = 2^-24 per rounding.

Gate: z = r + dt_bias (in log2 units: its two terms and the sum are rounded, 3 u of each, at
most |z| + 2 |dt_bias|) enters exp(-|z|), whose exp2 adds 2 u; log2(1 + e) is off by 6 u, the
sum and the product with exp(A_log) (3 u) by 5 u.  So g is off by
eg = (15 + 2 |z| + 2 |dt_bias|) u of itself (log-decays: u).  a = exp(g): the exponent's product and the
hardware's exp2 make (2 + 3 |g|) u, g's error |g| eg.  m = sqrt(1 - exp(2 g)): 1 - exp(y) off
by at most 22 u + 2 eg of itself (beyond |y| = 0.17 it is 1 - a a, where the exp2's 2 u of a
become 4 u 0.84 / 0.16), its root by half of that and u.  sigmoid(i): (4 + 3 |i|) u.  So b = m s x: eb = (20 + 3 |i|) u + eg (4 u for the products).

h: with H_t = a H_{t-1} + |b_t| (the recurrence of absolute values, which bounds |h|):
- a token's own b: eb;
- inside a wave's tokens (at most 16) a and the sums round 4 times a token, inside a tile (at
  most 8 waves) folds round 4 times a wave: 96 u of H;
- the decay over longer stretches is exp of a sum s of log-decays, or 1 - (1 - exp(s)) beside
  1: off by (8 u + eg) |s| of itself, and each tile's fold rounds 3 times, in 64 tokens.
The last part adds up along the decay: D_t = a D_{t-1} + (u (3 / 64 + 8 |g|) + eg |g|) H_t.
  |h error| <= 96 u H + B + D,   B_t = a B_{t-1} + eb |b_t|
R (the gradient of h): the same backwards with dh in the place of b.
"""
import math

import torch

U = 2.0 ** -24
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
F64 = torch.float64


def gate(x, r, i, A_log, dt_bias, normalize):
    f = {"x": x.to(F64)}
    r = r.to(F64)
    if A_log is not None:
        z = r + (dt_bias.to(F64) if dt_bias is not None else 0.0)
        f["k"] = -torch.exp(A_log.to(F64))
        f["sz"] = torch.sigmoid(z)
        f["g"] = f["k"] * torch.logaddexp(z, torch.zeros_like(z))
        bias = dt_bias.to(F64).abs() if dt_bias is not None else 0.0
        f["eg"] = (15 + 2 * torch.nan_to_num(z).abs() + 2 * bias) * U
        f["z"] = z
    else:
        f["g"] = torch.where(r > 0, torch.zeros_like(r), r)
        f["eg"] = torch.full_like(r, U)
    f["a"] = torch.exp(f["g"])
    f["s"] = torch.sigmoid(i.to(F64)) if i is not None else torch.ones_like(r)
    f["es"] = (4 + 3 * i.to(F64).abs().clamp(max=100)) * U if i is not None else torch.zeros_like(r)
    f["m"] = torch.sqrt(-torch.expm1(2 * f["g"])) if normalize else torch.ones_like(r)
    f["em"] = (12 * U + f["eg"]) if normalize else torch.zeros_like(r)
    f["b"] = f["m"] * f["s"] * f["x"]
    f["eb"] = 4 * U + f["es"] + f["em"]
    return f


def _along(f):
    """What the decay's error adds per token, of H."""
    g = torch.nan_to_num(f["g"], neginf=-200.0).clamp(min=-200.0).abs()
    return U * (3 / 64 + 8 * g) + f["eg"] * g


def scan(x, r, i, A_log, dt_bias, normalize, cu, S0):
    """dict: h [T, C], S [N, C], their bounds eh, eS (before any rounding of the outputs)."""
    f = gate(x, r, i, A_log, dt_bias, normalize)
    T, C = x.shape
    N = len(cu) - 1
    new = lambda n: torch.zeros(n, C, dtype=F64)  # noqa: E731
    h, eh, H = new(T), new(T), new(T)
    S, eS = new(N), new(N)
    if S0 is not None:
        S += S0.to(F64)
    f["S0"] = S.clone()
    along = _along(f)
    for n in range(N):
        s, A, B, D = S[n].clone(), S[n].abs(), torch.zeros(C, dtype=F64), torch.zeros(C, dtype=F64)
        for t in range(cu[n], cu[n + 1]):
            a = f["a"][t]
            s = a * s + f["b"][t]
            A = a * A + f["b"][t].abs()
            B = a * B + f["eb"][t] * f["b"][t].abs()
            D = a * D + along[t] * A
            h[t], H[t], eh[t] = s, A, 96 * U * A + B + D
        S[n] = s
        if cu[n + 1] > cu[n]:
            eS[n] = eh[cu[n + 1] - 1]
    f.update(h=h, H=H, eh=eh, S=S, eS=eS)
    return f


def backward(x, r, i, A_log, dt_bias, normalize, cu, S0, dh, dS):
    """dict: dx, dr, di, dA, db, dS0 with bounds e<name>; None where there is no such output."""
    f = scan(x, r, i, A_log, dt_bias, normalize, cu, S0)
    T, C = x.shape
    N = len(cu) - 1
    new = lambda n: torch.zeros(n, C, dtype=F64)  # noqa: E731
    dh = dh.to(F64) if dh is not None else new(T)
    R, eR = new(T), new(T)
    E = dS.to(F64).clone() if dS is not None else new(N)
    eE = new(N)
    prev, eprev = new(T), new(T)
    along = _along(f)
    for n in range(N):
        lo, hi = cu[n], cu[n + 1]
        if lo == hi:
            continue
        prev[lo] = f["S0"][n]
        prev[lo + 1:hi], eprev[lo + 1:hi] = f["h"][lo:hi - 1], f["eh"][lo:hi - 1]
        e, A, D = E[n].clone(), E[n].abs(), torch.zeros(C, dtype=F64)
        for t in range(hi - 1, lo - 1, -1):
            R[t] = dh[t] + e
            A = dh[t].abs() + A
            eR[t] = 96 * U * A + D
            D = f["a"][t] * (D + along[t] * A)
            A = f["a"][t] * A
            e = f["a"][t] * R[t]
        E[n], eE[n] = e, 96 * U * A + D
    a, m, s, g = f["a"], f["m"], f["s"], f["g"]
    gg = torch.nan_to_num(g, neginf=-200.0).clamp(min=-200.0)
    ea = (2 + 3 * gg.abs()) * U + f["eg"] * gg.abs()  # of a
    du = m * R
    edu = m * eR + (f["em"] + U) * du.abs()
    out = dict(f, dx=du * s, edx=edu * s + (f["es"] + 2 * U) * (du * s).abs())
    out["di"], out["edi"] = None, None
    if i is not None:
        p = out["dx"] * f["x"]
        out["di"] = p * (1 - s)  # 1 - s keeps s's own error
        out["edi"] = out["edx"] * (f["x"] * (1 - s)).abs() + p.abs() * ((f["es"] + U) * s + 3 * U)
    first = a * prev * R
    dg = first.clone()
    edg = (ea + 4 * U) * first.abs() + a * (eprev * R.abs() + (prev.abs() + eprev) * eR)
    if normalize:
        w = torch.where(m > 0, a * a / m, torch.zeros_like(m)) * s * f["x"]
        dg = dg - w * R
        edg = edg + w.abs() * eR + (2 * ea + f["em"] + f["es"] + 10 * U) * (w * R).abs()
    edg = edg + 2 * U * dg.abs()
    out["dA"] = out["db"] = out["edA"] = out["edb"] = None
    if A_log is not None:
        k, sz = f["k"], f["sz"]
        esz = (4 + 4 * torch.nan_to_num(f["z"]).abs().clamp(max=100)) * U
        out["dr"] = dg * k * sz
        out["edr"] = (k * sz).abs() * edg + (esz + 6 * U) * out["dr"].abs()
        # eight tokens and eight waves are added in fp32, the rest in 64 bits
        out["dA"] = (dg * gg).sum(0)
        out["edA"] = (edg * gg.abs() + (f["eg"] + 20 * U) * (dg * gg).abs()).sum(0)
        out["db"] = out["dr"].sum(0)
        out["edb"] = (out["edr"] + 20 * U * out["dr"].abs()).sum(0)
    else:
        on = (r <= 0).to(F64)
        out["dr"], out["edr"] = dg * on, edg * on
    out["dS0"], out["edS0"] = E, eE
    return out


def within(name, got, want, bound, dtype):
    """got against want: bound, and the rounding to dtype.  The worst share of it."""
    assert got.dtype == dtype, name
    got = got.detach().to("cpu", F64)
    assert got.shape == want.shape, name
    if not want.numel():
        return 0.0
    bound = bound * (1 + ROUND[dtype]) + ROUND[dtype] * want.abs() + 1e-36
    worst = ((got - want).abs() / bound).max().item()
    assert math.isfinite(worst) and worst <= 1.0, "%s: %.3g times its bound" % (name, worst)
    return worst


# ------------------------------------------------------------------ RMS norm
def rms_sum(x, residual):
    """s as it is stored."""
    if residual is None:
        return x
    return (x.float() + residual.float()).to(residual.dtype)


def rmsnorm(s, w, eps):
    """y in 64 bits, and the bound of its fp32 value: the mean square is a sum of d positive
    values (at most log2 d + 12 roundings in a row), its root halves that."""
    s = s.to(F64)
    d = s.shape[-1]
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.to(F64)
    return y, ((math.log2(d) + 12) / 2 + 6) * U * y.abs()


def rmsnorm_backward(dy, s, w, dres, eps):
    """(dx, bound, dweight, bound)."""
    s, dy = s.to(F64), dy.to(F64)
    d = s.shape[-1]
    n = (math.log2(d) + 12) * U
    r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    t = dy * (w.to(F64) if w is not None else 1.0)
    xh = s * r
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    dx = r * (t - xh * mean(t * xh))
    e = r * ((n + 6 * U) * t.abs() + (4 * n + 8 * U) * xh.abs() * mean((t * xh).abs()))
    if dres is not None:
        dx = dx + dres.to(F64)
        e = e + 2 * U * dx.abs()
    if w is None:
        return dx, e, None, None
    over = tuple(range(dy.dim() - w.dim()))
    rows = dy.numel() // (d * (w.shape[0] if w.dim() > 1 else 1))
    sums = lambda v: v.sum(over) if over else v  # noqa: E731
    return dx, e, sums(dy * xh), (n + (min(rows, 4096) + 32) * U) * sums((dy * xh).abs())
