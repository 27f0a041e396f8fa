"""64-bit reference of the per-head-decay linear attention and of layer norm,
written from the recurrence, one token after the other, and the bounds that the
GPU results are held to.

    S_t = exp(g_t) S_{t-1} + k_t v_t^T          o_t = scale S_t^T q_t

Bounds.  With every input replaced by its absolute value the same recurrence
gives, for each output, the sum of the absolute values of all terms it is made
of ("abs" below).  A computed output is off by at most rel * abs plus its own
rounding, where rel counts, per term and in units of u = 2^-24 (fp32):
  - the scores' sum over d channels and the sums over 64 tokens of a chunk and
    over d channels of the state: d + 64 + d
  - one rounding of the state a chunk and product: 4 a chunk
  - the decays: the exponent is a difference of fp32 pairs whose size matters up
    to 104 (exp(-104) is 0 in fp32), 104 u, through two such factors, and an ulp
    or two of the exponential: 256
  - factors that enter the products as p bf16 values are off by 2^-8 per value,
    2^-8p of themselves.  For bf16 inputs each term of o holds one such factor, an
    element of the scores or of the state: p = 1 where the output is bf16 (2^-8),
    p = 2 where it is fp32 (2^-16, 2^-15 with what the first product passes on to the
    second).  dv is like o; dq and dk, whose dots make dg, and everything else
    have p = 3 (a few u).
"""
import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _heads(x, H):
    return x.repeat_interleave(H // x.shape[1], 1)


def _per_token(g, T, H):
    return torch.clamp(g.double().expand(T, H), min=-110.0)


def forward(q, k, v, g, cu, S0=None, scale=1.0):
    """o [T, H, dv], final states [N, H, dk, dv]; cu a list of N + 1 ints."""
    T, H = v.shape[0], v.shape[1]
    q, k, v = _heads(q.double(), H), _heads(k.double(), H), v.double()
    a = torch.exp(_per_token(g, T, H))
    o = torch.zeros(T, H, v.shape[2], dtype=torch.float64)
    fin = []
    for n in range(len(cu) - 1):
        S = torch.zeros(H, q.shape[2], v.shape[2], dtype=torch.float64)
        if S0 is not None:
            S = S0[n].double().clone()
        for t in range(cu[n], cu[n + 1]):
            S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * torch.einsum("hcj,hc->hj", S, q[t])
        fin.append(S)
    return o, torch.stack(fin)


def backward(q, k, v, g, cu, d_o=None, S0=None, dS=None, scale=1.0, signs=True):
    """(dq, dk, dv, dg, dS0).  signs False: the sums of the terms' absolute values
    (the inputs given as absolute values), dg's with both of its sums added."""
    T, H, Hk = v.shape[0], v.shape[1], q.shape[1]
    per = g.dim() == 2
    q_, k_, v_ = _heads(q.double(), H), _heads(k.double(), H), v.double()
    do = torch.zeros_like(v_) if d_o is None else d_o.double()
    a = torch.exp(_per_token(g, T, H))
    dq, dk, dv = torch.zeros_like(q_), torch.zeros_like(k_), torch.zeros_like(v_)
    dg = torch.zeros(T, H, dtype=torch.float64)
    dS0 = []
    for n in range(len(cu) - 1):
        S = torch.zeros(H, q.shape[2], v.shape[2], dtype=torch.float64)
        if S0 is not None:
            S = S0[n].double().clone()
        before = []
        for t in range(cu[n], cu[n + 1]):
            before.append(S)
            S = a[t][:, None, None] * S + k_[t][:, :, None] * v_[t][:, None, :]
            dq[t] = scale * torch.einsum("hcj,hj->hc", S, do[t])
        D = torch.zeros_like(S) if dS is None else dS[n].double().clone()
        loose = (S * D).sum((-1, -2))
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            D = D + scale * q_[t][:, :, None] * do[t][:, None, :]
            dk[t] = torch.einsum("hcj,hj->hc", D, v_[t])
            dv[t] = torch.einsum("hcj,hc->hj", D, k_[t])
            dg[t] = a[t] * (D * before[t - cu[n]]).sum((-1, -2))
            if not signs:
                loose = loose + (q_[t] * dq[t]).sum(-1) + (k_[t] * dk[t]).sum(-1)
                dg[t] = loose
            D = a[t][:, None, None] * D
        dS0.append(D)
    share = lambda x: x.view(T, Hk, H // Hk, x.shape[2]).sum(2)  # noqa: E731
    # log-decays below -110 count as -110; the gradient is that of the recurrence there
    return share(dq), share(dk), dv, dg if per else dg.sum(0), torch.stack(dS0)


def _abs(x):
    return None if x is None else x.double().abs()


def rel_of(q, v, cu, values):
    """values: bf16 values a factor of the output's products is made of."""
    d = max(q.shape[2], v.shape[2])
    chunks = max([-(-(b - a) // 64) for a, b in zip(cu, cu[1:])] + [1])
    return (2 * d + 64 + 4 * chunks + 256) * U + {1: 2.0 ** -8, 2: 2.0 ** -15, 3: 0.0}[values]


def _values(wide, dtype):
    return 3 if wide else 1 if dtype == torch.bfloat16 else 2


def check(name, got, want, size, rel, dtype):
    """|got - want| <= rel * size (1 + round) + round * |want|, elementwise."""
    got = got.detach().to("cpu", torch.float64)
    assert torch.isfinite(got).all(), name
    bound = rel * size * (1 + ROUND[dtype]) + ROUND[dtype] * want.abs() + 1e-30
    worst = ((got - want).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g times its bound" % (name, worst)
    return worst


def check_forward(o, S, q, k, v, g, cu, S0=None, scale=1.0, o_rows=None):
    """o and the states S (None: not checked) against the reference; o_rows limits o."""
    want, want_S = forward(q, k, v, g, cu, S0, scale)
    size, size_S = forward(_abs(q), _abs(k), _abs(v), g, cu, _abs(S0), abs(scale))
    wide = q.dtype == torch.float32
    rel = rel_of(q, v, cu, _values(wide, o.dtype))
    m = want.shape[0] if o_rows is None else o_rows
    r = [check("o", o[:m], want[:m], size[:m], rel, o.dtype)]
    if S is not None:
        # the state itself is made of three-value factors
        r.append(check("state", S, want_S, size_S, rel_of(q, v, cu, 3), S.dtype))
    return r


def check_backward(got, q, k, v, g, cu, d_o=None, S0=None, dS=None, scale=1.0):
    want = backward(q, k, v, g, cu, d_o, S0, dS, scale)
    size = backward(_abs(q), _abs(k), _abs(v), g, cu, _abs(d_o), _abs(S0), _abs(dS), abs(scale),
                    signs=False)
    wide = q.dtype == torch.float32 or (d_o is not None and d_o.dtype == torch.float32)
    rel = rel_of(q, v, cu, 3)
    # dg: 128 more fp32 terms a dot and the state's inner product of 16,384 / 256 a lane
    rels = [rel, rel, rel_of(q, v, cu, _values(wide, got[2].dtype)), rel + 256 * U,
            rel_of(q, v, cu, 3)]
    out = []
    for name, x, w, s, r in zip(("dq", "dk", "dv", "dg", "dS0"), got, want, size, rels):
        if x is not None:
            out.append(check(name, x, w, s, r, x.dtype))
    return out


# ------------------------------------------------------------- layer norm
def norm(x, w=None, b=None, eps=1e-5):
    x = x.double()
    c = x - x.mean(-1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    y = y * w.double() if w is not None else y
    return y + b.double() if b is not None else y


def norm_backward(dy, x, w=None, eps=1e-5):
    x, dy = x.double(), dy.double()
    c = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    xh = c * r
    t = dy * w.double() if w is not None else dy
    dx = r * (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True))
    over = tuple(range(x.dim() - (w.dim() if w is not None else 1)))
    return dx, (dy * xh).sum(over) if over else dy * xh, dy.sum(over) if over else dy
