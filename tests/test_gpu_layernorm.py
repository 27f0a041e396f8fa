"""GPU: layer norm forward and backward against 64-bit formulas.

Bounds, in u = 2^-24 per fp32 rounding.  A row's mean is a sum of d values off
by at most (log2 d + 8) u times the mean of their absolute values A (a thread
adds up to 16 values in turn, the rest are pairwise), so x - mean is off by
e = (log2 d + 10) u (A + |x|); the mean square and the root add (log2 d + 12) u
relative, and a shift of the mean by e changes the variance by e^2 only (the sum
of the differences is 0).  With r = 1 / sqrt(var + eps):
  |xh error| <= E = r e + (log2 d + 14) u |xh|
  y: E |w| + 4 u (|xh w| + |b|), and the rounding of y
  dx: t = dy w is off by u |t|; its two means by (log2 d + 10) u of their absolute
  means, mean(|t| E) from xh; |xh| mean(t xh) adds its own xh error:
     r (4 u |t| + L u mean|t| + |xh| (L u mean|t xh| + mean(|t| E)) + E |mean(t xh)|)
     + L u |dx|,   L = log2 d + 16
  dw: sum over rows of |dy| E plus (rows a thread adds in turn + 32) u sum |dy xh|
  db: the same with |dy| alone
"""
import math

import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import linattn_ref as ref
from tests.gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = ref.U


def _xh_error(x, eps):
    x = x.double()
    d = x.shape[-1]
    lg = math.log2(d) if d > 1 else 0.0
    c = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    e = (lg + 10) * U * (x.abs().mean(-1, keepdim=True) + x.abs())
    # the shift of the mean against the variance itself: relative e^2 r^2, only near var = 0
    rel = (lg + 14) * U + (e * r).amax(-1, keepdim=True) ** 2
    return c * r, r, r * e + rel * (c * r).abs(), lg


def _within(name, got, want, bound, dtype):
    got = got.detach().to("cpu", torch.float64)
    bound = bound * (1 + ref.ROUND[dtype]) + ref.ROUND[dtype] * want.abs() + 1e-30
    worst = ((got - want).abs() / bound).max().item() if want.numel() else 0.0
    assert math.isfinite(worst) and worst <= 1.0, "%s: %.3g times its bound" % (name, worst)
    return worst


def _make(shape, wshape, dtype, seed, offset=1.0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (rnd(*shape) * 1.5 + offset * rnd(*shape[:-1], 1)).to(dtype)
    w = None if wshape is None else 1 + 0.3 * rnd(*wshape)
    b = None if wshape is None else rnd(*wshape)
    return x, w, b, rnd(*shape).to(dtype)


CASES = [  # x's shape, weight's shape
    ((1, 1), (1,)), ((5, 1), None), ((3, 2), (2,)), ((7, 9), (9,)), ((2, 63), (63,)),
    ((9, 64), (64,)), ((4, 65), None), ((50, 3, 128), (3, 128)), ((50, 3, 128), (128,)),
    ((6, 5, 129), (5, 129)), ((1, 2, 64), (2, 64)), ((33, 255), (255,)), ((11, 4, 256), (4, 256)),
    ((17, 511), (511,)), ((6, 1000), (1000,)), ((5, 1025), (1025,)), ((3, 2, 2048), (2, 2048)),
    ((4, 4095), (4095,)), ((3, 4097), (4097,)), ((3, 8192), (8192,)), ((2, 8193), None),
    ((2, 16384), (16384,)), ((2, 16383), (16383,)), ((700, 5, 33), (5, 33)), ((0, 64), (64,)),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_layernorm(case, dtype):
    need_gpu()
    shape, wshape = CASES[case]
    say("layernorm", shape, wshape, dtype)
    x, w, b, dy = _make(shape, wshape, dtype, 10 + case)
    eps = 1e-5
    dev = [None if t is None else t.to(DEV) for t in (x, w, b, dy)]
    y = kda.layernorm(dev[0], dev[1], dev[2], eps=eps)
    xh, r, E, lg = _xh_error(x, eps)
    aw = torch.ones(1, dtype=torch.float64) if w is None else w.double().abs()
    ab = torch.zeros(1, dtype=torch.float64) if b is None else b.double().abs()
    say(_within("y", y, ref.norm(x, w, b, eps), E * aw + 4 * U * (xh.abs() * aw + ab), dtype))
    dx, dw, db = kda.layernorm_backward(dev[3], dev[0], dev[1], eps=eps)
    want = ref.norm_backward(dy, x, w, eps)
    t = dy.double() * (w.double() if w is not None else 1.0)
    L = lg + 16
    m = lambda z: z.mean(-1, keepdim=True)  # noqa: E731
    bound = r * (4 * U * t.abs() + L * U * m(t.abs())
                 + xh.abs() * (L * U * m((t * xh).abs()) + m(t.abs() * E))
                 + E * m(t * xh).abs()) + L * U * want[0].abs()
    say(_within("dx", dx, want[0], bound, dtype))
    if w is None:
        assert dw is None and db is None
        return
    over = tuple(range(x.dim() - w.dim()))
    rows = x.numel() // max(x.shape[-1], 1)
    n = (min(rows, 4096) + 32) * U
    s = lambda z: z.sum(over) if over else z  # noqa: E731
    say(_within("dw", dw, want[1], s(dy.double().abs() * E) + n * s((dy.double() * xh).abs()), F32))
    say(_within("db", db, want[2], n * s(dy.double().abs()), F32))


def test_mixed_dtypes_in_place_and_alignment():
    need_gpu()
    say("layernorm mixed")
    x, w, b, dy = _make((40, 4, 128), (4, 128), BF, 1)
    X, W, B, DY = (t.to(DEV) for t in (x, w, b, dy))
    y = kda.layernorm(X, W, B)
    y32 = kda.layernorm(X, W, B, out_dtype=F32)
    assert torch.equal(y32.to(BF), y)
    assert torch.equal(kda.layernorm(X.float(), W, B, out_dtype=BF), y)
    z = X.clone()
    assert kda.layernorm(z, W, B, out=z) is z and torch.equal(z, y)
    # rows that start at any element of an allocation
    buf = torch.empty(40 * 512 + 3, dtype=BF, device=DEV)
    odd = buf[3:].view(40, 4, 128)
    odd.copy_(X)
    assert torch.equal(kda.layernorm(odd, W, B), y)
    g = kda.layernorm_backward(DY, X, W)
    assert all(torch.equal(a, c) for a, c in zip(g, kda.layernorm_backward(DY, odd, W)))
    assert all(torch.equal(a, c) for a, c in zip(g, kda.layernorm_backward(DY, X, W)))
    g32 = kda.layernorm_backward(DY.float(), X, W)
    assert all(torch.equal(a, c) for a, c in zip(g, g32))
    only = kda.layernorm_backward(DY, X, W, want_dbias=False)
    assert only[2] is None and torch.equal(only[1], g[1])


def test_large_means_and_constant_rows():
    """A mean of 1,000 spreads costs no digits beyond its own rounding; a constant row gives
    its bias exactly."""
    need_gpu()
    say("layernorm large means")
    x, w, b, _ = _make((20, 777), (777,), F32, 2, offset=1000.0)
    y = kda.layernorm(x.to(DEV), w.to(DEV), b.to(DEV))
    xh, r, E, _ = _xh_error(x, 1e-5)
    aw = w.double().abs()
    _within("y", y, ref.norm(x, w, b), E * aw + 4 * U * (xh.abs() * aw + b.double().abs()), F32)
    c = torch.full((3, 128), 2.0, device=DEV)
    assert torch.equal(kda.layernorm(c, torch.ones(128, device=DEV), torch.ones(128, device=DEV)),
                       torch.ones(3, 128, device=DEV))


def test_a_bad_row_stays_alone():
    """NaN and infinity in one row reach that row's y and dx only."""
    need_gpu()
    say("layernorm bad rows")
    x, w, b, dy = _make((300, 2, 128), (2, 128), BF, 3)
    X, W, B, DY = (t.to(DEV) for t in (x, w, b, dy))
    y, dx = kda.layernorm(X, W, B), kda.layernorm_backward(DY, X, W)[0]
    X2 = X.clone()
    X2[7, 1, 5] = float("nan")
    X2[9, 0, 127] = float("inf")
    y2, dx2 = kda.layernorm(X2, W, B), kda.layernorm_backward(DY, X2, W)[0]
    keep = torch.ones(300, 2, dtype=torch.bool, device=DEV)
    keep[7, 1] = keep[9, 0] = False
    assert torch.equal(y[keep], y2[keep]) and torch.equal(dx[keep], dx2[keep])
    assert torch.isnan(y2[7, 1]).all()
