"""GPU: layer norm of rows whose spread is small beside their mean, against 64-bit
formulas.

Bounds, in u = 2^-24 per fp32 rounding and with l = log2 d + 10 roundings on the way of
a sum (a thread adds up to 16 values in turn, the rest are pairwise) and of the division
by d.  A = max |x|, c = x - mean, r = 1 / sqrt(var + eps).
  The first mean is off by e1 = l u A at most.  x - mean' is rounded once, relative to
  |c| + e1.  The mean of these differences, which is the error e1, is known to l u of
  their mean absolute value, and taking it off rounds once more:
     e = u (|c| + e1) + l u (mean|c| + e1) + u (|c| + 2 e1)
  The mean square of the differences is var + e1^2 to (l + 2) u of itself, and so is its
  difference with the square of their mean from var; r is off by half of that relative
  to var + eps:
     rel = (l + 4) u (var + 2 e1^2) / (var + eps) + 4 u
  |xh error| <= E = r e + rel |xh|
From E on the bounds of y, dx, dw and db are those of tests/test_gpu_layernorm.py, with
mean(t (x - mean)) formed as a sum of t (x - mean') less e1 times the sum of t: 2 l u e1
mean|t| r more in mean(t xh).
"""
import math

import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import linattn_ref as ref
from tests.gpu_util import DEV, need_gpu, say
from tests.test_gpu_layernorm import _within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = ref.U
EPS = 1e-5


def _bounds(x, w, b, dy):
    """Bounds of y, dx, dw, db and xh's reference, as above."""
    x, dy = x.double(), dy.double()
    d = x.shape[-1]
    m = lambda z: z.mean(-1, keepdim=True)  # noqa: E731
    n = (math.log2(d) + 10) * U
    c = x - m(x)
    var = m(c * c)
    r = 1.0 / torch.sqrt(var + EPS)
    xh = c * r
    e1 = n * x.abs().amax(-1, keepdim=True)
    e = U * (c.abs() + e1) + n * (m(c.abs()) + e1) + U * (c.abs() + 2 * e1)
    rel = (n + 4 * U) * (var + 2 * e1 * e1) / (var + EPS) + 4 * U
    E = r * e + rel * xh.abs()
    aw, ab = w.double().abs(), b.double().abs()
    y = E * aw + 4 * U * (xh.abs() * aw + ab)
    t = dy * w.double()
    L = n + 6 * U
    mt = L * m((t * xh).abs()) + m(t.abs() * E) + 2 * n * e1 * m(t.abs()) * r
    dx = r * (4 * U * t.abs() + L * m(t.abs()) + xh.abs() * mt + E * m(t * xh).abs()) + (
        L + rel) * ref.norm_backward(dy, x, w, EPS)[0].abs()
    over = tuple(range(x.dim() - w.dim()))
    rows = (min(x.numel() // d, 4096) + 32) * U
    dw = (dy.abs() * E).sum(over) + rows * (dy * xh).abs().sum(over)
    return y, dx, dw, rows * dy.abs().sum(over)


def _check(x, w, b, dy):
    dev = [t.to(DEV) for t in (x, w, b, dy)]
    y = kda.layernorm(*dev[:3], eps=EPS)
    dx, dw, db = kda.layernorm_backward(dev[3], dev[0], dev[1], eps=EPS)
    by, bdx, bdw, bdb = _bounds(x, w, b, dy)
    want = ref.norm_backward(dy, x, w, EPS)
    say(_within("y", y, ref.norm(x, w, b, EPS), by, y.dtype),
        _within("dx", dx, want[0], bdx, dx.dtype), _within("dw", dw, want[1], bdw, F32),
        _within("db", db, want[2], bdb, F32))


@pytest.mark.parametrize("d", [3, 33, 128, 200, 1000, 1500, 5003, 5120, 12288, 16383])
def test_constant_rows_give_their_bias(d):
    """A constant row has no spread: xh is 0 to the rounding of its values' differences."""
    need_gpu()
    say("layernorm constant rows", d)
    gen = torch.Generator().manual_seed(d)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = torch.tensor([777.7, 1000.0, 0.1, -53.123, 1e4, 1 / 3]).unsqueeze(1).expand(6, d)
    _check(x.contiguous(), 1 + 0.3 * rnd(d), rnd(d), rnd(6, d))


@pytest.mark.parametrize("d", [100, 777, 4097, 12288])
@pytest.mark.parametrize("mean", [1e3, 3e4])
def test_a_spread_far_below_the_mean(d, mean):
    need_gpu()
    say("layernorm far means", d, mean)
    gen = torch.Generator().manual_seed(d)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (mean + rnd(6, d)).float()
    _check(x, 1 + 0.3 * rnd(d), rnd(d), rnd(6, d))


# x's shape, weight's shape: owners of rows have several and some of them one more, in
# the backward always, in the forward where there are more rows than lanes for the card
MANY = [
    ((70001, 64), (64,)), ((140000, 64), (64,)), ((1500, 96, 128), (96, 128)), ((9001, 250), (250,)),
    ((40000, 250), (250,)),
    ((30011, 1000), (1000,)), ((9001, 1500), (1500,)), ((4500, 2049), (2049,)),
    ((2250, 2, 5003), (2, 5003)), ((1100, 12288), (12288,)),
]


def _in_place(x, w, b, dy):
    """The calls whose output is one of their inputs: (y over x, dx over dy, dx over x)."""
    from gated_delta_rule_58_amd import linattn
    rows, groups, d = linattn._norm_rows(x, w, b)
    dt, s = linattn._dt(x), torch.cuda.current_stream().cuda_stream
    n = kda.layernorm_backward_workspace_bytes(rows, groups, d)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    y = x.clone()
    kda.layernorm(y, w, b, eps=EPS, out=y)
    out = []
    for over in (0, 1):
        args = [dy.clone(), x.clone()]
        dw, db = torch.empty_like(w), torch.empty_like(w)
        assert linattn._fn("kda_layernorm_backward")(
            args[0].data_ptr(), dt, args[1].data_ptr(), dt, w.data_ptr(), groups,
            args[over].data_ptr(), dw.data_ptr(), db.data_ptr(), rows, d, EPS, ws.data_ptr(), n,
            s) == 0
        out.append((args[over], dw, db))
    return y, out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_in_place_over_many_rows(case, dtype):
    """y over x, dx over dy and dx over x, with several rows an owner: the bits of the calls
    with outputs of their own."""
    need_gpu()
    shape, wshape = MANY[case]
    say("layernorm in place", shape, wshape, dtype)
    gen = torch.Generator(device=DEV).manual_seed(case)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    x, dy, w, b = rnd(*shape).to(dtype), rnd(*shape).to(dtype), 1 + 0.3 * rnd(*wshape), rnd(*wshape)
    y = kda.layernorm(x, w, b, eps=EPS)
    g = kda.layernorm_backward(dy, x, w, eps=EPS)
    y2, outs = _in_place(x, w, b, dy)
    assert torch.equal(y, y2)
    for out in outs:
        for a, c in zip(g, out):
            assert torch.equal(a, c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows_an_owner(case, dtype):
    """Values where an owner walks down several rows: the next row's load, the turns of the
    sums' LDS buffers, the running sums of dw and db.  The 64-bit formulas run on the device."""
    need_gpu()
    shape, wshape = MANY[case]
    say("layernorm many rows", shape, wshape, dtype)
    gen = torch.Generator(device=DEV).manual_seed(100 + case)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    x = (1.5 * rnd(*shape) + rnd(*shape[:-1], 1)).to(dtype)
    dy, w, b = rnd(*shape).to(dtype), 1 + 0.3 * rnd(*wshape), rnd(*wshape)
    y = kda.layernorm(x, w, b, eps=EPS)
    dx, dw, db = kda.layernorm_backward(dy, x, w, eps=EPS)
    by, bdx, bdw, bdb = _bounds(x, w, b, dy)
    want = ref.norm_backward(dy, x, w, EPS)
    for name, got, ref64, bound in (("y", y, ref.norm(x, w, b, EPS), by), ("dx", dx, want[0], bdx),
                                    ("dw", dw, want[1], bdw), ("db", db, want[2], bdb)):
        say(_within(name, got, ref64.cpu(), bound.cpu(), got.dtype))


@pytest.mark.parametrize("d", [777, 1000, 5120, 12288])
def test_rows_whose_squares_overflow(d):
    """Values whose differences' squares are beyond fp32: 1 / sqrt(inf) is 0, and the row
    gives its bias, not NaN."""
    need_gpu()
    say("layernorm overflow", d)
    x = torch.full((4, d), 1e32, device=DEV)
    x[1] = -3.3e33
    x[2, ::2] *= -1.0
    x[3, 5] = 1e30
    w, b = torch.ones(d, device=DEV) * 1.5, torch.randn(d, device=DEV)
    assert torch.equal(kda.layernorm(x, w, b), b.expand(4, d))
