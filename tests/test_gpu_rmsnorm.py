"""GPU: RMS norm forward (with the residual, to 8 bits) and backward against 64-bit formulas;
the bounds are derived in gatedrec_ref.py."""
import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import gatedrec_ref as ref
from tests.gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

CASES = [  # x's shape, weight's shape
    ((1, 1), (1,)), ((5, 1), None), ((3, 2), (2,)), ((7, 9), (9,)), ((2, 63), (63,)),
    ((9, 64), (64,)), ((4, 65), None), ((50, 3, 128), (3, 128)), ((50, 3, 128), (128,)),
    ((6, 5, 129), (5, 129)), ((1, 2, 64), (2, 64)), ((33, 255), (255,)), ((11, 4, 256), (4, 256)),
    ((17, 511), (511,)), ((6, 1000), (1000,)), ((5, 1025), (1025,)), ((3, 2, 2048), (2, 2048)),
    ((4, 4095), (4095,)), ((3, 4097), (4097,)), ((3, 8192), (8192,)), ((2, 8193), None),
    ((2, 16384), (16384,)), ((2, 16383), (16383,)), ((700, 5, 33), (5, 33)), ((0, 64), (64,)),
    ((1, 12288), (12288,)), ((900, 640), (640,)),
]


def _make(shape, wshape, dtype, seed, rdt=None):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (rnd(*shape) * 1.5).to(dtype)
    w = None if wshape is None else 1 + 0.3 * rnd(*wshape)
    return x, w, None if rdt is None else (rnd(*shape) * 2).to(rdt), rnd(*shape).to(dtype)


def _scales(y, per):
    """Exact scales of y [..., d] for each `per` columns (0: the row)."""
    d = y.shape[-1]
    n = per or d
    k = -(-d // n)
    v = torch.nn.functional.pad(y.abs(), (0, k * n - d)).unflatten(-1, (k, n))
    return v.amax(-1) / 448, n


@pytest.mark.parametrize("dtype, rdt", [(BF, None), (F32, None), (BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_rmsnorm(case, dtype, rdt):
    need_gpu()
    shape, wshape = CASES[case]
    say("rmsnorm", shape, wshape, dtype, rdt)
    x, w, res, dy = _make(shape, wshape, dtype, 20 + case, rdt)
    eps = 1e-5
    X, W, RES, DY = (None if t is None else t.to(DEV) for t in (x, w, res, dy))
    y, s = kda.rmsnorm(X, W, RES, eps)
    stored = ref.rms_sum(x, res)
    if res is None:
        assert s is None
    else:
        assert s.dtype == rdt and torch.equal(s.cpu(), stored)
    want, bound = ref.rmsnorm(stored, w, eps)
    say(ref.within("y", y, want, bound, dtype))
    # 8 bits: half a step of e4m3 (2^-4 of the value, at least half of its least step, 2^-10) of
    # what the scale makes of y, with y's and the scale's own errors
    for per in (128, 0):
        q, scales, s2 = kda.rmsnorm_e4m3(X, W, RES, eps, scale_group=per)
        assert q.dtype == E4 and (s2 is None if s is None else torch.equal(s2, s))
        ws, n = _scales(want, per)
        eb, _ = _scales(bound, per)
        ref.within("scales", scales, ws, eb + 2 * ref.U * ws, F32)
        full = ws.repeat_interleave(n, -1)[..., :shape[-1]]
        got = q.cpu().double()
        v = want / full
        rel = 2 ** -4 * (1 + 1e-3)
        off = (got - v).abs() - torch.maximum(rel * v.abs(), torch.full_like(v, 2 ** -10))
        assert not got.numel() or off.max() <= 448 * 64 * ref.U
        assert not got.numel() or got.abs().amax() == 448
    dx, dw = kda.rmsnorm_backward(DY, X if s is None else s, W, eps=eps)
    wdx, edx, wdw, edw = ref.rmsnorm_backward(dy, stored, w, None, eps)
    say(ref.within("dx", dx, wdx, edx, stored.dtype))
    if w is None:
        assert dw is None
    else:
        say(ref.within("dw", dw, wdw, edw, F32))
    if res is not None and res.dtype == dtype:
        dx2, dw2 = kda.rmsnorm_backward(DY, s, W, d_residual=RES, eps=eps)
        wdx, edx, _, _ = ref.rmsnorm_backward(dy, stored, w, res, eps)
        ref.within("dx", dx2, wdx, edx, dtype)
        assert dw is None or torch.equal(dw, dw2)


def test_e4m3_is_the_nearest_value():
    """Every quotient that the kernel forms rounds like torch's own conversion: rows whose scale
    is 1 (their largest value is 448) come out as x itself converted."""
    need_gpu()
    say("rmsnorm e4m3 rounding")
    gen = torch.Generator().manual_seed(1)
    y = (torch.rand(64, 128, generator=gen) * 2 - 1) * 448 * torch.exp2(
        -12 * torch.rand(64, 128, generator=gen))
    y[:, 0] = 448.0
    # weight = y with all of x alike: x / rms(x) = 1 for eps = 0 (powers of two: exactly)
    x = torch.full((64, 64, 128), 2.0)
    q, scales, _ = kda.rmsnorm_e4m3(x.to(DEV), y.to(DEV), eps=0.0)
    assert (scales == 1.0).all()
    want = y.to(E4).float()
    assert torch.equal(q.float().cpu(), want.expand(64, 64, 128))


def test_in_place_strides_and_alignment():
    need_gpu()
    say("rmsnorm in place")
    x, w, res, dy = _make((40, 4, 128), (4, 128), BF, 1, BF)
    X, W, RES, DY = (t.to(DEV) for t in (x, w, res, dy))
    y, s = kda.rmsnorm(X, W, RES)
    y32, _ = kda.rmsnorm(X, W, RES, out_dtype=F32)
    assert torch.equal(y32.to(BF), y)
    x2, r2 = X.clone(), RES.clone()
    y2, s2 = kda.rmsnorm(x2, W, r2, out=x2, residual_out=r2)
    assert y2 is x2 and s2 is r2 and torch.equal(y2, y) and torch.equal(s2, s)
    x3 = X.clone()
    y3, s3 = kda.rmsnorm(x3, W, RES, residual_out=x3)
    assert s3 is x3 and torch.equal(s3, s) and torch.equal(y3, y)
    q, sc, _ = kda.rmsnorm_e4m3(X, W, RES)
    # tokens of a fused projection, and rows that start at any element
    wide = torch.empty(40, 4 * 128 + 37, dtype=BF, device=DEV)
    col = wide[:, 5:5 + 512].unflatten(1, (4, 128))
    col.copy_(X)
    assert torch.equal(kda.rmsnorm(col, W, RES)[0], y)
    q2, sc2, _ = kda.rmsnorm_e4m3(col, W, RES)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(sc2, sc)
    a, b = kda.rmsnorm_backward(DY, X, W, RES), kda.rmsnorm_backward(DY, col, W, RES)
    assert all(torch.equal(p, r) for p, r in zip(a, b))
    buf = torch.empty(40 * 512 + 3, dtype=BF, device=DEV)
    odd = buf[3:].view(40, 4, 128)
    odd.copy_(X)
    assert torch.equal(kda.rmsnorm(odd, W, RES)[0], y)
    flat = X.view(160, 128)
    assert torch.equal(kda.rmsnorm(flat[::2], W[0])[0], kda.rmsnorm(flat[::2].contiguous(), W[0])[0])
    with pytest.raises(ValueError, match="contiguous"):
        kda.rmsnorm(X[:, ::2], W[0])
    with pytest.raises(kda.KdaError):
        kda.rmsnorm(col, W, out=col.as_strided(X.shape, X.stride(), col.storage_offset()))


def test_bad_and_empty_rows():
    """A NaN or an infinity stays in its row; a row of zeros gives zeros."""
    need_gpu()
    say("rmsnorm bad rows")
    x, w, res, dy = _make((300, 2, 128), (2, 128), BF, 3)
    X, W, DY = (t.to(DEV) for t in (x, w, dy))
    keep = torch.ones(300, 2, dtype=torch.bool, device=DEV)
    X2 = X.clone()
    X2[7, 1, 5] = float("nan")
    X2[9, 0, 127] = float("inf")
    X2[11, 1] = 0.0
    keep[7, 1] = keep[9, 0] = keep[11, 1] = False
    for per in (128, 0):
        q, sc, _ = kda.rmsnorm_e4m3(X, W, scale_group=per)
        q2, sc2, _ = kda.rmsnorm_e4m3(X2, W, scale_group=per)
        assert torch.equal(q.float()[keep], q2.float()[keep]) and torch.equal(sc[keep], sc2[keep])
        assert torch.isnan(q2.float()[7, 1]).all() and torch.isnan(sc2[7, 1]).all()
        assert torch.isnan(sc2[9, 0]).all() and torch.isnan(q2.float()[9, 0, 127])
        assert not q2.float()[11, 1].any() and 0 < sc2[11, 1] < 1e-30
    y, dx = kda.rmsnorm(X, W)[0], kda.rmsnorm_backward(DY, X, W)[0]
    y2, dx2 = kda.rmsnorm(X2, W)[0], kda.rmsnorm_backward(DY, X2, W)[0]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(dx[keep], dx2[keep])
    assert torch.isnan(y2[7, 1]).all() and not y2[11, 1].any() and torch.isfinite(dx2[11, 1]).all()


@pytest.mark.parametrize("shape, wshape", [((20000, 128), (128,)), ((3000, 7, 64), (7, 64)),
                                           ((5000, 1024), (1024,)), ((3000, 4096), (4096,)),
                                           ((1500, 8192), (8192,)), ((1300, 12288), (12288,))])
def test_owners_walk_down_rows(shape, wshape):
    """More rows than owners: each owner walks several, forward and backward."""
    need_gpu()
    say("rmsnorm walks", shape)
    gen = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(*shape, generator=gen, device=DEV).to(BF)
    res = torch.randn(*shape, generator=gen, device=DEV).to(BF)
    dy = torch.randn(*shape, generator=gen, device=DEV).to(BF)
    w = 1 + 0.1 * torch.randn(*wshape, generator=gen, device=DEV)
    y, s = kda.rmsnorm(x, w, res)
    q, sc, s2 = kda.rmsnorm_e4m3(x, w, res, scale_group=0)
    assert torch.equal(s, x + res) and torch.equal(s, s2)
    sd = s.double()
    r = 1 / torch.sqrt((sd * sd).mean(-1, keepdim=True) + 1e-5)
    want = sd * r * w.double()
    assert ((y.double() - want).abs() <= (2 ** -8 + 1e-5) * want.abs()).all()
    assert ((sc.double() - want.abs().amax(-1, keepdim=True) / 448).abs() <= 1e-5 * sc).all()
    assert ((q.double() * sc - want).abs() <= 2 ** -4 * 1.01 * want.abs() + sc * 2 ** -10 * 1.01).all()
    dx, dw = kda.rmsnorm_backward(dy, s, w, d_residual=res)
    t = dy.double() * w.double()
    xh = sd * r
    wdx = r * (t - xh * (t * xh).mean(-1, keepdim=True)) + res.double()
    # fp32: |dx| up to 10, its parts within 30 roundings of 2^-24
    assert ((dx.double() - wdx).abs() <= 2 ** -8 * wdx.abs() + 2e-5).all()
    over = tuple(range(dy.dim() - w.dim()))
    wdw, adw = (dy.double() * xh).sum(over), (dy.double() * xh).abs().sum(over)
    rows = x.numel() // w.numel()
    assert ((dw.double() - wdw).abs() <= (min(rows, 4096) + 64) * ref.U * adw).all()
