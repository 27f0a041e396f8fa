"""GPU: the linear attention over sequences of many segments, cut and whole, and at the
sizes it is made for.

dg of a long sequence.  The elementwise bound of tests/linattn_ref.py adds up every later
token's terms and grows with the length beyond dg itself.  Here dg is held to its size
too: the library states an error of 1e-6 to 5e-6 of dg's norm over a call.  A part of a
call has fewer terms to average over and may lie in a quiet stretch, so per (sequence,
head) the bound is four times the worst stated value, 2e-5 of the norm, and over the 64
tokens before a border of two segments (512 tokens apart at least) the same, relative to
the larger of the sequence's and the stretch's root mean square.  What a wrong border
would do is 1e-1 and more: the value that is handed on is there times e^g, the sum of a
few thousand such products."""
import math

import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import linattn_ref as ref
from tests.gpu_util import DEV, need_gpu, sample_heads, say
from tests.test_gpu_linattn import _cu, _draw, _gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DG = 2e-5


def _rms(x):
    return x.double().square().mean(0).sqrt()


def _check_dg(got, want, cu):
    """got, want [T, H]; per sequence and head, and before every multiple of 64 tokens that
    a border can be at."""
    got = got.detach().cpu().double()
    worst = 0.0
    for a, b in zip(cu, cu[1:]):
        if b - a < 256:
            continue
        size = _rms(want[a:b])
        worst = max(worst, (_rms(got[a:b] - want[a:b]) / (DG * size)).max().item())
        for t in range(a + 64, b + 1, 64):
            part = torch.maximum(size, _rms(want[t - 64:t]))
            worst = max(worst, (_rms(got[t - 64:t] - want[t - 64:t]) / (DG * part)).max().item())
    assert math.isfinite(worst) and worst <= 1.0, "dg: %.3g times its bound" % worst
    return worst


def _check_backward(got, q, k, v, g, cu, do, S0, dS, scale):
    """ref.check_backward, with dg's own bound beside it."""
    want = ref.backward(q, k, v, g, cu, do, S0, dS, scale)
    size = ref.backward(*[x.abs().double() for x in (q, k, v)], g, cu, do.abs(), S0.abs(), dS.abs(),
                        scale, signs=False)
    wide = q.dtype == F32
    rel = ref.rel_of(q, v, cu, 3)
    rels = [rel, rel, ref.rel_of(q, v, cu, 3 if wide else 1 if got[2].dtype == BF else 2),
            rel + 256 * ref.U, rel]
    worst = [ref.check(n, x, w, s, r, x.dtype)
             for n, x, w, s, r in zip(("dq", "dk", "dv", "dg", "dS0"), got, want, size, rels)]
    if g.dim() == 2:
        return worst + [_check_dg(got[3], want[3], cu)]
    # one value a head, the sum of every token's: at most the sum of their errors
    each = ref.backward(q, k, v, g.expand(cu[-1], g.shape[0]), cu, do, S0, dS, scale)[3]
    bound = DG * sum((b - a) * _rms(each[a:b]) for a, b in zip(cu, cu[1:]) if b > a)
    bound = bound + ref.U * want[3].abs()
    err = ((got[3].cpu().double() - want[3]).abs() / bound).max().item()
    assert err <= 1.0, "dg: %.3g times its bound" % err
    return worst + [err]


def _terms(cu, H, dk, dv, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    do = torch.randn(cu[-1], H, dv, generator=gen).to(dtype)
    return do, torch.randn(len(cu) - 1, H, dk, dv, generator=gen)


# lens, H, Hk, dk, dv: one head, cut into segments of 4 chunks; a batch of three that is
# cut; grouped heads, cut; sequences walked whole with borders of 32 chunks
LONG = [
    ([2300, 30], 1, 1, 128, 128), ([5000, 0, 900], 2, 2, 64, 128), ([2600], 6, 2, 128, 64),
    ([2100, 0, 2050], 24, 12, 64, 64),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay", ["mild", "head"])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_backward_of_many_segments(case, decay, dtype):
    """With the host's lengths and without: these batches are cut (or not) alike, and give
    the same bits."""
    need_gpu()
    lens, H, Hk, dk, dv = LONG[case]
    say("linattn long backward", LONG[case], decay, dtype)
    q, k, v, g, cu, S0 = _draw(lens, H, Hk, dk, dv, dtype, decay, 60 + case)
    do, dS = _terms(cu, H, dk, dv, dtype, 70 + case)
    dev = _gpu(q, k, v, g, do, S0, dS)
    got, other = (kda.linattn_chunk_prefill_backward(
        *dev[:5], **kw, initial_state=dev[5], d_final_state=dev[6], scale=0.6)
        for kw in (_cu(cu), dict(cu_seqlens=_cu(cu)["cu_seqlens"])))
    say(_check_backward(got, q, k, v, g, cu, do, S0, dS, 0.6))
    for x, y in zip(got, other):
        assert torch.equal(x, y)


def test_the_dg_bound_sees_a_lost_border_factor():
    """The bound of this file refuses a dg whose segments hand <S, dL/dS> on without the
    decay of the token behind the border (made on the reference)."""
    lens, H = [2100], 2
    q, k, v, g, cu, S0 = _draw(lens, H, H, 64, 64, BF, "mild", 500)
    do, dS = _terms(cu, H, 64, 64, BF, 4)
    want = ref.backward(q, k, v, g, cu, do, S0, dS)[3]
    bad = want.clone()
    t = 2048  # the border of the first segment of 32 chunks: dg_{t-1} holds e^{g_t} <S, D>
    a = torch.exp(g[t].double())
    handed = want[t]  # a <D_t, S_{t-1}> = the pairs over the border
    bad[:t] += (handed / a - handed)[None]
    with pytest.raises(AssertionError, match="dg"):
        _check_dg(bad, want, cu)


@pytest.mark.parametrize("decay", ["mild", "head"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sdt", [F32, BF])
def test_cut_prefill_into_a_pool_in_place(sdt, dtype, decay):
    """A batch that is cut into segments, over a pool of slots in place, one entry outside
    it, and with and without the host's lengths."""
    need_gpu()
    say("linattn cut prefill, pool", sdt, dtype, decay)
    lens, H, Hk, idx = [4300, 0, 700, 40], 2, 1, [5, 2, -1, 0]
    q, k, v, g, cu, _ = _draw(lens, H, Hk, 128, 128, dtype, decay, 80, state=False)
    assert kda.linattn_chunk_prefill_workspace_bytes(cu[-1], 4, H) > 0
    gen = torch.Generator().manual_seed(81)
    pool = torch.randn(7, H, 128, 128, generator=gen).to(sdt)
    S0 = torch.stack([pool[i] if i >= 0 else torch.zeros_like(pool[0]) for i in idx])
    want, wS = ref.forward(q, k, v, g, cu, S0, 0.9)
    _, aS = ref.forward(q.abs(), k.abs(), v.abs(), g, cu, S0.abs(), 0.9)
    ind = torch.tensor(idx, dtype=torch.int32, device=DEV)
    dev = _gpu(q, k, v, g)
    for kw in (_cu(cu), dict(cu_seqlens=_cu(cu)["cu_seqlens"])):
        P = pool.to(DEV)
        o, same = kda.linattn_chunk_prefill(*dev, **kw, initial_state=P, final_state=P,
                                            state_indices=ind, scale=0.9)
        assert same is P
        say(ref.check_forward(o, None, q, k, v, g, cu, S0, 0.9))
        for n, s in enumerate(idx):
            if s >= 0:
                ref.check("pool", P[s:s + 1], wS[n:n + 1], aS[n:n + 1], ref.rel_of(q, v, cu, 3), sdt)
        for s in (1, 3, 4, 6):
            assert torch.equal(P[s].cpu(), pool[s])


def _slices(h, H, Hk, *ts):
    """The q/k head that heads h read (one group), as tensors of a smaller problem."""
    grp = H // Hk
    out = []
    for t in ts:
        if t is None:
            out.append(None)
        elif t.dim() >= 3 and t.shape[1] == Hk and Hk != H:
            out.append(t[:, h // grp:h // grp + 1].cpu())
        else:
            lo = h // grp * grp
            out.append((t[:, lo:lo + grp] if t.dim() > 1 else t[lo:lo + grp]).cpu())
    return out


@pytest.mark.parametrize("H, Hk, decay", [(96, 96, "mild"), (96, 24, "head")])
def test_a_layer_at_its_size(H, Hk, decay):
    """4,096 tokens x 96 heads of 128 dims, forward and backward: sampled heads whole."""
    need_gpu()
    say("linattn layer at its size", H, Hk, decay)
    T = 4096
    q, k, v, g, cu, S0 = _draw([T], H, Hk, 128, 128, BF, decay, 90)
    do, dS = _terms(cu, H, 128, 128, BF, 91)
    dev = _gpu(q, k, v, g, do, S0, dS)
    o, S = kda.linattn_chunk_prefill(*dev[:4], initial_state=dev[5], scale=0.3)
    got = kda.linattn_chunk_prefill_backward(*dev[:5], initial_state=dev[5], d_final_state=dev[6],
                                             scale=0.3)
    for h in sample_heads(H, 2, 5):
        q1, k1, v1, g1, do1, S1, dS1 = _slices(h, H, Hk, q, k, v, g, do, S0, dS)
        o1, Sf1, *got1 = _slices(h, H, Hk, o, S, *got)
        say(ref.check_forward(o1, Sf1, q1, k1, v1, g1, cu, S1, 0.3))
        say(_check_backward(got1, q1, k1, v1, g1, cu, do1, S1, dS1, 0.3))


def test_a_long_document_at_its_size():
    """131,072 tokens x 16 heads, 2 of q/k, one decay a head, cut into segments.  A state
    forgets: with decays of at most e^-0.02 a token what lies 2,500 tokens back is e^-50 of
    itself, so stretches of the document are checked from zeros."""
    need_gpu()
    say("linattn document at its size")
    T, H, Hk = 131072, 16, 2
    gen = torch.Generator(device=DEV).manual_seed(92)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = unit(r(T, Hk, 128)).to(BF), unit(r(T, Hk, 128)).to(BF)
    v = r(T, H, 128).to(BF)
    g = -0.02 - 0.3 * torch.rand(H, generator=gen, device=DEV)
    o, S = kda.linattn_chunk_prefill(q, k, v, g, scale=0.7)
    back, n = 2500, 200
    for t in (64 * 64 * 3 + 10, 70000, T):
        lo, h = t - back - n, (t // 7) % H
        q1, k1, v1, g1, o1, S1 = _slices(h, H, Hk, q[lo:t], k[lo:t], v[lo:t], g, o[lo:t], S)
        want, wS = ref.forward(q1, k1, v1, g1, [0, back + n], None, 0.7)
        size, aS = ref.forward(q1.abs(), k1.abs(), v1.abs(), g1, [0, back + n], None, 0.7)
        rel = ref.rel_of(q1, v1, [0, T], 1)
        say(ref.check("o", o1[back:], want[back:], size[back:], rel, BF))
        if t == T:
            say(ref.check("state", S1, wS, aS, ref.rel_of(q1, v1, [0, T], 3), F32))
