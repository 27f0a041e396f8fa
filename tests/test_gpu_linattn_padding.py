"""GPU: batches whose last sequence ends before the last row (cu_seqlens without the
host's copy), forward and backward: what the rows behind it hold reaches nothing, and
what the binding returns for them is zeros."""
import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import linattn_ref as ref
from tests.gpu_util import DEV, need_gpu, say
from tests.test_gpu_linattn import _draw, _gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _poisoned(monkeypatch):
    """torch.empty gives NaN: memory that nothing wrote is seen."""
    empty = torch.empty

    def nans(*a, **kw):
        t = empty(*a, **kw)
        return t.fill_(float("nan")) if t.is_floating_point() else t.fill_(255)

    monkeypatch.setattr(torch, "empty", nans)


def _padded(lens, behind, H, Hk, dk, dv, dtype, decay, seed):
    """A draw whose last `behind` rows belong to no sequence and hold NaN."""
    q, k, v, g, cu, S0 = _draw(lens + [behind], H, Hk, dk, dv, dtype, decay, seed)
    end = cu[-2]
    for t in (q, k, v) + ((g,) if decay != "head" else ()):
        t[end:] = float("nan")
    dev_cu = torch.tensor(cu[:-1], dtype=torch.int32, device=DEV)
    return q, k, v, g, cu[:-1], S0[:-1], end, dev_cu


def _live(end, *ts):
    return [t[:end] if t.dim() > 1 else t for t in ts]


@pytest.mark.parametrize("H, Hk", [(4, 4), (4, 2)])
@pytest.mark.parametrize("decay", ["mild", "head"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_behind_the_last_sequence_are_zeros(H, Hk, decay, dtype, monkeypatch):
    need_gpu()
    say("linattn rows behind", H, Hk, decay, dtype)
    q, k, v, g, cu, S0, end, dev_cu = _padded([70, 0, 41], 29, H, Hk, 128, 64, dtype, decay, 31)
    gen = torch.Generator().manual_seed(8)
    do = torch.randn(q.shape[0], H, 64, generator=gen).to(dtype)
    do[end:] = float("nan")
    dS = torch.randn(3, H, 128, 64, generator=gen)
    dev = _gpu(q, k, v, g, do, S0, dS)
    _poisoned(monkeypatch)
    o, S = kda.linattn_chunk_prefill(*dev[:4], cu_seqlens=dev_cu, initial_state=dev[5])
    got = kda.linattn_chunk_prefill_backward(*dev[:5], cu_seqlens=dev_cu, initial_state=dev[5],
                                             d_final_state=dev[6])
    for t in (o,) + got[:3] + (() if decay == "head" else (got[3],)):
        assert torch.equal(t[end:], torch.zeros_like(t[end:]))
    q, k, v, g, do = _live(end, q, k, v, g, do)
    say(ref.check_forward(o[:end], S, q, k, v, g, cu, S0))
    got = _live(end, *got[:4]) + [got[4]]
    say(ref.check_backward(got, q, k, v, g, cu, do, S0, dS))


def test_rows_behind_stay_as_they_were_in_given_memory():
    """The library itself writes the rows of sequences only, the gradients' too."""
    need_gpu()
    say("linattn backward into given memory")
    from gated_delta_rule_58_amd import linattn
    H, Hk, T = 4, 2, 140
    q, k, v, g, cu, S0, end, dev_cu = _padded([70, 0, 41], 29, H, Hk, 128, 128, BF, "mild", 32)
    dev = _gpu(q, k, v, g, torch.randn(T, H, 128, generator=torch.Generator().manual_seed(9)).to(BF))
    outs = [torch.full(s, 7.0, dtype=d, device=DEV)
            for s, d in (((T, Hk, 128), BF), ((T, Hk, 128), BF), ((T, H, 128), BF), ((T, H), F32))]
    n = kda.linattn_chunk_prefill_backward_workspace_bytes(T, 3, H, Hk)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    st = linattn._fn("kda_linattn_chunk_prefill_backward")(
        dev[0].data_ptr(), Hk * 128, dev[1].data_ptr(), Hk * 128, dev[2].data_ptr(), H * 128, 1,
        dev[3].data_ptr(), T * H, dev_cu.data_ptr(), None, 3, None, dev[4].data_ptr(), 1, None,
        *[t.data_ptr() for t in outs[:3]], 1, outs[3].data_ptr(), None, T, H, Hk, 128, 128, 1.0,
        ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want = kda.linattn_chunk_prefill_backward(*dev, cu_seqlens=dev_cu)
    for t, w in zip(outs, want):
        assert torch.all(t[end:] == 7.0)
        assert torch.equal(t[:end], w[:end])


def test_gradients_of_many_sequences_without_host_lengths():
    """65,536 sequences that could each hold all 262,144 tokens as far as the host knows:
    the same bits as with the host's lengths, and the reference's values."""
    need_gpu()
    say("linattn many sequences")
    N, T = 1 << 16, 1 << 18
    gen = torch.Generator().manual_seed(33)
    cu = torch.cat([torch.zeros(1, dtype=torch.long),
                    torch.randint(0, 9, (N,), generator=gen).cumsum(0)]).clamp(max=T)
    cu[-1] = T
    cu = cu.to(torch.int32)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v, do = (rnd(T, 1, 64).to(BF) * 0.3 for _ in range(4))
    for g in (-0.3 * torch.rand(T, 1, generator=gen), -0.3 * torch.rand(1, generator=gen)):
        dev = _gpu(q, k, v, g, do, cu)
        run = lambda **kw: kda.linattn_chunk_prefill_backward(  # noqa: E731
            *dev[:5], cu_seqlens=dev[5], want_d_initial_state=False, **kw)
        a, b = run(), run(cu_seqlens_host=cu)
        for x, y in zip(a[:4], b[:4]):
            assert torch.equal(x, y)
        for n0 in (0, 40000, N - 40):  # a few neighbouring sequences
            c = [int(x) for x in cu[n0:n0 + 41]]
            lo, hi = c[0], c[-1]
            got = [x[lo:hi] for x in a[:3]] + [a[3][lo:hi] if g.dim() == 2 else None]
            ref.check_backward(got, q[lo:hi], k[lo:hi], v[lo:hi],
                               g[lo:hi] if g.dim() == 2 else g, [x - lo for x in c], do[lo:hi])


@pytest.mark.parametrize("lens", [[3000, 0, 0, 100], [5, 0, 2100, 64, 0, 4097], [0, 0, 7], [4500]])
@pytest.mark.parametrize("decay", ["mild", "head"])
def test_decay_gradients_with_and_without_host_lengths(lens, decay):
    """Several segments a sequence, empty sequences between: bit for bit the same dg."""
    need_gpu()
    say("linattn host lengths", lens, decay)
    q, k, v, g, cu, S0 = _draw(lens, 40, 40, 64, 64, BF, decay, 34)
    gen = torch.Generator().manual_seed(35)
    do = torch.randn(cu[-1], 40, 64, generator=gen).to(BF)
    dS = torch.randn(len(lens), 40, 64, 64, generator=gen)
    dev = _gpu(q, k, v, g, do, S0, dS)
    h = torch.tensor(cu, dtype=torch.int32)
    run = lambda **kw: kda.linattn_chunk_prefill_backward(  # noqa: E731
        *dev[:5], cu_seqlens=h.to(DEV), initial_state=dev[5], d_final_state=dev[6], **kw)
    for x, y in zip(run(), run(cu_seqlens_host=h)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("end", [-3, 0, 1, 77, 499, 500, 700])
def test_zero_rows_behind(end):
    """Rows from cu_seqlens[N] on, of every row size and alignment, and nothing else."""
    need_gpu()
    say("zero rows behind", end)
    T = 500
    cu = torch.tensor([0, 7, end], dtype=torch.int32, device=DEV)
    odd = torch.full((T * 6 + 2,), 7.0, dtype=BF, device=DEV)
    ts = [torch.full((T, 3, 128), 7.0, dtype=BF, device=DEV), torch.full((T, 5), 7.0, device=DEV),
          odd[2:].view(T, 6), torch.full((T, 4000), 7.0, device=DEV)]
    kda.zero_rows_behind(cu, *ts)
    cut = min(max(end, 0), T)
    for t in ts:
        assert torch.all(t[:cut] == 7.0) and torch.all(t[cut:] == 0.0)
    assert torch.all(odd[:2] == 7.0)
    kda.zero_rows_behind(cu, torch.empty(0, 4, device=DEV))


def test_rows_behind_in_a_replayed_graph():
    """Lengths that change between replays: each replay clears what lies behind its own."""
    need_gpu()
    say("linattn rows behind, graph")
    q, k, v, g, cu, S0 = _draw([100, 60], 2, 2, 128, 128, BF, "mild", 36)
    dev = _gpu(q, k, v, g, torch.ones(160, 2, 128, dtype=BF))
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)

    def run():
        return (kda.linattn_chunk_prefill(*dev[:4], cu_seqlens=cu)[0],
                ) + kda.linattn_chunk_prefill_backward(*dev, cu_seqlens=cu)[:4]

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = run()
    for end in (160, 120, 150, 101):
        cu[2] = end
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y) and not x[end:].any()


@pytest.mark.parametrize("cu", [[5, 30, 90], [-4, 200, 300], [60, 20, 90], [0, 140, 70], [200, 300, 500]])
def test_lengths_out_of_order_stay_inside_the_tensors(cu):
    """Device lengths that no host copy was checked for: ranges are clamped, rows of no
    sequence stay as they were, and what lies before and behind the tensors too."""
    need_gpu()
    say("linattn bad device lengths", cu)
    from gated_delta_rule_58_amd import linattn
    H, Hk, T = 4, 2, 140
    q, k, v, g, _, _ = _draw([T], H, Hk, 128, 64, BF, "mild", 37)
    do = torch.randn(T, H, 64, generator=torch.Generator().manual_seed(38)).to(BF)
    dev = _gpu(q, k, v, g, do)
    dev_cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    shapes = [((Hk, 128), BF), ((Hk, 128), BF), ((H, 64), BF), ((H,), F32), ((H, 64), BF)]
    whole = [torch.full((T + 128,) + s, 7.0, dtype=d, device=DEV) for s, d in shapes]
    outs = [w[64:64 + T] for w in whole]
    n = kda.linattn_chunk_prefill_backward_workspace_bytes(T, 2, H, Hk, 128, 64)
    ws = torch.full((n + 4096,), 255, dtype=torch.uint8, device=DEV)
    st = linattn._fn("kda_linattn_chunk_prefill_backward")(
        dev[0].data_ptr(), Hk * 128, dev[1].data_ptr(), Hk * 128, dev[2].data_ptr(), H * 64, 1,
        dev[3].data_ptr(), T * H, dev_cu.data_ptr(), None, 2, None, dev[4].data_ptr(), 1, None,
        *[t.data_ptr() for t in outs[:3]], 1, outs[3].data_ptr(), None, T, H, Hk, 128, 64, 1.0,
        ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    kda.linattn_chunk_prefill(*dev[:4], cu_seqlens=dev_cu, out=outs[4])
    assert torch.all(ws[n:] == 255)
    clamp = lambda x: min(max(x, 0), T)  # noqa: E731
    mine = torch.zeros(T, dtype=torch.bool, device=DEV)
    for a, b in zip(cu, cu[1:]):
        mine[clamp(a):max(clamp(b), clamp(a))] = True
    for w, t in zip(whole, outs):
        assert torch.all(w[:64] == 7.0) and torch.all(w[64 + T:] == 7.0)
        if cu == sorted(cu):
            assert torch.all(t[~mine] == 7.0)
            assert torch.isfinite(t[mine]).all()
