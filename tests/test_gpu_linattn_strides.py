"""GPU: strided q, k and v in the backward and the decode, calls at the same time, and
graphs that share a workspace."""
import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import linattn_ref as ref
from tests.gpu_util import DEV, need_gpu, say
from tests.test_gpu_linattn import _cu, _draw, _gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _fused(q, k, v, pad):
    """q, k and v as slices of one projection whose other columns are NaN."""
    T, Hk, d = q.shape
    H = v.shape[1]
    whole = torch.full((T, (2 * Hk + H) * d + pad), float("nan"), dtype=q.dtype)
    at = [0, Hk * d, 2 * Hk * d, (2 * Hk + H) * d]
    parts = []
    w = whole.to(DEV)
    for t, a, b in zip((q, k, v), at, at[1:]):
        p = w[:, a:b].unflatten(1, (t.shape[1], d))
        p.copy_(t)
        parts.append(p)
    return parts


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens, H, Hk", [([77, 100, 1], 4, 2), ([2300], 2, 2)])
def test_backward_of_strided_inputs(dtype, lens, H, Hk):
    """Bit for bit the dense call; the second batch is cut into segments."""
    need_gpu()
    say("linattn backward strides", dtype, lens)
    q, k, v, g, cu, S0 = _draw(lens, H, Hk, 128, 128, dtype, "mild", 51)
    do = torch.randn(cu[-1], H, 128, generator=torch.Generator().manual_seed(52)).to(dtype)
    dev = _gpu(q, k, v, g, do, S0)
    a = kda.linattn_chunk_prefill_backward(*dev[:5], **_cu(cu), initial_state=dev[5])
    b = kda.linattn_chunk_prefill_backward(*_fused(q, k, v, 24), *dev[3:5], **_cu(cu),
                                           initial_state=dev[5])
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    if len(lens) > 1:
        say(ref.check_backward(b, q, k, v, g, cu, do, S0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [3, 200])
def test_decode_of_strided_inputs(N, dtype):
    need_gpu()
    say("linattn decode strides", N, dtype)
    H, Hk = 6, 3
    q, k, v, g, _, _ = _draw([N], H, Hk, 128, 128, dtype, "mild", 53, state=False)
    S = torch.randn(N, H, 128, 128, generator=torch.Generator().manual_seed(54)).to(DEV)
    P1, P2 = S.clone(), S.clone()
    a = kda.linattn_recurrent_decode(*_gpu(q, k, v, g), P1)
    b = kda.linattn_recurrent_decode(*_fused(q, k, v, 8), g.to(DEV), P2)
    assert torch.equal(a, b) and torch.equal(P1, P2)


def test_broadcast_rows_are_refused():
    need_gpu()
    say("linattn broadcast rows")
    q, k, v, g, cu, _ = _draw([40], 2, 2, 128, 128, BF, "mild", 55, state=False)
    q, k, v, g = _gpu(q, k, v, g)
    with pytest.raises(kda.KdaError, match="stride"):
        kda.linattn_chunk_prefill(q[:1].expand(40, 2, 128), k, v, g)
    with pytest.raises(ValueError, match="dense"):
        kda.linattn_chunk_prefill(q[:, :1].expand(40, 2, 128), k, v, g)


def test_backwards_at_the_same_time():
    """On two other streams, with workspaces of their own, and twice: the same bits."""
    need_gpu()
    say("linattn backwards at once")
    draws = [_draw([2300, 0, 300], 3, 3, 128, 64, BF, "head", 56 + i) for i in range(2)]
    do = torch.randn(2600, 3, 64, generator=torch.Generator().manual_seed(58)).to(BF).to(DEV)
    dev = [_gpu(*d[:4]) for d in draws]
    kw = _cu(draws[0][4])
    alone = [kda.linattn_chunk_prefill_backward(*x, do, **kw) for x in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(2):
        got = []
        for x, s in zip(dev, streams):
            with torch.cuda.stream(s):
                got.append(kda.linattn_chunk_prefill_backward(*x, do, **kw))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_two_graphs_over_one_workspace():
    """Graphs of two sizes that were captured over the same workspace, replayed in turn: no
    replay finds anything of the other's in it."""
    need_gpu()
    say("linattn graphs over one workspace")
    draws = [_draw(lens, 2, 1, 128, 128, BF, "head", 59) for lens in ([2300], [1300, 500, 11])]
    dev = [_gpu(*d[:4]) for d in draws]
    cus = [_cu(d[4]) for d in draws]
    dos = [torch.ones(d[4][-1], 2, 128, dtype=BF, device=DEV) for d in draws]
    n = max(kda.linattn_chunk_prefill_backward_workspace_bytes(d[4][-1], len(d[4]) - 1, 2, 1)
            for d in draws)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)

    def run(i):
        o, S = kda.linattn_chunk_prefill(*dev[i], **cus[i], workspace=ws)
        return (o, S) + kda.linattn_chunk_prefill_backward(*dev[i], dos[i], **cus[i], workspace=ws)

    want = [[x.clone() for x in run(i)] for i in range(2)]
    graphs, outs = [], []
    for i in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=side):
            outs.append(run(i))
    for i in (0, 1, 1, 0, 0, 1):
        ws.fill_(255)
        graphs[i].replay()
        torch.cuda.synchronize()
        for x, y in zip(outs[i], want[i]):
            assert torch.equal(x, y)
