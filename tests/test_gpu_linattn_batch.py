"""GPU: what a sequence gets does not depend on what it is packed with, and short
sequences of a large batch have the digits of a short call."""
import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import linattn_ref as ref
from tests.gpu_util import DEV, need_gpu, say
from tests.test_gpu_linattn import _cu, _draw, _gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _run(q, k, v, g, cu, S0, do, dS):
    """(o, dq, dk, dv, dg), (states, dS0)"""
    dev = _gpu(q, k, v, g, do, S0, dS)
    o, S = kda.linattn_chunk_prefill(*dev[:4], **_cu(cu), initial_state=dev[5], scale=0.7)
    b = kda.linattn_chunk_prefill_backward(*dev[:5], **_cu(cu), initial_state=dev[5],
                                           d_final_state=dev[6], scale=0.7)
    return (o,) + b[:4], (S, b[4])


# the second batch has one head, so that its long sequence is cut into segments
@pytest.mark.parametrize("lens, H, Hk", [([40, 300, 1, 64, 65, 0, 9], 4, 2), ([4200, 40, 64, 1], 1, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_sequence_alone_and_packed(lens, H, Hk, dtype):
    """Bit for bit: o and the gradients of every token of the sequences that run in one
    piece, and where the batch is not cut their states too."""
    need_gpu()
    say("linattn alone and packed", lens, H, Hk, dtype)
    q, k, v, g, cu, S0 = _draw(lens, H, Hk, 128, 128, dtype, "mild", 40)
    gen = torch.Generator().manual_seed(41)
    do = torch.randn(cu[-1], H, 128, generator=gen).to(dtype)
    dS = torch.randn(len(lens), H, 128, 128, generator=gen)
    whole = kda.linattn_chunk_prefill_workspace_bytes(cu[-1], len(lens), H) == 0
    assert whole == (H > 1)
    rows, states = _run(q, k, v, g, cu, S0, do, dS)
    for n in range(len(lens)):
        if lens[n] > 300:
            continue
        a, b = cu[n], cu[n + 1]
        one = _run(q[a:b], k[a:b], v[a:b], g[a:b], [0, b - a], S0[n:n + 1], do[a:b], dS[n:n + 1])
        for name, x, y in zip(("o", "dq", "dk", "dv", "dg"), rows, one[0]):
            assert torch.equal(x[a:b], y), (name, n, lens[n])
        if whole:
            for name, x, y in zip(("state", "dS0"), states, one[1]):
                assert torch.equal(x[n:n + 1], y), (name, n, lens[n])


@pytest.mark.parametrize("lens", [[1] * 100, [64, 64, 3, 20, 64]])
def test_short_sequences_of_a_large_call(lens):
    """Sequences of at most 64 tokens make bf16 o and dv of two-value factors: besides
    their rounding they are off by 2^-15 and not by 2^-8 of their terms."""
    need_gpu()
    say("linattn short sequences", len(lens), max(lens))
    H, Hk = 3, 3
    q, k, v, g, cu, S0 = _draw(lens, H, Hk, 128, 64, BF, "mild", 42)
    do = torch.randn(cu[-1], H, 64, generator=torch.Generator().manual_seed(43)).to(BF)
    (o, _, _, dv, _), _ = _run(q, k, v, g, cu, S0, do, None)
    rel = ref.rel_of(q, v, cu, 2)
    want, _ = ref.forward(q, k, v, g, cu, S0, 0.7)
    size, _ = ref.forward(q.abs(), k.abs(), v.abs(), g, cu, S0.abs(), 0.7)
    say(ref.check("o", o, want, size, rel, BF))
    want = ref.backward(q, k, v, g, cu, do, S0, None, 0.7)[2]
    size = ref.backward(q.abs(), k.abs(), v.abs(), g, cu, do.abs(), S0.abs(), None, 0.7)[2]
    say(ref.check("dv", dv, want, size, rel, BF))


@pytest.mark.parametrize("lens", [[96, 90, 101, 100], [300, 40, 7, 0]])
def test_the_order_of_the_gradients_work_does_not_show(lens):
    """Batches of 576 workgroups, of like and of different lengths: the order they start in
    depends on the lengths where the host knows them, the gradients do not."""
    need_gpu()
    say("linattn order of work", lens)
    H = 24
    q, k, v, g, cu, S0 = _draw(lens, H, H, 128, 128, BF, "mild", 44)
    do = torch.randn(cu[-1], H, 128, generator=torch.Generator().manual_seed(45)).to(BF)
    dev = _gpu(q, k, v, g, do, S0)
    got = [kda.linattn_chunk_prefill_backward(*dev[:5], **kw, initial_state=dev[5])
           for kw in (_cu(cu), dict(cu_seqlens=_cu(cu)["cu_seqlens"]))]
    for x, y in zip(*got):
        assert torch.equal(x, y)
    heads = slice(0, 2)
    part = [t[:, heads] for t in (q, k, v, g, do, S0)]
    ref.check_backward([t[:, heads] for t in got[0]], *part[:4], cu, part[4], part[5])
