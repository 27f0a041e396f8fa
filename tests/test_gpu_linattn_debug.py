"""GPU: KDA_DEBUG=1 on the linear attention calls beyond the cases of the other files."""
import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests.gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def test_every_state_of_a_large_pool_is_scanned(monkeypatch):
    """More states than the scan has workgroups."""
    need_gpu()
    say("linattn KDA_DEBUG large pool")
    monkeypatch.setenv("KDA_DEBUG", "1")
    N = 70001
    q = torch.full((N, 1, 64), 0.125, dtype=BF, device=DEV)
    g = torch.full((1,), -0.5, device=DEV)
    pool = torch.ones(N, 1, 64, 64, dtype=BF, device=DEV)
    kda.linattn_recurrent_decode(q, q, q, g, pool)
    pool[N - 1, 0, 63, 63] = float("nan")
    pool[3, 0, 0, 0] = float("inf")
    with pytest.raises(kda.KdaError, match=r"state not finite \(2 of"):
        kda.linattn_recurrent_decode(q, q, q, g, pool)


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_no_sequence_are_not_scanned(decay, dtype, monkeypatch):
    """Rows behind the last sequence may hold anything; the last row of a sequence not."""
    need_gpu()
    say("linattn KDA_DEBUG rows behind", decay, dtype)
    monkeypatch.setenv("KDA_DEBUG", "1")
    T, end, H, Hk = 90, 71, 4, 2
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    q, k, v, do = r(T, Hk, 128), r(T, Hk, 128), r(T, H, 64), r(T, H, 64)
    g = -torch.rand(*((T, H) if decay == "token" else (H,)), generator=gen).to(DEV)
    for t in (q, k, v, do) + ((g,) if decay == "token" else ()):
        t[end:] = float("nan")
    cu = torch.tensor([0, 40, end], dtype=torch.int32, device=DEV)
    out = torch.full((T, H, 64), float("inf"), dtype=dtype, device=DEV)
    kda.linattn_chunk_prefill(q, k, v, g, cu_seqlens=cu, out=out)
    assert torch.isinf(out[end:]).all() and torch.isfinite(out[:end]).all()
    kda.linattn_chunk_prefill_backward(q, k, v, g, do, cu_seqlens=cu)
    for name, t in (("q", q), ("k", k), ("v", v), ("d_o", do)) + (
            (("g", g),) if decay == "token" else ()):
        keep = t[end - 1].clone()
        t.view(T, -1)[end - 1, -1] = float("nan")
        with pytest.raises(kda.KdaError, match=r"%s not .* \(1 of" % name):
            kda.linattn_chunk_prefill_backward(q, k, v, g, do, cu_seqlens=cu)
        t[end - 1] = keep
    kda.linattn_chunk_prefill_backward(q, k, v, g, do, cu_seqlens=cu)


def test_skipped_sequences_of_a_decode_are_not_scanned(monkeypatch):
    need_gpu()
    say("linattn KDA_DEBUG skipped sequences")
    monkeypatch.setenv("KDA_DEBUG", "1")
    N, H = 5, 3
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(N, H, 128, generator=gen).to(BF).to(DEV) for _ in range(3))
    g = -torch.rand(N, H, generator=gen).to(DEV)
    pool = torch.randn(4, H, 128, 128, generator=gen).to(DEV)
    idx = torch.tensor([2, -1, 0, 4, 1], dtype=torch.int32, device=DEV)
    for t in (q, k, v, g):
        t[1] = t[3] = float("nan")
    o = kda.linattn_recurrent_decode(q, k, v, g, pool, state_indices=idx)
    assert not o[1].any() and not o[3].any() and torch.isfinite(o).all()
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        keep = t[4].clone()
        t[4, 1] = float("nan")
        with pytest.raises(kda.KdaError, match="%s not" % name):
            kda.linattn_recurrent_decode(q, k, v, g, pool, state_indices=idx)
        t[4] = keep
