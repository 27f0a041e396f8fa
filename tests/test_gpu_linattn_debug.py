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
