"""GPU: the 8-bit values of RMS norm are the fp32 quotient y / scale rounded to nearest even, also
where that lies beside the middle of two codes."""
import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests.gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


def _beside_the_middles(heads, d, seed):
    """[heads, d] fp32: in every row a largest value of its own, the others within a step of the
    scale times the middle of two codes; and the rows' scales."""
    gen = torch.Generator().manual_seed(seed)
    top = torch.exp2(torch.rand(heads, 1, generator=gen) * 40 - 20)
    scale = top / 448
    codes = torch.arange(1, 0x7e, dtype=torch.uint8)  # positive, up to 416; 448 is the last one
    lo, hi = codes.view(E4).float(), (codes + 1).view(E4).float()
    mid = (lo + hi) / 2
    pick = mid[torch.randint(len(mid), (heads, d), generator=gen)]
    y = (pick.double() * scale.double()).float()
    bits = y.view(torch.int32) + torch.randint(-1, 2, (heads, d), generator=gen, dtype=torch.int32)
    y = bits.view(torch.float32) * (torch.randint(0, 2, (heads, d), generator=gen) * 2 - 1)
    y[:, ::128] = top  # the largest of every 128 columns
    return y, scale


@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("heads, d", [(512, 64), (512, 128), (128, 512), (32, 2048), (16, 8192),
                                      (8, 16384), (64, 1000)])
def test_e4m3_rounds_the_quotient(heads, d, group):
    """Rows of x alike and eps = 0: x / rms(x) is 1 up to the sum's rounding (exactly where d is a
    power of two), so y is the weight.  The quotient is fp32's, correctly rounded, on both sides:
    equal."""
    need_gpu()
    say("rmsnorm e4m3 quotient", heads, d, group)
    y, scale = _beside_the_middles(heads, d, d + group)
    x = torch.full((1, heads, d), 2.0)
    got_y, _ = kda.rmsnorm(x.to(DEV), y.to(DEV), eps=0.0)
    got_y = got_y[0].cpu()
    if d & (d - 1) == 0:
        assert torch.equal(got_y, y)
    q, scales, _ = kda.rmsnorm_e4m3(x.to(DEV), y.to(DEV), eps=0.0, scale_group=group)
    scales = scales[0].cpu()
    n = group or d
    k = -(-d // n)
    tops = torch.nn.functional.pad(got_y.abs(), (0, k * n - d)).unflatten(-1, (k, n)).amax(-1)
    assert torch.equal(scales, tops / 448)
    want = (got_y / scales.repeat_interleave(n, -1)[:, :d]).to(E4)
    off = (q[0].cpu().float() != want.float()).sum().item()
    say("values of another code", off, "of", want.numel())
    assert off == 0
