"""GPU: dweight of RMS norm over many rows keeps fp32's digits: the rows' owners' sums are added in
64 bits."""
import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests.gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("rows, heads, d", [(65536, 1, 128), (16384, 6, 64), (200000, 1, 33),
                                            (8192, 1, 1024)])
def test_sums_over_many_rows(rows, heads, d):
    """Random values, so that a column's sum grows like sqrt(rows), and so do errors of its terms:
    each term's few roundings (2 u together in the mean of squares, with its row's 1 / rms) make
    2 u of the sum, an owner's eight to sixteen rows added in fp32 1.5 u, the result's rounding
    0.3: 2.6 u.  Hundreds of owners added one after the other in fp32 would be 6 u."""
    need_gpu()
    say("rmsnorm dweight", rows, heads, d)
    gen = torch.Generator(device=DEV).manual_seed(rows + d)
    x = torch.randn(rows, heads, d, generator=gen, device=DEV)
    dy = torch.randn(rows, heads, d, generator=gen, device=DEV)
    w = 1 + 0.1 * torch.randn(heads, d, generator=gen, device=DEV)
    dw = kda.rmsnorm_backward(dy, x, w, eps=1e-5)[1].double()
    xd = x.double()
    want = (dy.double() * xd / (xd.square().mean(-1, keepdim=True) + 1e-5).sqrt()).sum(0)
    off = ((dw - want).norm() / want.norm()).item() / U
    say("%.2f u" % off)
    assert off <= 2.6
    again = kda.rmsnorm_backward(dy, x, w, eps=1e-5)[1].double()
    assert torch.equal(again, dw)
