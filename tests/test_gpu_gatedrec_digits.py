"""GPU: the digits of the recurrence's gate in fp32.  h of one-token sequences with x = 1 and no
entry state is m = sqrt(1 - exp(2 g)) itself.  u = 2^-24."""
import math

import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests.gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _m(how, r, A_log):
    """m of every value of r [N, C], by the scan or by a step."""
    x = torch.ones_like(r)
    A = None if A_log is None else torch.full((r.shape[1],), A_log, device=DEV)
    if how == "scan":
        return kda.gatedrec_scan(x, r, None, A, None, True, num_seqs=r.shape[0])[0]
    return kda.gatedrec_decode(x, r, None, torch.zeros_like(r), A, None, True)


@pytest.mark.parametrize("how", ["scan", "step"])
def test_softplus(how):
    """m is about sqrt(2 exp(A_log) softplus(r)), so half of the softplus' error shows.  Averaged
    over 4,096 values of r roundings leave 0.02 u; what depends on r slowly is left: of log(1 + e),
    which is to be within 1 u before its roundings, 0.5 u, and of the constant log2(e) (0.2 u of
    |r| up to 1.4) 0.1 u, beside a common factor from exp(A_log), which the mean takes away.  0.8 u
    leaves 0.2 for the hardware's exp2; a polynomial that is off by 3.7 u shows 1.8."""
    need_gpu()
    say("gatedrec softplus", how)
    A_log = -8.0
    r = torch.linspace(-1, 1, 64 * 4096 + 1, dtype=torch.float64)[:-1].float().view(4096, 64)
    m = _m(how, r.to(DEV), A_log).double().cpu().view(-1)
    z = r.double().view(-1)
    g = -math.exp(A_log) * torch.logaddexp(z, torch.zeros_like(z))
    off = ((m / torch.sqrt(-torch.expm1(2 * g)) - 1) / U).view(64, 4096).mean(1)
    off = (off - off.mean()).abs().max().item()
    say("%.2f u" % off)
    assert off <= 0.8


@pytest.mark.parametrize("how", ["scan", "step"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_root(how, dtype):
    """1 - exp(2 g) for 2 g from -0.35 to -0.17, by a polynomial: its last two roundings leave 0.4 u
    of m, the root 0.5 and g's product with log2(e) 0.3, in the mean of squares 0.7 u (as is an
    error of 1 u of the hardware's root, 0.6, with them: 0.9).  As 1 - a a it would be a's 0.3 to
    0.6 u times 3: 1.3 to 2.5."""
    need_gpu()
    say("gatedrec root", how, dtype)
    gen = torch.Generator().manual_seed(1)
    r = (-0.0867 - 0.0863 * torch.rand(2048, 64, generator=gen)).to(dtype)
    X = r.to(DEV)
    if how == "scan":
        m = kda.gatedrec_scan(torch.ones_like(X), X, normalize=True, num_seqs=2048,
                              h_dtype=torch.float32)[0]
    else:
        m = kda.gatedrec_decode(torch.ones_like(X), X, None, torch.zeros_like(X, dtype=torch.float32),
                                normalize=True, h_dtype=torch.float32)
    want = torch.sqrt(-torch.expm1(2 * r.double()))
    off = ((m.double().cpu() / want - 1) / U).square().mean().sqrt().item()
    say("%.2f u" % off)
    assert off <= 1.0
