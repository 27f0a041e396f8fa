"""GPU: the slope of m = sqrt(1 - exp(2 g)) in the recurrence's gradients, s x / m, where the
input gate's s = sigmoid(i) is so small that m s is not a normal fp32 number, and where m is 0."""
import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import gatedrec_ref as ref
from tests.gpu_util import DEV, need_gpu, say
from tests.test_gpu_gatedrec import dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dx", "dr", "di")


def _closed_gates(T, C, dtype, seed, lowest):
    """x, dh, i from -40 down to `lowest` and log-decays from -1e-2 to -1e-30 and 0."""
    gen = torch.Generator().manual_seed(seed)
    u = lambda: torch.rand(T, C, generator=gen)  # noqa: E731
    x = torch.randn(T, C, generator=gen).to(dtype)
    dh = torch.randn(T, C, generator=gen).to(dtype)
    i = (-40 - u() * (-40 - lowest)).to(dtype)
    r = (-torch.pow(10.0, -2 - 28 * u())).to(dtype)
    r[::7] = 0.0
    return x, r, i, dh


@pytest.mark.parametrize("T", [7, 200])
@pytest.mark.parametrize("dtype, C", [(BF, 66), (BF, 65), (F32, 33)])
def test_slope_of_closed_input_gates(dtype, C, T):
    """From an entry state of 0 the slope is all that dr has.  Down to -80 (1.8e-35) s is a normal
    number while m s need not be."""
    need_gpu()
    say("gatedrec slope", dtype, C, T)
    x, r, i, dh = _closed_gates(T, C, dtype, C + T, -80.0)
    want = ref.backward(x, r, i, None, None, True, [0, T], None, dh, None)
    X, R, I, DH = dev(x, r, i, dh)
    g = kda.gatedrec_scan_backward(X, R, I, DH, normalize=True, grad_dtype=F32)
    for key, t in zip(NAMES, g):
        say(key, "%.2g" % ref.within(key, t, want[key], want["e" + key], F32))
    assert (g[1] != 0).float().mean() > 0.5


@pytest.mark.parametrize("dtype, C", [(BF, 66), (F32, 33)])
def test_gradients_of_closed_input_gates(dtype, C):
    """Down to i = -100, where s (4e-44) is no fp32 number either, beside states of order 1."""
    need_gpu()
    say("gatedrec closed gates", dtype, C)
    T = 150
    x, r, i, dh = _closed_gates(T, C, dtype, C, -100.0)
    dh[::3] = 0.0
    S0 = torch.randn(1, C, generator=torch.Generator().manual_seed(C))
    want = ref.backward(x, r, i, None, None, True, [0, T], S0, dh, None)
    X, R, I, DH, S = dev(x, r, i, dh, S0)
    g = kda.gatedrec_scan_backward(X, R, I, DH, normalize=True, initial_state=S, grad_dtype=F32)
    for key, t in zip(NAMES + ("dA", "db", "dS0"), g):
        if t is not None:
            say(key, "%.2g" % ref.within(key, t, want[key], want["e" + key], F32))


@pytest.mark.parametrize("value", [-0.001, -1e-5, -0.01, 0.0])
def test_infinite_slopes_that_were(value):
    """m s of 1e-39: its reciprocal is not a number that fp32 has, the slope is 1e-36 x; and no
    gradient comes back at all where dh is 0."""
    need_gpu()
    say("gatedrec slope at", value)
    i = torch.arange(-100.0, -80.0, 0.25)[None].repeat(9, 1).to(DEV)
    x = torch.ones_like(i)
    r = torch.full_like(i, value)
    for dh in (torch.ones_like(i), torch.zeros_like(i)):
        dx, dr, di, _, _, dS = kda.gatedrec_scan_backward(x, r, i, dh, normalize=True)
        # |dr| is at most 9 tokens' R times (h + s x / m): s below 2e-35, 1 / m below 230
        assert dr.abs().max() <= 1e-30 and torch.isfinite(di).all() and torch.isfinite(dx).all()


@pytest.mark.parametrize("low", [-float("inf"), -200.0])
@pytest.mark.parametrize("dtype, C", [(BF, 66), (F32, 33)])
def test_large_values_where_the_gate_keeps_everything(dtype, C, low):
    """m = 0: the slope's part is 0 whatever x is.  Without it dr is exp(g) h R times the softplus'
    own slope, which is 0 there."""
    need_gpu()
    say("gatedrec large values", dtype, C, low)
    T = 40
    gen = torch.Generator().manual_seed(C)
    x = (torch.randn(T, C, generator=gen) * 1e25).to(dtype).to(DEV)
    i = torch.randn(T, C, generator=gen).to(dtype).to(DEV)
    r = torch.full((T, C), low).to(dtype).to(DEV)
    A = torch.zeros(C, device=DEV)
    for gate in (i, None):
        g = kda.gatedrec_scan_backward(x, r, gate, torch.ones_like(x), A, A, normalize=True)
        assert all(torch.isfinite(t).all() for t in g if t is not None)
        assert not g[1].any() and not g[3].any() and not g[4].any() and not g[0].any()
