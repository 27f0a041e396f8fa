"""GPU: stretches of the gated linear recurrence whose decay is exactly 1 keep the state (and, in
the gradients, what comes back): log-decays of 0, of either sign, and above, and logits so low that
softplus is 0; over a token, a wave's tokens, whole tiles and whole sequences."""
import itertools

import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import gatedrec_ref as ref
from tests.gpu_util import DEV, need_gpu, say
from tests.test_gpu_gatedrec import cu_of, dev, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dx", "dr", "di", "dA", "db", "dS0")

# tokens of decay 1: eight and sixteen at multiples of them, other places, whole tiles of 32 to 128
SPANS = [(0, 16), (24, 32), (48, 64), (67, 71), (128, 256), (300, 420), (448, 640)]


@pytest.mark.parametrize("gated, norm", list(itertools.product([True, False], repeat=2)))
@pytest.mark.parametrize("dtype, C", [(BF, 66), (BF, 65), (F32, 33)])
@pytest.mark.parametrize("lens", [[700], [16, 0, 112, 128, 300, 144], [30] * 23 + [10]])
def test_log_decays_of_zero(lens, dtype, C, gated, norm):
    need_gpu()
    say("gatedrec kept, log-decays", lens, dtype, C, gated, norm)
    cu, N = cu_of(lens), len(lens)
    T = cu[-1]
    x, r, i, _, _, rnd = make(T, C, dtype, gate=False, gated=gated, seed=C)
    for lo, hi in SPANS:
        r[lo:hi, 0::4], r[lo:hi, 1::4], r[lo:hi, 2::4] = 0.0, -0.0, 0.25
    S0, dS, dh = rnd(N, C), rnd(N, C), rnd(T, C).to(dtype)
    want = ref.backward(x, r, i, None, None, norm, cu, S0, dh, dS)
    X, R, I, S, DS, DH = dev(x, r, i, S0, dS, dh)
    args = dict(normalize=norm, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                initial_state=S)
    h, Sf, starts = kda.gatedrec_scan(X, R, I, output_starts=True, **args)
    say("h %.2g" % ref.within("h", h, want["h"], want["eh"], dtype),
        "S %.2g" % ref.within("S", Sf, want["S"], want["eS"], F32))
    for st in (starts, None):
        g = kda.gatedrec_scan_backward(X, R, I, DH, d_final_state=DS, starts=st, **args)
        for k, (key, t) in enumerate(zip(NAMES, g)):
            if want[key] is not None:
                say(key, "%.2g" % ref.within(key, t, want[key], want["e" + key],
                                             dtype if k < 3 else F32))


@pytest.mark.parametrize("low", [-float("inf"), -200.0])
@pytest.mark.parametrize("dtype, C", [(BF, 66), (F32, 33)])
def test_logits_that_keep_everything(dtype, C, low):
    """-inf is the limit of -200, whose softplus (1e-87) fp32 does not have either."""
    need_gpu()
    say("gatedrec kept, logits", dtype, C, low)
    lens = [600, 128, 40]
    cu, N = cu_of(lens), len(lens)
    T = cu[-1]
    x, r, i, A, B, rnd = make(T, C, dtype, seed=C + 1)
    for lo, hi in SPANS:
        r[lo:hi, ::2] = -200.0
    S0, dS, dh = rnd(N, C), rnd(N, C), rnd(T, C).to(dtype)
    for norm in (True, False):
        want = ref.backward(x, r, i, A, B, norm, cu, S0, dh, dS)
        X, R, I, A_, B_, S, DS, DH = dev(x, r, i, A, B, S0, dS, dh)
        R[R == -200.0] = low
        args = dict(normalize=norm, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                    initial_state=S)
        h, Sf, starts = kda.gatedrec_scan(X, R, I, A_, B_, output_starts=True, **args)
        say("h %.2g" % ref.within("h", h, want["h"], want["eh"], dtype),
            "S %.2g" % ref.within("S", Sf, want["S"], want["eS"], F32))
        g = kda.gatedrec_scan_backward(X, R, I, DH, A_, B_, d_final_state=DS, starts=starts, **args)
        for k, (key, t) in enumerate(zip(NAMES, g)):
            say(key, "%.2g" % ref.within(key, t, want[key], want["e" + key],
                                         dtype if k < 3 else F32))


@pytest.mark.parametrize("sdt", [F32, BF])
@pytest.mark.parametrize("dtype, C", [(BF, 66), (BF, 33), (F32, 130)])
def test_a_step_keeps_the_state(dtype, C, sdt):
    """A step of decay 1 adds to the slot: with sums of small whole numbers, exactly."""
    need_gpu()
    say("gatedrec kept, step", dtype, C, sdt)
    N = 5
    gen = torch.Generator().manual_seed(C)
    whole = lambda: torch.randint(-50, 51, (N, C), generator=gen).float()  # noqa: E731
    x, S = whole(), whole()
    for gate, value in ((False, 0.0), (False, -0.0), (False, 0.5), (True, -200.0),
                        (True, -float("inf"))):
        r = torch.full((N, C), value)
        A = torch.zeros(C, device=DEV) if gate else None
        for norm in (False, True):
            P = S.to(sdt).to(DEV)
            h = kda.gatedrec_decode(x.to(dtype).to(DEV), r.to(dtype).to(DEV), None, P, A, None, norm)
            want = S if norm else S + x  # m is 0
            assert torch.equal(h.float().cpu(), want), (gate, value, norm)
            assert torch.equal(P.float().cpu(), want), (gate, value, norm)


def test_a_long_sequence_that_keeps_everything():
    """More tiles than a look back reaches, all of decay 1: h is the sum of x, in whole numbers, and
    R the sum of dh."""
    need_gpu()
    say("gatedrec kept, many tiles")
    T, C = 20000, 66
    gen = torch.Generator().manual_seed(5)
    x = torch.randint(-2, 3, (T, C), generator=gen).float()
    dh = torch.randint(-2, 3, (T, C), generator=gen).float()
    for dtype in (F32, BF):
        X, DH = x.to(dtype).to(DEV), dh.to(dtype).to(DEV)
        R = torch.zeros_like(X)
        h, S, starts = kda.gatedrec_scan(X, R, h_dtype=F32, output_starts=True)
        assert torch.equal(h.cpu(), x.cumsum(0)) and torch.equal(S[0].cpu(), x.sum(0))
        for st in (starts, None):
            g = kda.gatedrec_scan_backward(X, R, None, DH, starts=st, grad_dtype=F32)
            assert torch.equal(g[0].cpu(), dh.flip(0).cumsum(0).flip(0))
            assert torch.equal(g[5][0].cpu(), dh.sum(0))
