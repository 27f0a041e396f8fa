"""GPU: the gated linear recurrence (scan, gradients, one-token step) against 64-bit
recurrences on the CPU; the bounds are derived in gatedrec_ref.py."""
import itertools

import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import gatedrec_ref as ref
from tests.gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(T, C, dtype, gate=True, gated=True, seed=0, slow=False):
    """x, r, i as columns of one projection, the gate's parameters; CPU tensors."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    proj = rnd(T, (3 if gated else 2) * C).to(dtype)
    A_log = dt_bias = None
    if gate:
        A_log = torch.rand(C, generator=gen) * 1.25 - 0.75
        dt_bias = rnd(C) * 1.2 - (11.0 if slow else 4.6)
    else:
        g = -torch.exp(-6.0 * torch.rand(C, generator=gen) - (6.0 if slow else 0.0))
        proj[:, C:2 * C] = (g * torch.rand(T, C, generator=gen)).to(dtype)
    x, r = proj[:, :C], proj[:, C:2 * C]
    return x, r, proj[:, 2 * C:] if gated else None, A_log, dt_bias, rnd


def dev(*ts):
    """To the GPU; columns of one CPU tensor stay columns of one GPU tensor."""
    out, seen = [], {}
    for t in ts:
        if t is None:
            out.append(None)
        elif t._base is not None:
            b = seen.setdefault(id(t._base), t._base.to(DEV))
            out.append(b.as_strided(t.shape, t.stride(), t.storage_offset()))
        else:
            out.append(t.to(DEV))
    return out


def cu_of(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def run_scan(lens, C, dtype, gate=True, gated=True, norm=True, state=True, seed=0, slow=False,
             h_dtype=None, host=True, name="", backward=True):
    cu = cu_of(lens)
    T, N = cu[-1], len(lens)
    x, r, i, A_log, dt_bias, rnd = make(T, C, dtype, gate, gated, seed, slow)
    S0 = rnd(N, C) if state else None
    dS = rnd(N, C) if state else None
    dh = rnd(T, C).to(dtype)
    want = (ref.backward if backward else ref.scan)(
        x, r, i, A_log, dt_bias, norm, cu, S0, *([dh, dS] if backward else []))
    X, R, I, A, B, S = dev(x, r, i, A_log, dt_bias, S0)
    cud = torch.tensor(cu, dtype=torch.int32)
    args = dict(A_log=A, dt_bias=B, normalize=norm, cu_seqlens=cud.to(DEV),
                cu_seqlens_host=cud if host else None, initial_state=S)
    h, Sf, starts = kda.gatedrec_scan(X, R, I, h_dtype=h_dtype, output_starts=backward, **args)
    say(name, "h %.2g" % ref.within("h", h, want["h"], want["eh"], h_dtype or dtype),
        "S %.2g" % ref.within("S", Sf, want["S"], want["eS"], F32))
    if not backward:
        return h, Sf
    DH, DS = dev(dh, dS)
    both = []
    for st in (starts, None):
        g = kda.gatedrec_scan_backward(X, R, I, DH, d_final_state=DS, starts=st, **args)
        both.append(g)
        for k, (key, t) in enumerate(zip(("dx", "dr", "di", "dA", "db", "dS0"), g)):
            if want[key] is None:
                assert t is None
            else:
                say(key, "%.2g" % ref.within(key, t, want[key], want["e" + key],
                                             dtype if k < 3 else F32))
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(*both))  # starts change nothing
    return h, Sf


@pytest.mark.parametrize("gate, gated, norm", list(itertools.product([True, False], repeat=3)))
@pytest.mark.parametrize("dtype, C", [(BF, 130), (F32, 70), (BF, 65)])
def test_forms(dtype, C, gate, gated, norm):
    need_gpu()
    say("gatedrec forms", dtype, C, gate, gated, norm)
    run_scan([37, 0, 1, 190, 100], C, dtype, gate, gated, norm, seed=C)


LENS = [
    [1], [2], [15], [16], [17], [63], [64], [65], [127], [128], [129], [255], [257], [1024],
    [1] * 40, [0, 0, 5, 0, 0], [128, 128], [64, 64, 64], [16] * 9, [130, 0, 0, 126, 1, 1, 500],
    [31, 33, 0, 64, 3, 125, 128, 1, 127],
]


@pytest.mark.parametrize("case", range(len(LENS)))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths(case, dtype):
    need_gpu()
    say("gatedrec lengths", LENS[case], dtype)
    run_scan(LENS[case], 6, dtype, seed=case, state=case % 2 == 0, host=case % 3 != 0)


@pytest.mark.parametrize("C", [1, 2, 3, 63, 64, 66, 127, 128, 129, 254, 256, 258, 1000, 1001])
def test_channels(C):
    need_gpu()
    say("gatedrec channels", C)
    run_scan([90, 150], C, BF, seed=C)


def test_mixed_dtypes():
    need_gpu()
    say("gatedrec mixed dtypes")
    a, _ = run_scan([200, 77], 66, BF, h_dtype=F32, seed=3)
    b, _ = run_scan([200, 77], 66, BF, seed=3)
    assert torch.equal(a.to(BF), b)
    run_scan([200, 77], 66, F32, h_dtype=BF, seed=4)
    x, r, i, A, B, rnd = make(150, 66, BF, seed=5)
    X, R, I, A, B, DH = dev(x, r, i, A, B, rnd(150, 66))
    g32 = kda.gatedrec_scan_backward(X, R, I, DH, A, B, grad_dtype=F32)
    gbf = kda.gatedrec_scan_backward(X, R, I, DH, A, B)
    assert all(torch.equal(a.to(BF), b) for a, b in zip(g32[:3], gbf[:3]))
    assert all(torch.equal(a, b) for a, b in zip(g32[3:], gbf[3:]))
    none = kda.gatedrec_scan_backward(X, R, I, None, A, B)
    assert all(not t.any() for t in none)
    assert kda.gatedrec_scan_backward(X, R, I, DH, A, B, want_d_initial_state=False)[5] is None
    assert kda.gatedrec_scan_backward(X, R, I, DH, A)[4] is None  # no dt_bias


@pytest.mark.parametrize("gate", [True, False])
def test_slow_channels_do_not_drift(gate):
    """Decays of 1e-5 to 1e-3 a token, of one value a channel: a rounding of exp(g) to fp32
    would be the same in every step and add up."""
    need_gpu()
    say("gatedrec slow channels", gate)
    T, C = 6000, 32
    x, r, i, A, B, rnd = make(T, C, F32, gate, True, seed=1, slow=True)
    r[:] = r[:1].clone()
    for norm in (False, True):
        want = ref.scan(x, r, i, A, B, norm, [0, T], None)
        X, R, I, A_, B_ = dev(x, r, i, A, B)
        h, S, _ = kda.gatedrec_scan(X, R, I, A_, B_, norm)
        say(ref.within("h", h, want["h"], want["eh"], F32))
        rel = ((h.double().cpu() - want["h"]).norm() / want["h"].norm()).item()
        say("rel %.2g" % rel)
        assert rel < 4e-6


def test_fast_and_infinite_gates():
    need_gpu()
    say("gatedrec infinite gates")
    T, C = 200, 66
    x, r, i, A, B, rnd = make(T, C, F32, seed=2)
    r[3] = float("inf")      # forgets everything
    r[50:60] = -float("inf")  # keeps everything, m = 0
    r[100] = 60.0
    i[7] = float("inf")
    i[8] = -float("inf")
    for norm in (True, False):
        f = ref.scan(x, r, i, A, B, norm, [0, T], None)
        X, R, I, A_, B_ = dev(x, r, i, A, B)
        h, S, _ = kda.gatedrec_scan(X, R, I, A_, B_, norm)
        assert torch.isfinite(h).all()
        err = (h.double().cpu() - f["h"]).abs().max() / f["h"].abs().max()
        say("err %.2g" % err)
        assert err < 1e-5
        g = kda.gatedrec_scan_backward(X, R, I, torch.ones(T, C, device=DEV), A_, B_, norm)
        assert all(torch.isfinite(t).all() for t in g if t is not None)
        if norm:
            assert torch.equal(h[49], h[59])


def test_bad_values_stay_in_their_channel_and_sequence():
    need_gpu()
    say("gatedrec bad values")
    lens = [100, 140, 30, 260, 11]
    cu = torch.tensor(cu_of(lens), dtype=torch.int32)
    T, C = int(cu[-1]), 130
    x, r, i, A, B, rnd = make(T, C, BF, seed=6)
    DH = rnd(T, C).to(BF).to(DEV)
    args = dict(normalize=True, cu_seqlens=cu.to(DEV), cu_seqlens_host=cu)
    X, R, I, A, B = dev(x, r, i, A, B)
    h, S, _ = kda.gatedrec_scan(X, R, I, A, B, **args)
    g = kda.gatedrec_scan_backward(X, R, I, DH, A, B, **args)
    X2, R2, I2 = (t.clone() for t in (X, R, I))
    X2[270, 5] = float("nan")   # sequence 3
    X2[239, 7] = float("inf")   # the last token of sequence 1
    R2[105, 9] = float("nan")   # sequence 1
    I2[529, 64] = float("nan")  # the last token of sequence 3
    bad = torch.zeros(T, C, dtype=torch.bool, device=DEV)   # what h may show
    bad[270:530, 5] = bad[239, 7] = bad[105:240, 9] = bad[529, 64] = True
    h2, S2, _ = kda.gatedrec_scan(X2, R2, I2, A, B, **args)
    assert torch.equal(h[~bad], h2[~bad]) and not torch.isfinite(h2[bad]).any()
    whole = torch.zeros(T, C, dtype=torch.bool, device=DEV)  # gradients: the sequence's channel
    whole[270:530, 5] = whole[100:240, 7] = whole[100:240, 9] = whole[270:530, 64] = True
    g2 = kda.gatedrec_scan_backward(X2, R2, I2, DH, A, B, **args)
    for a, b in zip(g[:3], g2[:3]):
        assert torch.equal(a[~whole], b[~whole])
    keep = torch.ones(C, dtype=torch.bool, device=DEV)
    keep[[5, 7, 9, 64]] = False
    assert torch.equal(g[3][keep], g2[3][keep]) and torch.equal(g[4][keep], g2[4][keep])
    for n in (0, 2, 4):
        assert torch.equal(S[n], S2[n]) and torch.equal(g[5][n], g2[5][n])


def test_log_decays_above_zero_are_zero():
    need_gpu()
    say("gatedrec positive log-decays")
    x, r, i, _, _, rnd = make(100, 10, F32, gate=False, seed=8)
    r[5:9, ::2] = 0.3
    X, R, I, DH = dev(x, r, i, rnd(100, 10))
    R0 = R.clamp(max=0)
    a = kda.gatedrec_scan(X, R, I)[0]
    assert torch.equal(a, kda.gatedrec_scan(X, R0, I)[0])
    g, g0 = kda.gatedrec_scan_backward(X, R, I, DH), kda.gatedrec_scan_backward(X, R0, I, DH)
    assert torch.equal(g[0], g0[0]) and not g[1][5:9, ::2].any() and g0[1][5:9, ::2].all()


def test_gradients_against_differences():
    """Central differences of the 64-bit loss, at the library's own gradients (fp32): the step's
    own error is h^2/6 of the third derivative, 1e-6 here; values are of order 1 to 10."""
    need_gpu()
    say("gatedrec differences")
    T, C, cu = 9, 3, [0, 4, 9]
    x, r, i, A, B, rnd = make(T, C, F32, seed=9)
    B = B + 4.0  # decays away from 0
    S0, dh, dS = rnd(2, C), rnd(T, C), rnd(2, C)
    X, R, I, A_, B_, S, DH, DS = dev(x, r, i, A, B, S0, dh, dS)
    cut = torch.tensor(cu, dtype=torch.int32)
    got = kda.gatedrec_scan_backward(X, R, I, DH, A_, B_, True, cut.to(DEV), S, DS)
    leaves = [t.double().clone() for t in (x, r, i, A, B, S0)]

    def loss():
        f = ref.scan(leaves[0], leaves[1], leaves[2], leaves[3], leaves[4], True, cu, leaves[5])
        return (f["h"] * dh).sum() + (f["S"] * dS).sum()

    for k, t in enumerate(leaves):
        flat = t.view(-1)
        for j in range(flat.numel()):
            old = flat[j].item()
            flat[j] = old + 1e-4
            up = loss()
            flat[j] = old - 1e-4
            down = loss()
            flat[j] = old
            num = ((up - down) / 2e-4).item()
            assert abs(got[k].view(-1)[j].item() - num) <= 2e-5 * max(1.0, abs(num)), (k, j)


@pytest.mark.parametrize("C", [6, 65])
def test_long_sequence_many_tiles(C):
    """Several times more tiles than a look back reaches, all waiting at once; the same call
    gives the same bits."""
    need_gpu()
    say("gatedrec long", C)
    T = 33000
    run_scan([T], C, BF, seed=10, slow=True, backward=True)
    x, r, i, A, B, rnd = make(T, C, BF, seed=10, slow=True)
    X, R, I, A, B, DH = dev(x, r, i, A, B, rnd(T, C))
    a = kda.gatedrec_scan(X, R, I, A, B, True, output_starts=True)
    g = kda.gatedrec_scan_backward(X, R, I, DH, A, B, True)
    for _ in range(4):
        assert all(torch.equal(p, q) for p, q in zip(
            a, kda.gatedrec_scan(X, R, I, A, B, True, output_starts=True)))
        assert all(torch.equal(p, q) for p, q in zip(
            g, kda.gatedrec_scan_backward(X, R, I, DH, A, B, True)))


def test_wide():
    """The layer's width over many tiles and channel blocks at once, against the reference on a
    few channels; the same call gives the same bits."""
    need_gpu()
    say("gatedrec wide")
    T, C = 3000, 12288
    gen = torch.Generator(device=DEV).manual_seed(11)
    proj = torch.randn(T, 3 * C, generator=gen, device=DEV).to(BF)
    X, R, I = proj[:, :C], proj[:, C:2 * C], proj[:, 2 * C:]
    A = torch.rand(C, generator=gen, device=DEV) - 0.5
    B = torch.randn(C, generator=gen, device=DEV) - 4.0
    cu = torch.tensor([0, 1000, 1001, 3000], dtype=torch.int32)
    args = dict(normalize=True, cu_seqlens=cu.to(DEV), cu_seqlens_host=cu)
    DH = torch.randn(T, C, generator=gen, device=DEV).to(BF)
    a = kda.gatedrec_scan(X, R, I, A, B, output_starts=True, **args)
    g = kda.gatedrec_scan_backward(X, R, I, DH, A, B, starts=a[2], **args)
    cols = [0, 1, 63, 64, 127, 128, 5000, 12287]
    take = lambda t: t[..., cols].cpu()  # noqa: E731
    want = ref.backward(take(X), take(R), take(I), take(A), take(B), True, cu.tolist(), None,
                        take(DH), None)
    ref.within("h", take(a[0]), want["h"], want["eh"], BF)
    ref.within("S", take(a[1]), want["S"], want["eS"], F32)
    for k, (key, t) in enumerate(zip(("dx", "dr", "di", "dA", "db", "dS0"), g)):
        say(key, "%.2g" % ref.within(key, take(t), want[key], want["e" + key], BF if k < 3 else F32))
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(
            a, kda.gatedrec_scan(X, R, I, A, B, output_starts=True, **args)))
        assert all(torch.equal(p, q) for p, q in zip(
            g, kda.gatedrec_scan_backward(X, R, I, DH, A, B, **args)))


# ------------------------------------------------------------------- decode
@pytest.mark.parametrize("sdt", [F32, BF])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N, C", [(1, 1), (1, 130), (3, 65), (5, 256), (40, 1000)])
def test_decode(N, C, dtype, sdt):
    """Steps over a pool with padding entries; untouched slots stay."""
    need_gpu()
    say("gatedrec decode", N, C, dtype, sdt)
    for gate, gated, norm in itertools.product([True, False], repeat=3):
        x, r, i, A, B, rnd = make(N, C, dtype, gate, gated, seed=N * C)
        slots = N + 2
        pool = rnd(slots, C).to(sdt)
        idx = torch.randperm(slots, generator=torch.Generator().manual_seed(N))[:N].to(torch.int32)
        idx[N // 2::3] = -1
        if N > 3:
            idx[1] = slots
        live = [(n, int(s)) for n, s in enumerate(idx) if 0 <= s < slots]
        X, R, I, A_, B_, P = dev(x, r, i, A, B, pool)
        h = kda.gatedrec_decode(X, R, I, P, A_, B_, norm, state_indices=idx.to(DEV))
        f = ref.gate(x, r, i, A, B, norm)
        want, bound = torch.zeros(N, C, dtype=ref.F64), torch.zeros(N, C, dtype=ref.F64)
        new, eb = pool.double(), torch.zeros(slots, C, dtype=ref.F64)
        along = ref._along(f)
        for n, s in live:
            st = pool[s].double()
            want[n] = f["a"][n] * st + f["b"][n]
            bound[n] = (8 * ref.U * (f["a"][n] * st).abs() + along[n] * st.abs()
                        + (f["eb"][n] + 4 * ref.U) * f["b"][n].abs())
            new[s], eb[s] = want[n], bound[n]
        ref.within("h", h, want, bound, dtype)
        ref.within("pool", P, new, eb, sdt)
        dead = [s for s in range(slots) if s not in [q for _, q in live]]
        assert torch.equal(P[dead].cpu(), pool[dead])


def test_decode_continues_a_scan():
    """A prompt through the scan into a pool, then steps, against one long scan: the same to
    rounding."""
    need_gpu()
    say("gatedrec decode after scan")
    lens, C, extra = [70, 200, 1], 130, 20
    N = len(lens)
    tot = [n + extra for n in lens]
    x, r, i, A, B, rnd = make(sum(tot), C, F32, seed=12, slow=True)
    want = ref.scan(x, r, i, A, B, True, cu_of(tot), None)
    X, R, I, A, B = dev(x, r, i, A, B)
    first = cu_of(tot)
    rows = torch.cat([torch.arange(first[n], first[n] + lens[n]) for n in range(N)]).to(DEV)
    pool = torch.full((5, C), 7.0, device=DEV)
    idx = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    cu = torch.tensor(cu_of(lens), dtype=torch.int32, device=DEV)
    kda.gatedrec_scan(X[rows], R[rows], I[rows], A, B, True, cu, final_state=pool, state_indices=idx)
    for t in range(extra):
        at = torch.tensor([first[n] + lens[n] + t for n in range(N)], device=DEV)
        h = kda.gatedrec_decode(X[at], R[at], I[at], pool, A, B, True, state_indices=idx)
        # a step rounds like a fold of its own
        ref.within("h", h, want["h"][at.cpu()],
                   want["eh"][at.cpu()] + 4 * extra * ref.U * want["H"][at.cpu()], F32)
    assert (pool[[1, 3]] == 7.0).all()
