"""GPU: linear attention with one decay per head (chunked prefill, its
gradients, one-token decode) against the 64-bit recurrence, elementwise within
the bounds of tests/linattn_ref.py."""
import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import linattn_ref as ref
from tests.gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _draw(lens, H, Hk, dk, dv, dtype, decay, seed, state=True):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, N = cu[-1], len(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)  # noqa: E731
    q, k, v = unit(rnd(T, Hk, dk)).to(dtype), unit(rnd(T, Hk, dk)).to(dtype), rnd(T, H, dv).to(dtype)
    u = torch.rand(T, H, generator=gen)
    g = {"mild": -0.02 - 0.1 * u, "strong": -3.0 - 4.0 * u, "none": torch.zeros(T, H),
         # a weak decay everywhere but for tokens that wipe the state
         "resets": torch.where(u < 0.05, torch.full_like(u, -1e4), -0.05 * u),
         "gone": torch.full((T, H), float("-inf")),
         "head": -0.001 - 0.4 * torch.rand(H, generator=gen)}[decay]
    S0 = rnd(N, H, dk, dv) * 0.5 if state else None
    return q, k, v, g.float(), cu, S0


def _gpu(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def _cu(cu):
    h = torch.tensor(cu, dtype=torch.int32)
    return dict(cu_seqlens=h.to(DEV), cu_seqlens_host=h)


SHAPES = [  # lens, H, Hk, dk, dv
    ([1], 1, 1, 128, 128),
    ([64], 2, 2, 128, 128),
    ([65], 3, 1, 128, 128),
    ([63, 0, 1, 130, 17], 4, 2, 128, 128),
    ([100, 29], 2, 2, 64, 128),
    ([33, 64, 96], 3, 3, 128, 64),
    ([2, 200], 2, 1, 64, 64),
    ([0, 0], 2, 2, 128, 128),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_prefill(shape, dtype):
    need_gpu()
    lens, H, Hk, dk, dv = SHAPES[shape]
    say("linattn prefill", SHAPES[shape], dtype)
    q, k, v, g, cu, S0 = _draw(lens, H, Hk, dk, dv, dtype, "mild", 100 + shape)
    o, S = kda.linattn_chunk_prefill(*_gpu(q, k, v, g), **_cu(cu), initial_state=S0.to(DEV),
                                     scale=0.3, o_dtype=F32)
    say(ref.check_forward(o, S, q, k, v, g, cu, S0, 0.3))


@pytest.mark.parametrize("decay", ["strong", "none", "resets", "gone", "head"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_decays(decay, dtype):
    need_gpu()
    say("linattn prefill decays", decay, dtype)
    q, k, v, g, cu, S0 = _draw([150, 70], 3, 3, 128, 128, dtype, decay, 200)
    o, S = kda.linattn_chunk_prefill(*_gpu(q, k, v, g), **_cu(cu), initial_state=S0.to(DEV))
    assert o.dtype == dtype
    say(ref.check_forward(o, S, q, k, v, g, cu, S0))


def test_prefill_without_host_lengths_and_rows_behind_the_last():
    """No host copy: nothing is waited for; rows past cu[N] stay as they were, and what
    they hold (NaN) does not reach the sequences."""
    need_gpu()
    say("linattn prefill padded batch")
    q, k, v, g, cu, S0 = _draw([90, 37, 20], 2, 2, 128, 128, BF, "mild", 3)
    cut = cu[2]
    for t in (q, k, v, g):
        t[cut:] = float("nan")
    out = torch.full((cu[-1], 2, 128), 7.0, dtype=BF, device=DEV)
    o, S = kda.linattn_chunk_prefill(*_gpu(q, k, v, g), initial_state=S0[:2].to(DEV), out=out,
                                     cu_seqlens=torch.tensor(cu[:3], dtype=torch.int32, device=DEV))
    assert torch.all(o[cut:] == 7.0)
    ref.check_forward(o, S, q[:cut], k[:cut], v[:cut], g[:cut], cu[:3], S0[:2], o_rows=cut)


def test_prefill_equal_lengths():
    need_gpu()
    say("linattn prefill equal lengths")
    q, k, v, g, cu, S0 = _draw([70, 70, 70], 2, 1, 128, 128, BF, "head", 4, state=False)
    o, S = kda.linattn_chunk_prefill(*_gpu(q, k, v, g), num_seqs=3)
    ref.check_forward(o, S, q, k, v, g, cu)


def test_prefill_strided_inputs_are_the_dense_ones():
    """q, k, v as slices of one projection: bit for bit the dense call."""
    need_gpu()
    say("linattn prefill strides")
    q, k, v, g, cu, S0 = _draw([77, 100], 4, 2, 128, 128, BF, "mild", 5)
    T = cu[-1]
    whole = torch.full((T, 2 + 2 + 4 + 1, 128), float("nan"), dtype=BF)
    whole[:, 0:2], whole[:, 2:4], whole[:, 4:8] = q, k, v
    w = whole.to(DEV)
    a = kda.linattn_chunk_prefill(*_gpu(q, k, v, g), **_cu(cu))
    b = kda.linattn_chunk_prefill(w[:, 0:2], w[:, 2:4], w[:, 4:8], g.to(DEV), **_cu(cu))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ref.check_forward(b[0], b[1], q, k, v, g, cu)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_cut_into_segments(dtype):
    """Few heads and long sequences run in segments; a call without a workspace walks
    them whole; both hold the bounds."""
    need_gpu()
    say("linattn prefill segments", dtype)
    lens, H = [1700, 0, 40, 1111], 1
    q, k, v, g, cu, S0 = _draw(lens, H, H, 128, 128, dtype, "mild", 6)
    nbytes = kda.linattn_chunk_prefill_workspace_bytes(cu[-1], len(lens), H)
    assert nbytes == 0
    q, k, v, g, cu, S0 = _draw([2300, 40], H, H, 128, 128, dtype, "mild", 6)
    nbytes = kda.linattn_chunk_prefill_workspace_bytes(cu[-1], 2, H)
    assert nbytes > 0
    for ws in (torch.empty(nbytes, dtype=torch.uint8, device=DEV),
               torch.empty(256, dtype=torch.uint8, device=DEV)):
        o, S = kda.linattn_chunk_prefill(*_gpu(q, k, v, g), **_cu(cu), initial_state=S0.to(DEV),
                                         workspace=ws)
        say(ref.check_forward(o, S, q, k, v, g, cu, S0))
    # without the host's lengths the grid covers every possible segment
    o2, S2 = kda.linattn_chunk_prefill(*_gpu(q, k, v, g), cu_seqlens=_cu(cu)["cu_seqlens"],
                                       initial_state=S0.to(DEV))
    ref.check_forward(o2, S2, q, k, v, g, cu, S0)


@pytest.mark.parametrize("sdt", [F32, BF])
def test_pool_prefill_then_decode(sdt):
    """A prefill into a pool of slots (one padding entry), then decode steps from it, as a
    server runs them; untouched slots keep their bits."""
    need_gpu()
    say("linattn pool", sdt)
    H, Hk, N = 4, 2, 3
    q, k, v, g, cu, _ = _draw([66, 5, 40], H, Hk, 128, 128, BF, "mild", 9, state=False)
    gen = torch.Generator().manual_seed(1)
    pool = torch.randn(6, H, 128, 128, generator=gen).to(sdt)
    idx = [4, -1, 1]
    P = pool.to(DEV)
    ind = torch.tensor(idx, dtype=torch.int32, device=DEV)
    o, same = kda.linattn_chunk_prefill(*_gpu(q, k, v, g), **_cu(cu), initial_state=P,
                                        final_state=P, state_indices=ind)
    assert same is P
    S0 = torch.stack([pool[i] if i >= 0 else torch.zeros_like(pool[0]) for i in idx])
    got = torch.stack([P.cpu()[i] for i in idx if i >= 0])
    ref.check_forward(o, None, q, k, v, g, cu, S0)
    keep = [i for i in range(3) if idx[i] >= 0]
    _, wantS = ref.forward(q, k, v, g, cu, S0)
    _, absS = ref.forward(q.abs(), k.abs(), v.abs(), g, cu, S0.abs())
    ref.check("pool", got, wantS[keep], absS[keep], ref.rel_of(q, v, cu, 3), sdt)
    for step in range(3):
        q1, k1, v1, g1, _, _ = _draw([N], H, Hk, 128, 128, BF, "mild", 50 + step, state=False)
        before = P.cpu()
        o1 = kda.linattn_recurrent_decode(*_gpu(q1, k1, v1, g1), P, state_indices=ind, scale=0.5,
                                          o_dtype=F32)
        after = P.cpu()
        assert torch.all(o1[1] == 0)
        for n, s in enumerate(idx):
            if s < 0:
                continue
            args = (q1[n:n + 1], k1[n:n + 1], v1[n:n + 1], g1[n:n + 1], [0, 1])
            wo, wS = ref.forward(*args, before[s:s + 1], 0.5)
            ao, aS = ref.forward(*[x.abs() for x in args[:3]], g1[n:n + 1], [0, 1],
                                 before[s:s + 1].abs(), 0.5)
            # fp32 throughout: a few u a term, 128 terms a sum
            ref.check("decode o", o1[n:n + 1], wo, ao, 160 * ref.U, F32)
            ref.check("decode state", after[s:s + 1], wS, aS, 8 * ref.U, sdt)
        for s in (0, 2, 3, 5):
            assert torch.equal(after[s], pool[s])


@pytest.mark.parametrize("N, H, Hk, dk, dv", [(1, 1, 1, 128, 128), (3, 5, 5, 64, 128),
                                              (130, 4, 2, 128, 64), (600, 1, 1, 64, 64)])
@pytest.mark.parametrize("sdt", [F32, BF])
def test_decode(N, H, Hk, dk, dv, sdt):
    need_gpu()
    say("linattn decode", N, H, Hk, dk, dv, sdt)
    for dtype, decay in ((BF, "strong"), (F32, "head"), (BF, "gone")):
        q, k, v, g, _, _ = _draw([N], H, Hk, dk, dv, dtype, decay, 70 + N, state=False)
        S = torch.randn(N, H, dk, dv, generator=torch.Generator().manual_seed(2)).to(sdt)
        P = S.to(DEV)
        o = kda.linattn_recurrent_decode(*_gpu(q, k, v, g), P, scale=0.2)
        cu = list(range(N + 1))
        wo, wS = ref.forward(q, k, v, g, cu, S, 0.2)
        ao, aS = ref.forward(q.abs(), k.abs(), v.abs(), g, cu, S.abs(), 0.2)
        # exp's own error and its argument's, below 4 u, at each term
        say(ref.check("o", o, wo, ao, 160 * ref.U, dtype))
        say(ref.check("state", P, wS, aS, 8 * ref.U, sdt))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_backward(shape, dtype):
    need_gpu()
    lens, H, Hk, dk, dv = SHAPES[shape]
    say("linattn backward", SHAPES[shape], dtype)
    q, k, v, g, cu, S0 = _draw(lens, H, Hk, dk, dv, dtype, "mild", 300 + shape)
    gen = torch.Generator().manual_seed(shape)
    do = torch.randn(cu[-1], H, dv, generator=gen).to(dtype)
    dS = torch.randn(len(lens), H, dk, dv, generator=gen) * 0.1
    got = kda.linattn_chunk_prefill_backward(*_gpu(q, k, v, g, do), **_cu(cu),
                                             initial_state=S0.to(DEV), d_final_state=dS.to(DEV),
                                             scale=0.3, grad_dtype=F32)
    say(ref.check_backward(got, q, k, v, g, cu, do, S0, dS, 0.3))


@pytest.mark.parametrize("decay", ["strong", "none", "resets", "gone", "head"])
@pytest.mark.parametrize("terms", ["do", "dS", "both fp32"])
def test_backward_decays_and_terms(decay, terms):
    need_gpu()
    say("linattn backward", decay, terms)
    H, Hk = 4, 2
    q, k, v, g, cu, S0 = _draw([150, 1, 70], H, Hk, 128, 128, BF, decay, 400,
                               state=terms != "do")
    gen = torch.Generator().manual_seed(3)
    do = torch.randn(cu[-1], H, 128, generator=gen).to(F32 if terms == "both fp32" else BF)
    dS = torch.randn(3, H, 128, 128, generator=gen)
    do = None if terms == "dS" else do
    dS = None if terms == "do" else dS
    got = kda.linattn_chunk_prefill_backward(*_gpu(q, k, v, g, do), **_cu(cu),
                                             initial_state=None if S0 is None else S0.to(DEV),
                                             d_final_state=None if dS is None else dS.to(DEV),
                                             scale=1.5)
    assert got[0].dtype == BF
    say(ref.check_backward(got, q, k, v, g, cu, do, S0, dS, 1.5))


@pytest.mark.parametrize("H", [1, 40])
def test_backward_long(H):
    """Segments: cut sequences (H = 1) and dg's borders in sequences walked whole (H = 40)."""
    need_gpu()
    say("linattn backward long", H)
    lens = [2300, 30] if H == 1 else [2100]
    q, k, v, g, cu, S0 = _draw(lens, H, H, 64, 64, BF, "mild", 500)
    gen = torch.Generator().manual_seed(4)
    do = torch.randn(cu[-1], H, 64, generator=gen).to(BF)
    dS = torch.randn(len(lens), H, 64, 64, generator=gen)
    got = kda.linattn_chunk_prefill_backward(*_gpu(q, k, v, g, do), **_cu(cu),
                                             initial_state=S0.to(DEV), d_final_state=dS.to(DEV))
    say(ref.check_backward(got, q, k, v, g, cu, do, S0, dS))


# lens, H, Hk, dk, dv: more heads than the card's XCDs but no multiple of them, and the
# backward's workgroups in mixed order (88 heads); one long sequence of several, cut
# into segments, with heads that fill the XCDs unevenly; the same with dk != dv
UNEVEN = [
    ([70, 3], 88, 44, 128, 128),
    ([3200, 5, 7], 12, 3, 64, 64),
    ([1300, 0, 40], 9, 9, 128, 64),
]


@pytest.mark.parametrize("case", range(len(UNEVEN)))
def test_uneven_heads_and_lengths(case):
    need_gpu()
    lens, H, Hk, dk, dv = UNEVEN[case]
    say("linattn uneven", UNEVEN[case])
    q, k, v, g, cu, S0 = _draw(lens, H, Hk, dk, dv, BF, "mild", 550 + case)
    o, S = kda.linattn_chunk_prefill(*_gpu(q, k, v, g), **_cu(cu), initial_state=S0.to(DEV))
    say(ref.check_forward(o, S, q, k, v, g, cu, S0))
    gen = torch.Generator().manual_seed(case)
    do = torch.randn(cu[-1], H, dv, generator=gen).to(BF)
    dS = torch.randn(len(lens), H, dk, dv, generator=gen)
    got = kda.linattn_chunk_prefill_backward(*_gpu(q, k, v, g, do), **_cu(cu),
                                             initial_state=S0.to(DEV), d_final_state=dS.to(DEV))
    say(ref.check_backward(got, q, k, v, g, cu, do, S0, dS))


@pytest.mark.parametrize("decay", ["mild", "head"])
def test_a_first_token_has_no_decay_gradient(decay):
    """Sequences of one token from zeros: nothing decays, so dg is exactly 0 (its sums leave
    the pairs of a token with itself out, they do not cancel)."""
    need_gpu()
    say("linattn first tokens", decay)
    q, k, v, g, cu, _ = _draw([1, 0, 1, 1], 3, 3, 128, 64, BF, decay, 560, state=False)
    do = torch.randn(cu[-1], 3, 64, generator=torch.Generator().manual_seed(6)).to(BF)
    got = kda.linattn_chunk_prefill_backward(*_gpu(q, k, v, g, do), **_cu(cu))
    assert torch.equal(got[3].cpu(), torch.zeros_like(g))
    say(ref.check_backward(got[:3], q, k, v, g, cu, do))


def test_backward_is_deterministic_and_leaves_rows_behind():
    need_gpu()
    say("linattn backward twice")
    q, k, v, g, cu, S0 = _draw([300, 200], 4, 2, 128, 128, BF, "mild", 600)
    do = torch.randn(cu[-1], 4, 128, generator=torch.Generator().manual_seed(5)).to(BF)
    args = _gpu(q, k, v, g, do)
    a = kda.linattn_chunk_prefill_backward(*args, **_cu(cu), initial_state=S0.to(DEV))
    b = kda.linattn_chunk_prefill_backward(*args, **_cu(cu), initial_state=S0.to(DEV))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_streams_and_two_calls_at_once():
    """Calls on two other streams, at the same time, each with its own workspace."""
    need_gpu()
    say("linattn streams")
    draws = [_draw([2300], 2, 2, 128, 128, BF, "mild", 700 + i) for i in range(2)]
    dev = [_gpu(*d[:4]) for d in draws]
    alone = [kda.linattn_chunk_prefill(*x) for x in dev]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got[i] = kda.linattn_chunk_prefill(*dev[i])
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_replays_of_a_serving_step_and_a_training_step():
    """Decode and norm, and prefill, norm and their gradients, captured and replayed with
    eager work between: every replay equals the eager calls on the same inputs."""
    need_gpu()
    say("linattn graphs")
    H, T = 4, 200
    q, k, v, g, cu, S0 = _draw([120, 80], H, 2, 128, 128, BF, "mild", 800)
    do = torch.randn(T, H, 128, generator=torch.Generator().manual_seed(6)).to(BF).to(DEV)
    q, k, v, g, S0 = _gpu(q, k, v, g, S0)
    w = torch.rand(H, 128, device=DEV) + 0.5
    b = torch.rand(H, 128, device=DEV)
    cu_d = torch.tensor(cu, dtype=torch.int32, device=DEV)
    P = S0.clone()

    def train():
        o, S = kda.linattn_chunk_prefill(q, k, v, g, cu_seqlens=cu_d, initial_state=S0)
        y = kda.layernorm(o, w, b)
        dx, dw, db = kda.layernorm_backward(do, o, w)
        return (o, S, y, dw, db) + kda.linattn_chunk_prefill_backward(
            q, k, v, g, dx, cu_seqlens=cu_d, initial_state=S0)

    def serve():
        o = kda.linattn_recurrent_decode(q[:2], k[:2], v[:2], g[:2], P)
        return kda.layernorm(o, w, b), P

    train(), serve()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        t_out, s_out = train(), serve()
    for i in range(4):
        q.copy_(torch.roll(q, 1, 0))
        do.mul_(-1.0)
        P.copy_(S0)
        want_t = train()
        want_s = [x.clone() for x in serve()]
        torch.cuda.synchronize()
        P.copy_(S0)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(t_out, want_t):
            assert torch.equal(x, y), i
        for x, y in zip(s_out, want_s):
            assert torch.equal(x, y), i


def test_a_layer_from_prompt_to_tokens():
    """The operators as a layer uses them: norm of every head's output after the attention,
    prompts into a pool, then single tokens; the same tokens in one prefill give the same."""
    need_gpu()
    say("linattn layer")
    H, T, more = 4, 130, 5
    q, k, v, g, cu, _ = _draw([T + more], H, 2, 128, 128, BF, "mild", 900, state=False)
    q, k, v, g = _gpu(q, k, v, g)
    w = torch.rand(H, 128, device=DEV) + 0.5
    whole, S_all = kda.linattn_chunk_prefill(q, k, v, g, o_dtype=F32)
    o, pool = kda.linattn_chunk_prefill(q[:T], k[:T], v[:T], g[:T], o_dtype=F32)
    outs = [o] + [kda.linattn_recurrent_decode(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1],
                                               pool, o_dtype=F32) for t in range(T, T + more)]
    y = kda.layernorm(torch.cat(outs), w)
    qc, kc, vc, gc = (x.cpu() for x in (q, k, v, g))
    ref.check_forward(torch.cat(outs), pool, qc, kc, vc, gc, cu)
    ref.check_forward(whole, S_all, qc, kc, vc, gc, cu)
    want = ref.norm(torch.cat(outs).cpu(), w.cpu())
    assert ((y.cpu().double() - want).abs() <= 1e-5 * want.abs().max()).all()


def test_debug_mode_names_what_is_outside_the_domain(monkeypatch):
    need_gpu()
    say("linattn KDA_DEBUG")
    monkeypatch.setenv("KDA_DEBUG", "1")
    q, k, v, g, cu, S0 = _draw([70], 2, 2, 128, 64, BF, "mild", 11)
    args = _gpu(q, k, v, g)
    kda.linattn_chunk_prefill(*args, initial_state=S0.to(DEV))
    kda.linattn_chunk_prefill_backward(*args, args[2])
    bad = args[3].clone()
    bad[3, 1] = 0.5
    with pytest.raises(kda.KdaError, match="g not <= 0"):
        kda.linattn_chunk_prefill(*args[:3], bad)
    with pytest.raises(kda.KdaError, match="g not <= 0"):
        kda.linattn_recurrent_decode(args[0][:1], args[1][:1], args[2][:1], bad[3:4],
                                     S0.to(DEV))
    v2 = args[2].clone()
    v2[69, 1, 63] = float("inf")
    with pytest.raises(kda.KdaError, match="v not finite"):
        kda.linattn_chunk_prefill(args[0], args[1], v2, args[3])
    x = torch.ones(3, 64, device=DEV)
    x[2, 5] = float("nan")
    with pytest.raises(kda.KdaError, match="x not finite"):
        kda.layernorm(x)
