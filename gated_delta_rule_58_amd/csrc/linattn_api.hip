// C ABI of kda_linattn.h: argument validation and launches.  As in api.hip,
// every argument is checked before the first HIP call, and nothing is thrown
// across the boundary.
#include <exception>

#include "api_common.hpp"
#include "kda_linattn.h"
#include "linattn.hpp"

namespace {

using kda::api::aligned;
using kda::api::fail;
using kda::api::finite_scale;
using kda::api::known_dtype;
using kda::api::ok;
using kda::api::run_checked;
using kda::dbg::kFinite;
using kda::dbg::kNonPositive;

constexpr int64_t kMaxStride = int64_t(1) << 22;  // 64 rows of fp32 stay below 2^30 bytes
constexpr int64_t kMaxHeads = 16384;

size_t size_of(kda_dtype d) { return d == KDA_BF16 ? 2 : 4; }

struct Span {
  const void* p;
  size_t n;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}

// Runs a C entry's body; an exception (the debug mode's strings and lock) becomes a status.
template <class Body>
kda_status guarded(const char* fn, Body body) {
  try {
    return body();
  } catch (const std::exception& e) {
    return fail(KDA_ERR_LAUNCH, "%s: %s", fn, e.what());
  } catch (...) {
    return fail(KDA_ERR_LAUNCH, "%s: unknown exception", fn);
  }
}

// What the three linear attention calls have in common; `rows` is the token
// (sequence) axis of q, k and v.
struct Inputs {
  const void* q;
  int64_t qs;
  const void* k;
  int64_t ks;
  const void* v;
  int64_t vs;
  kda_dtype dt;
  const float* g;
  int64_t g_len;
  int64_t rows;
  int32_t H, Hk, dk, dv;
  float scale;
  bool per_token() const { return g_len == rows * H; }
  size_t bytes(int64_t stride, int64_t width) const {
    return rows > 0 ? ((size_t)(rows - 1) * stride + width) * size_of(dt) : 0;
  }
  Span span_q() const { return {q, bytes(qs, (int64_t)Hk * dk)}; }
  Span span_k() const { return {k, bytes(ks, (int64_t)Hk * dk)}; }
  Span span_v() const { return {v, bytes(vs, (int64_t)H * dv)}; }
  kda::linattn::Operand op_q() const { return {q, qs, H / Hk, dt == KDA_BF16}; }
  kda::linattn::Operand op_k() const { return {k, ks, H / Hk, dt == KDA_BF16}; }
  kda::linattn::Operand op_v() const { return {v, vs, 1, dt == KDA_BF16}; }
  void scan(kda::dbg::Session& c, const kda::dbg::Rows& which) const {
    const bool b = dt == KDA_BF16;
    c.add_rows("q", q, rows, (int64_t)Hk * dk, qs, b, kFinite, which);
    c.add_rows("k", k, rows, (int64_t)Hk * dk, ks, b, kFinite, which);
    c.add_rows("v", v, rows, (int64_t)H * dv, vs, b, kFinite, which);
    if (per_token()) c.add_rows("g", g, rows, H, H, false, kNonPositive, which);
    else c.add("g", g, g_len, false, kNonPositive);
  }
};

// The rows of a packed batch that belong to a sequence.
kda::dbg::Rows of_sequences(const int32_t* cu, int32_t N) {
  return {cu ? cu + N : nullptr, nullptr, 0};
}

kda_status check_inputs(const char* fn, const Inputs& a) {
  if (a.H <= 0 || a.Hk <= 0 || a.rows < 0)
    return fail(KDA_ERR_INVALID_ARG, "%s: need H > 0, Hk > 0 and no negative length", fn);
  if (a.H % a.Hk != 0)
    return fail(KDA_ERR_SHAPE, "%s: H = %d must be a multiple of Hk = %d", fn, a.H, a.Hk);
  if (!known_dtype(a.dt)) return fail(KDA_ERR_DTYPE, "%s: qkv_dt must be KDA_F32 or KDA_BF16", fn);
  if ((a.dk != 64 && a.dk != 128) || (a.dv != 64 && a.dv != 128))
    return fail(KDA_ERR_UNSUPPORTED, "%s: dk and dv must be 64 or 128 (got %d, %d)", fn, a.dk, a.dv);
  if (a.H > kMaxHeads) return fail(KDA_ERR_UNSUPPORTED, "%s: need H <= 16384", fn);
  if (a.rows > ((int64_t)1 << 31) - 1)
    return fail(KDA_ERR_UNSUPPORTED, "%s: T_tot must fit in int32", fn);
  if (!finite_scale(a.scale)) return fail(KDA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
  if (a.g_len != a.H && a.g_len != a.rows * a.H)
    return fail(KDA_ERR_SHAPE, "%s: g has %lld values; it must be one per head (%d) or one per "
                               "token and head (%lld)", fn, (long long)a.g_len, a.H,
                (long long)a.rows * a.H);
  const int64_t least_qk = (int64_t)a.Hk * a.dk, least_v = (int64_t)a.H * a.dv;
  if (a.qs < least_qk || a.ks < least_qk || a.vs < least_v)
    return fail(KDA_ERR_SHAPE, "%s: the strides of q and k must be at least Hk*dk = %lld, that of "
                               "v at least H*dv = %lld", fn, (long long)least_qk,
                (long long)least_v);
  if (a.qs > kMaxStride || a.ks > kMaxStride || a.vs > kMaxStride)
    return fail(KDA_ERR_UNSUPPORTED, "%s: strides must be at most %lld elements", fn,
                (long long)kMaxStride);
  const int64_t per = a.dt == KDA_BF16 ? 8 : 4;
  if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || a.qs % per || a.ks % per ||
      a.vs % per)
    return fail(KDA_ERR_ALIGNMENT, "%s: every row of q, k and v must be 16-byte aligned", fn);
  if (!aligned(a.g, 4)) return fail(KDA_ERR_ALIGNMENT, "%s: g must be 4-byte aligned", fn);
  if (a.rows > 0 && (!a.q || !a.k || !a.v || !a.g))
    return fail(KDA_ERR_INVALID_ARG, "%s: q, k, v and g must be non-NULL", fn);
  return KDA_OK;
}

kda_status check_batch(const char* fn, int64_t T_tot, int32_t N, int32_t H, const int32_t* cu,
                       const int32_t* cu_host) {
  if (N <= 0) return fail(KDA_ERR_INVALID_ARG, "%s: need N > 0 (got %d)", fn, N);
  if ((int64_t)N * H > ((int64_t)1 << 24))
    return fail(KDA_ERR_UNSUPPORTED, "%s: need N*H <= 2^24", fn);
  if (!aligned(cu, 4)) return fail(KDA_ERR_ALIGNMENT, "%s: cu_seqlens must be 4-byte aligned", fn);
  if (!cu) {
    if (cu_host)
      return fail(KDA_ERR_INVALID_ARG, "%s: cu_seqlens_host without cu_seqlens", fn);
    if (T_tot % N)
      return fail(KDA_ERR_SHAPE, "%s: without cu_seqlens T_tot = %lld must be a multiple of N = %d",
                  fn, (long long)T_tot, N);
  }
  if (cu_host) {
    if (cu_host[0] != 0 || cu_host[N] != T_tot)
      return fail(KDA_ERR_SHAPE, "%s: cu_seqlens must start at 0 and end at T_tot = %lld "
                                 "(got %d .. %d)", fn, (long long)T_tot, cu_host[0], cu_host[N]);
    for (int32_t n = 0; n < N; ++n)
      if (cu_host[n + 1] < cu_host[n])
        return fail(KDA_ERR_SHAPE, "%s: cu_seqlens decreases at index %d", fn, n);
  }
  return KDA_OK;
}

kda_status too_large(const char* fn, int32_t N, int32_t H) {
  return fail(KDA_ERR_UNSUPPORTED, "%s: N = %d sequences of H = %d heads are more than a launch "
                                   "holds", fn, N, H);
}

// `out` must not touch any of the others.
template <int K>
kda_status check_apart(const char* fn, const char* what, const Span& out, const Span (&others)[K]) {
  for (const Span& s : others)
    if (overlap(out, s)) return fail(KDA_ERR_INVALID_ARG, "%s: %s overlaps another tensor", fn, what);
  return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_linattn_chunk_prefill_workspace_bytes(int64_t T_tot, int32_t N, int32_t H, int32_t dk,
                                                 int32_t dv) {
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128) || T_tot < 0 || N <= 0 || H <= 0 ||
      H > kMaxHeads || T_tot > ((int64_t)1 << 31) - 1)
    return 0;
  return kda::linattn::prefill_workspace_bytes(T_tot, N, H, dk, dv);
}

kda_status kda_linattn_chunk_prefill(const void* q, int64_t q_stride, const void* k,
                                     int64_t k_stride, const void* v, int64_t v_stride,
                                     kda_dtype qkv_dt, const float* g, int64_t g_len,
                                     const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                                     int32_t N, const void* initial_state, void* final_state,
                                     kda_dtype state_dt, int64_t num_slots,
                                     const int32_t* state_indices, void* o, kda_dtype o_dt,
                                     int64_t T_tot, int32_t H, int32_t Hk, int32_t dk, int32_t dv,
                                     float scale, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  const char* fn = "kda_linattn_chunk_prefill";
  return guarded(fn, [&]() -> kda_status {
    const Inputs in{q, q_stride, k, k_stride, v, v_stride, qkv_dt, g, g_len, T_tot, H, Hk, dk, dv,
                    scale};
    if (const kda_status st = check_inputs(fn, in)) return st;
    if (const kda_status st = check_batch(fn, T_tot, N, H, cu_seqlens, cu_seqlens_host)) return st;
    const kda::linattn::Problem p{{g, in.per_token()}, cu_seqlens, cu_seqlens_host, N, T_tot, H,
                                  Hk, dk, dv, scale};
    if (!kda::linattn::prefill_fits(p, qkv_dt == KDA_F32)) return too_large(fn, N, H);
    if (!known_dtype(o_dt) || !known_dtype(state_dt))
      return fail(KDA_ERR_DTYPE, "%s: o_dt and state_dt must be KDA_F32 or KDA_BF16", fn);
    if (num_slots < 0)
      return fail(KDA_ERR_INVALID_ARG, "%s: num_slots must be >= 0 (got %lld)", fn,
                  (long long)num_slots);
    if ((initial_state || final_state) && !state_indices && num_slots < N)
      return fail(KDA_ERR_SHAPE, "%s: without state_indices sequence n uses slot n, so num_slots "
                                 "must be >= N (got %lld < %d)", fn, (long long)num_slots, N);
    if (T_tot > 0 && !o) return fail(KDA_ERR_INVALID_ARG, "%s: o must be non-NULL", fn);
    if (!aligned(o, 16) || !aligned(initial_state, 16) || !aligned(final_state, 16))
      return fail(KDA_ERR_ALIGNMENT, "%s: o and the states must be 16-byte aligned", fn);
    if (!aligned(state_indices, 4))
      return fail(KDA_ERR_ALIGNMENT, "%s: state_indices must be 4-byte aligned", fn);
    if (!aligned(workspace, 256))
      return fail(KDA_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    const size_t st_bytes = (size_t)num_slots * H * dk * dv * size_of(state_dt);
    const Span so{o, (size_t)T_tot * H * dv * size_of(o_dt)}, sf{final_state, st_bytes},
        si{initial_state, st_bytes}, sw{workspace, workspace ? workspace_bytes : 0},
        sx{state_indices, state_indices ? (size_t)N * 4 : 0},
        sc{cu_seqlens, cu_seqlens ? (size_t)(N + 1) * 4 : 0}, sg{g, (size_t)g_len * 4};
    if (const kda_status st = check_apart(fn, "o", so, {in.span_q(), in.span_k(), in.span_v(), sg,
                                                        sf, si, sw, sx, sc}))
      return st;
    if (const kda_status st = check_apart(fn, "the final-state pool", sf,
                                          {in.span_q(), in.span_k(), in.span_v(), sg, sw, sx, sc}))
      return st;
    if (final_state && final_state != initial_state && overlap(sf, si))
      return fail(KDA_ERR_INVALID_ARG, "%s: the state pools overlap without being the same", fn);
    if (const kda_status st = check_apart(fn, "the workspace", sw,
                                          {in.span_q(), in.span_k(), in.span_v(), sg, si, sx, sc}))
      return st;
    kda::StatePool pool;
    pool.in = initial_state;
    pool.out = final_state;
    pool.idx = state_indices;
    pool.slots = state_indices ? num_slots : (num_slots < N ? num_slots : N);
    pool.bf16 = state_dt == KDA_BF16;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_checked(
        fn, s,
        [&](kda::dbg::Session& c) {
          in.scan(c, of_sequences(cu_seqlens, N));
          c.add_states("initial_state", initial_state, pool.bf16, state_indices, pool.slots, N, H,
                       dk * dv);
        },
        [&] {
          return kda::linattn::launch_prefill(p, in.op_q(), in.op_k(), in.op_v(), pool, o,
                                              o_dt == KDA_BF16, workspace, workspace_bytes, s);
        },
        [&](kda::dbg::Session& c) {
          c.add_rows("o", o, T_tot, (int64_t)H * dv, (int64_t)H * dv, o_dt == KDA_BF16, kFinite,
                     of_sequences(cu_seqlens, N));
          c.add_states("final_state", final_state, pool.bf16, state_indices, pool.slots, N, H,
                       dk * dv);
        });
  });
}

size_t kda_linattn_chunk_prefill_backward_workspace_bytes(int64_t T_tot, int32_t N, int32_t H,
                                                          int32_t Hk, int32_t dk, int32_t dv) {
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128) || T_tot < 0 || N <= 0 || H <= 0 ||
      Hk <= 0 || H % Hk || H > kMaxHeads || T_tot > ((int64_t)1 << 31) - 1)
    return 0;
  return kda::linattn::backward_workspace_bytes(T_tot, N, H, Hk, dk, dv);
}

kda_status kda_linattn_chunk_prefill_backward(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, kda_dtype qkv_dt, const float* g, int64_t g_len, const int32_t* cu_seqlens,
    const int32_t* cu_seqlens_host, int32_t N, const float* initial_state, const void* d_o,
    kda_dtype do_dt, const float* d_final_state, void* dq, void* dk, void* dv, kda_dtype grad_dt,
    float* dg, float* d_initial_state, int64_t T_tot, int32_t H, int32_t Hk, int32_t dk_dim,
    int32_t dv_dim, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "kda_linattn_chunk_prefill_backward";
  return guarded(fn, [&]() -> kda_status {
    const Inputs in{q, q_stride, k, k_stride, v, v_stride, qkv_dt, g, g_len, T_tot, H, Hk, dk_dim,
                    dv_dim, scale};
    if (const kda_status st = check_inputs(fn, in)) return st;
    if (const kda_status st = check_batch(fn, T_tot, N, H, cu_seqlens, cu_seqlens_host)) return st;
    if (!known_dtype(do_dt) || !known_dtype(grad_dt))
      return fail(KDA_ERR_DTYPE, "%s: do_dt and grad_dt must be KDA_F32 or KDA_BF16", fn);
    const kda::linattn::Problem p{{g, in.per_token()}, cu_seqlens, cu_seqlens_host, N, T_tot, H,
                                  Hk, dk_dim, dv_dim, scale};
    if (!kda::linattn::backward_fits(p, qkv_dt == KDA_F32 || (d_o && do_dt == KDA_F32)))
      return too_large(fn, N, H);
    if (T_tot > 0 && (!dq || !dk || !dv))
      return fail(KDA_ERR_INVALID_ARG, "%s: dq, dk and dv must be non-NULL", fn);
    if (g_len > 0 && !dg) return fail(KDA_ERR_INVALID_ARG, "%s: dg must be non-NULL", fn);
    if (g_len > 0 && !g) return fail(KDA_ERR_INVALID_ARG, "%s: g must be non-NULL", fn);
    const void* ptrs[] = {initial_state, d_o, d_final_state, dq, dk, dv, d_initial_state};
    for (const void* x : ptrs)
      if (!aligned(x, 16))
        return fail(KDA_ERR_ALIGNMENT, "%s: d_o, the states and the gradients must be 16-byte "
                                       "aligned", fn);
    if (!aligned(dg, 4)) return fail(KDA_ERR_ALIGNMENT, "%s: dg must be 4-byte aligned", fn);
    const size_t need =
        kda::linattn::backward_workspace_bytes(T_tot, N, H, Hk, dk_dim, dv_dim);
    if (!workspace || workspace_bytes < need)
      return fail(KDA_ERR_WORKSPACE, "%s: need a workspace of at least %zu bytes (got %zu at %p)",
                  fn, need, workspace_bytes, workspace);
    if (!aligned(workspace, 256))
      return fail(KDA_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    const size_t T = (size_t)T_tot, ge = size_of(grad_dt);
    const size_t st_bytes = (size_t)N * H * dk_dim * dv_dim * 4;
    const Span outs[] = {{dq, T * Hk * dk_dim * ge}, {dk, T * Hk * dk_dim * ge},
                         {dv, T * H * dv_dim * ge},  {dg, (size_t)g_len * 4},
                         {d_initial_state, st_bytes}, {workspace, workspace_bytes}};
    const Span ins[] = {in.span_q(), in.span_k(), in.span_v(), {g, (size_t)g_len * 4},
                        {d_o, T * H * dv_dim * size_of(do_dt)}, {initial_state, st_bytes},
                        {d_final_state, st_bytes},
                        {cu_seqlens, cu_seqlens ? (size_t)(N + 1) * 4 : 0}};
    for (size_t i = 0; i < sizeof(outs) / sizeof(outs[0]); ++i) {
      if (const kda_status st = check_apart(fn, "an output or the workspace", outs[i], ins))
        return st;
      for (size_t j = 0; j < i; ++j)
        if (overlap(outs[i], outs[j]))
          return fail(KDA_ERR_INVALID_ARG, "%s: two outputs, or an output and the workspace, overlap",
                      fn);
    }
    const kda::linattn::Operand od{d_o, (int64_t)H * dv_dim, 1, do_dt == KDA_BF16};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const kda::dbg::Rows which = of_sequences(cu_seqlens, N);
    const int64_t wqk = (int64_t)Hk * dk_dim, wv = (int64_t)H * dv_dim;
    return run_checked(
        fn, s,
        [&](kda::dbg::Session& c) {
          in.scan(c, which);
          c.add_rows("d_o", d_o, T_tot, wv, wv, do_dt == KDA_BF16, kFinite, which);
          c.add_states("initial_state", initial_state, false, nullptr, N, N, H, dk_dim * dv_dim);
          c.add_states("d_final_state", d_final_state, false, nullptr, N, N, H, dk_dim * dv_dim);
        },
        [&] {
          return kda::linattn::launch_backward(p, in.op_q(), in.op_k(), in.op_v(), initial_state,
                                               od, d_final_state, dq, dk, dv, grad_dt == KDA_BF16,
                                               dg, d_initial_state, workspace, s);
        },
        [&](kda::dbg::Session& c) {
          const bool b = grad_dt == KDA_BF16;
          c.add_rows("dq", dq, T_tot, wqk, wqk, b, kFinite, which);
          c.add_rows("dk", dk, T_tot, wqk, wqk, b, kFinite, which);
          c.add_rows("dv", dv, T_tot, wv, wv, b, kFinite, which);
          if (in.per_token()) c.add_rows("dg", dg, T_tot, H, H, false, kFinite, which);
          else c.add("dg", dg, g_len, false, kFinite);
          c.add_states("d_initial_state", d_initial_state, false, nullptr, N, N, H,
                       dk_dim * dv_dim);
        });
  });
}

kda_status kda_zero_rows_behind(const int32_t* cu_seqlens, int32_t N, int64_t T_tot,
                                void* const* tensors, const int64_t* row_bytes, int32_t count,
                                void* stream) {
  const char* fn = "kda_zero_rows_behind";
  return guarded(fn, [&]() -> kda_status {
    if (N < 0 || T_tot < 0 || count < 0)
      return fail(KDA_ERR_INVALID_ARG, "%s: need N, T_tot and count >= 0", fn);
    if (T_tot > ((int64_t)1 << 31) - 1 || count > kda::linattn::kMaxCleared)
      return fail(KDA_ERR_UNSUPPORTED, "%s: T_tot must fit in int32, count be at most %d", fn,
                  kda::linattn::kMaxCleared);
    if (!cu_seqlens || (count > 0 && (!tensors || !row_bytes)))
      return fail(KDA_ERR_INVALID_ARG, "%s: cu_seqlens, tensors and row_bytes must be non-NULL", fn);
    if (!aligned(cu_seqlens, 4))
      return fail(KDA_ERR_ALIGNMENT, "%s: cu_seqlens must be 4-byte aligned", fn);
    const Span sc{cu_seqlens, (size_t)(N + (int64_t)1) * 4};
    for (int32_t i = 0; i < count; ++i) {
      if (row_bytes[i] < 0 || row_bytes[i] % 4 || row_bytes[i] > ((int64_t)1 << 30))
        return fail(KDA_ERR_SHAPE, "%s: row_bytes must be a multiple of 4 and at most 2^30", fn);
      if (!tensors[i] && T_tot * row_bytes[i] > 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: tensor %d is NULL", fn, i);
      if (!aligned(tensors[i], 4))
        return fail(KDA_ERR_ALIGNMENT, "%s: the tensors must be 4-byte aligned", fn);
      if (overlap(sc, {tensors[i], (size_t)(T_tot * row_bytes[i])}))
        return fail(KDA_ERR_INVALID_ARG, "%s: tensor %d overlaps cu_seqlens", fn, i);
    }
    int64_t bytes = 0;
    for (int32_t i = 0; i < count; ++i) bytes += T_tot * row_bytes[i];
    if (bytes == 0) return ok();
    return kda::api::launched(
        kda::linattn::launch_zero_rows_behind(cu_seqlens + N, (int)T_tot, tensors, row_bytes, count,
                                              static_cast<hipStream_t>(stream)),
        fn);
  });
}

kda_status kda_linattn_recurrent_decode(const void* q, int64_t q_stride, const void* k,
                                        int64_t k_stride, const void* v, int64_t v_stride,
                                        kda_dtype qkv_dt, const float* g, int64_t g_len,
                                        void* state, kda_dtype state_dt, int64_t num_slots,
                                        const int32_t* state_indices, void* o, kda_dtype o_dt,
                                        int32_t N, int32_t H, int32_t Hk, int32_t dk, int32_t dv,
                                        float scale, void* stream) {
  const char* fn = "kda_linattn_recurrent_decode";
  return guarded(fn, [&]() -> kda_status {
    const Inputs in{q, q_stride, k, k_stride, v, v_stride, qkv_dt, g, g_len, N, H, Hk, dk, dv,
                    scale};
    if (const kda_status st = check_inputs(fn, in)) return st;
    if (!known_dtype(o_dt) || !known_dtype(state_dt))
      return fail(KDA_ERR_DTYPE, "%s: o_dt and state_dt must be KDA_F32 or KDA_BF16", fn);
    if (num_slots < 0)
      return fail(KDA_ERR_INVALID_ARG, "%s: num_slots must be >= 0 (got %lld)", fn,
                  (long long)num_slots);
    if (!state_indices && num_slots < N)
      return fail(KDA_ERR_SHAPE, "%s: without state_indices sequence n uses slot n, so num_slots "
                                 "must be >= N (got %lld < %d)", fn, (long long)num_slots, N);
    if (N == 0) return ok();
    if (!o || (num_slots > 0 && !state))
      return fail(KDA_ERR_INVALID_ARG, "%s: state and o must be non-NULL", fn);
    if (!aligned(o, 16) || !aligned(state, 16))
      return fail(KDA_ERR_ALIGNMENT, "%s: state and o must be 16-byte aligned", fn);
    if (!aligned(state_indices, 4))
      return fail(KDA_ERR_ALIGNMENT, "%s: state_indices must be 4-byte aligned", fn);
    if ((int64_t)N * H > kda::linattn::kMaxDecodePairs)
      return fail(KDA_ERR_UNSUPPORTED, "%s: need N*H <= %lld", fn,
                  (long long)kda::linattn::kMaxDecodePairs);
    const Span sp{state, (size_t)num_slots * H * dk * dv * size_of(state_dt)},
        so{o, (size_t)N * H * dv * size_of(o_dt)},
        sx{state_indices, state_indices ? (size_t)N * 4 : 0}, sg{g, (size_t)g_len * 4};
    if (const kda_status st = check_apart(fn, "the state pool", sp, {in.span_q(), in.span_k(),
                                                                     in.span_v(), sg, so, sx}))
      return st;
    if (const kda_status st = check_apart(fn, "o", so, {in.span_q(), in.span_k(), in.span_v(), sg,
                                                        sx}))
      return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool sb = state_dt == KDA_BF16;
    return run_checked(
        fn, s,
        [&](kda::dbg::Session& c) {
          in.scan(c, {nullptr, state_indices, num_slots});
          c.add_states("state", state, sb, state_indices, num_slots, N, H, dk * dv);
        },
        [&] {
          return kda::linattn::launch_decode(in.op_q(), in.op_k(), in.op_v(),
                                             {g, in.per_token()}, state, sb, num_slots,
                                             state_indices, o, o_dt == KDA_BF16, N, H, dk, dv,
                                             scale, s);
        },
        [&](kda::dbg::Session& c) {
          c.add("o", o, (int64_t)N * H * dv, o_dt == KDA_BF16, kFinite);
          c.add_states("state", state, sb, state_indices, num_slots, N, H, dk * dv);
        });
  });
}

}  // extern "C"

namespace {

kda_status check_norm(const char* fn, int64_t rows, int64_t groups, int32_t d, float eps,
                      kda_dtype a, kda_dtype b) {
  if (rows < 0 || groups <= 0 || d <= 0)
    return fail(KDA_ERR_INVALID_ARG, "%s: need rows >= 0, groups > 0, d > 0 (got %lld, %lld, %d)",
                fn, (long long)rows, (long long)groups, d);
  if (rows % groups)
    return fail(KDA_ERR_SHAPE, "%s: rows = %lld must be a multiple of groups = %lld", fn,
                (long long)rows, (long long)groups);
  if (!known_dtype(a) || !known_dtype(b))
    return fail(KDA_ERR_DTYPE, "%s: the dtypes must be KDA_F32 or KDA_BF16", fn);
  if (d > kda::norm::kMaxD || groups > 65535)
    return fail(KDA_ERR_UNSUPPORTED, "%s: need d <= %d and groups <= 65535", fn, kda::norm::kMaxD);
  if (rows > ((int64_t)1 << 40))
    return fail(KDA_ERR_UNSUPPORTED, "%s: need rows <= 2^40", fn);
  if (!(eps >= 0.0f) || eps > 3.0e38f)
    return fail(KDA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_layernorm(const void* x, kda_dtype x_dt, const float* weight, const float* bias,
                         int64_t groups, void* y, kda_dtype y_dt, int64_t rows, int32_t d,
                         float eps, void* stream) {
  const char* fn = "kda_layernorm";
  return guarded(fn, [&]() -> kda_status {
    if (const kda_status st = check_norm(fn, rows, groups, d, eps, x_dt, y_dt)) return st;
    if (rows == 0) return ok();
    if (!x || !y) return fail(KDA_ERR_INVALID_ARG, "%s: x and y must be non-NULL", fn);
    if (!aligned(x, size_of(x_dt)) || !aligned(y, size_of(y_dt)) || !aligned(weight, 4) ||
        !aligned(bias, 4))
      return fail(KDA_ERR_ALIGNMENT, "%s: tensors must be aligned to their element size", fn);
    const size_t n = (size_t)rows * d, nw = (size_t)groups * d * 4;
    const Span sy{y, n * size_of(y_dt)}, sx{x, n * size_of(x_dt)};
    if (overlap(sy, sx) && !(x == y && x_dt == y_dt))
      return fail(KDA_ERR_INVALID_ARG, "%s: y overlaps x without being it", fn);
    if (const kda_status st = check_apart(fn, "y", sy, {Span{weight, nw}, Span{bias, nw}}))
      return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_checked(
        fn, s,
        [&](kda::dbg::Session& c) {
          c.add("x", x, (int64_t)n, x_dt == KDA_BF16, kFinite);
          c.add("weight", weight, groups * d, false, kFinite);
          c.add("bias", bias, groups * d, false, kFinite);
        },
        [&] {
          return kda::norm::launch_forward(x, x_dt == KDA_BF16, weight, bias, groups, y,
                                           y_dt == KDA_BF16, rows, d, eps, s);
        },
        [&](kda::dbg::Session& c) { c.add("y", y, (int64_t)n, y_dt == KDA_BF16, kFinite); });
  });
}

size_t kda_layernorm_backward_workspace_bytes(int64_t rows, int64_t groups, int32_t d) {
  if (rows < 0 || groups <= 0 || d <= 0 || d > kda::norm::kMaxD || groups > 65535 ||
      rows % groups || rows > ((int64_t)1 << 40))
    return 0;
  return kda::norm::backward_workspace_bytes(rows, groups, d);
}

kda_status kda_layernorm_backward(const void* dy, kda_dtype dy_dt, const void* x, kda_dtype x_dt,
                                  const float* weight, int64_t groups, void* dx, float* dweight,
                                  float* dbias, int64_t rows, int32_t d, float eps,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "kda_layernorm_backward";
  return guarded(fn, [&]() -> kda_status {
    if (const kda_status st = check_norm(fn, rows, groups, d, eps, dy_dt, x_dt)) return st;
    if (rows > 0 && (!dy || !x || !dx))
      return fail(KDA_ERR_INVALID_ARG, "%s: dy, x and dx must be non-NULL", fn);
    if (!aligned(dy, size_of(dy_dt)) || !aligned(x, size_of(x_dt)) || !aligned(dx, size_of(x_dt)) ||
        !aligned(weight, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
      return fail(KDA_ERR_ALIGNMENT, "%s: tensors must be aligned to their element size", fn);
    const size_t need =
        dweight || dbias ? kda::norm::backward_workspace_bytes(rows, groups, d) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(KDA_ERR_WORKSPACE, "%s: need a workspace of at least %zu bytes (got %zu)", fn,
                  need, workspace_bytes);
    if (!aligned(workspace, 16))
      return fail(KDA_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", fn);
    const size_t n = (size_t)rows * d, nw = (size_t)groups * d * 4;
    const Span sdx{dx, n * size_of(x_dt)}, sdy{dy, n * size_of(dy_dt)}, sx{x, n * size_of(x_dt)},
        sw{weight, nw}, sdw{dweight, nw}, sdb{dbias, nw}, sws{workspace, need};
    if ((overlap(sdx, sdy) && !(dx == dy && x_dt == dy_dt)) || (overlap(sdx, sx) && dx != x))
      return fail(KDA_ERR_INVALID_ARG, "%s: dx overlaps dy or x without being it", fn);
    if (const kda_status st = check_apart(fn, "dx", sdx, {sw, sdw, sdb, sws})) return st;
    if (const kda_status st = check_apart(fn, "dweight", sdw, {sdy, sx, sw, sdb, sws})) return st;
    if (const kda_status st = check_apart(fn, "dbias", sdb, {sdy, sx, sw, sws})) return st;
    if (const kda_status st = check_apart(fn, "the workspace", sws, {sdy, sx, sw})) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_checked(
        fn, s,
        [&](kda::dbg::Session& c) {
          c.add("dy", dy, (int64_t)n, dy_dt == KDA_BF16, kFinite);
          c.add("x", x, (int64_t)n, x_dt == KDA_BF16, kFinite);
          c.add("weight", weight, groups * d, false, kFinite);
        },
        [&] {
          return kda::norm::launch_backward(dy, dy_dt == KDA_BF16, x, x_dt == KDA_BF16, weight,
                                            groups, dx, dweight, dbias, rows, d, eps, workspace, s);
        },
        [&](kda::dbg::Session& c) {
          c.add("dx", dx, (int64_t)n, x_dt == KDA_BF16, kFinite);
          c.add("dweight", dweight, groups * d, false, kFinite);
          c.add("dbias", dbias, groups * d, false, kFinite);
        });
  });
}

}  // extern "C"
