// C ABI of kda_gatedrec.h: argument validation and launches.  As in api.hip, every argument
// is checked before the first HIP call, and nothing is thrown across the boundary.
#include "api_common.hpp"
#include "gatedrec.hpp"
#include "kda_gatedrec.h"

namespace {

using kda::api::aligned;
using kda::api::check_apart;
using kda::api::check_batch;
using kda::api::fail;
using kda::api::guarded;
using kda::api::known_dtype;
using kda::api::of_sequences;
using kda::api::ok;
using kda::api::overlap;
using kda::api::run_checked;
using kda::api::size_of;
using kda::api::Span;
using kda::dbg::kFinite;
using kda::dbg::kNonPositive;
using kda::dbg::kNotNaN;

constexpr int64_t kMaxStride = int64_t(1) << 24;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

// What the three calls of the recurrence have in common; `rows` is the token (sequence) axis.
struct Inputs {
  const void* x;
  int64_t xs;
  const void* r;
  int64_t rs;
  const void* i;
  int64_t is;
  kda_dtype dt;
  const float *A_log, *dt_bias;
  int32_t normalize;
  int64_t rows;
  int32_t C;
  Span span(const void* p, int64_t stride) const {
    return {p, rows > 0 ? ((size_t)(rows - 1) * stride + C) * size_of(dt) : 0};
  }
  Span span_x() const { return span(x, xs); }
  Span span_r() const { return span(r, rs); }
  Span span_i() const { return span(i, is); }
  Span span_A() const { return {A_log, (size_t)C * 4}; }
  Span span_b() const { return {dt_bias, (size_t)C * 4}; }
  kda::gatedrec::Inputs device() const {
    kda::gatedrec::Inputs d;
    d.x = {x, xs};
    d.r = {r, rs};
    d.i = {i, i ? is : 0};
    d.bf16 = dt == KDA_BF16;
    d.A_log = A_log;
    d.dt_bias = dt_bias;
    d.normalize = normalize != 0;
    return d;
  }
  void scan(kda::dbg::Session& c, const kda::dbg::Rows& which) const {
    const bool b = dt == KDA_BF16;
    c.add_rows("x", x, rows, C, xs, b, kFinite, which);
    c.add_rows("r", r, rows, C, rs, b, A_log ? kNotNaN : kNonPositive, which);
    if (i) c.add_rows("i", i, rows, C, is, b, kNotNaN, which);
    if (A_log) c.add("A_log", A_log, C, false, kFinite);
    if (dt_bias) c.add("dt_bias", dt_bias, C, false, kFinite);
  }
};

kda_status check_inputs(const char* fn, const Inputs& a) {
  if (a.C <= 0 || a.rows < 0)
    return fail(KDA_ERR_INVALID_ARG, "%s: need C > 0 and no negative length", fn);
  if (!known_dtype(a.dt)) return fail(KDA_ERR_DTYPE, "%s: in_dt must be KDA_F32 or KDA_BF16", fn);
  if (a.C > kda::gatedrec::kMaxC)
    return fail(KDA_ERR_UNSUPPORTED, "%s: need C <= %d", fn, kda::gatedrec::kMaxC);
  if (a.rows > kMaxRows)
    return fail(KDA_ERR_UNSUPPORTED, "%s: the number of rows must fit in int32", fn);
  if (a.normalize != 0 && a.normalize != 1)
    return fail(KDA_ERR_INVALID_ARG, "%s: normalize must be 0 or 1", fn);
  if (a.dt_bias && !a.A_log)
    return fail(KDA_ERR_INVALID_ARG, "%s: dt_bias without A_log (r is the log-decay then)", fn);
  if (a.xs < a.C || a.rs < a.C || (a.i && a.is < a.C))
    return fail(KDA_ERR_SHAPE, "%s: the strides must be at least C = %d", fn, a.C);
  if (a.xs > kMaxStride || a.rs > kMaxStride || (a.i && a.is > kMaxStride))
    return fail(KDA_ERR_UNSUPPORTED, "%s: strides must be at most %lld elements", fn,
                (long long)kMaxStride);
  const size_t es = size_of(a.dt);
  if (!aligned(a.x, es) || !aligned(a.r, es) || !aligned(a.i, es) || !aligned(a.A_log, 4) ||
      !aligned(a.dt_bias, 4))
    return fail(KDA_ERR_ALIGNMENT, "%s: tensors must be aligned to their element size", fn);
  if (a.rows > 0 && (!a.x || !a.r))
    return fail(KDA_ERR_INVALID_ARG, "%s: x and r must be non-NULL", fn);
  return KDA_OK;
}

kda_status check_pool(const char* fn, bool states, int64_t num_slots, const int32_t* state_indices,
                      int32_t N, int32_t C) {
  if (num_slots < 0)
    return fail(KDA_ERR_INVALID_ARG, "%s: num_slots must be >= 0 (got %lld)", fn,
                (long long)num_slots);
  if (num_slots > ((int64_t)1 << 58) / C)
    return fail(KDA_ERR_UNSUPPORTED, "%s: num_slots = %lld is more than memory holds", fn,
                (long long)num_slots);
  if (states && !state_indices && num_slots < N)
    return fail(KDA_ERR_SHAPE, "%s: without state_indices sequence n uses slot n, so num_slots "
                               "must be >= N (got %lld < %d)", fn, (long long)num_slots, N);
  if (!aligned(state_indices, 4))
    return fail(KDA_ERR_ALIGNMENT, "%s: state_indices must be 4-byte aligned", fn);
  return KDA_OK;
}

kda_status too_large(const char* fn, int64_t T, int32_t C) {
  return fail(KDA_ERR_UNSUPPORTED, "%s: T_tot = %lld tokens of C = %d channels are more than a "
                                   "launch holds", fn, (long long)T, C);
}

bool plausible(int64_t T_tot, int32_t C, bool (*fits)(const kda::gatedrec::Batch&)) {
  if (T_tot < 0 || T_tot > kMaxRows || C <= 0 || C > kda::gatedrec::kMaxC) return false;
  kda::gatedrec::Batch b;
  b.T = (int)T_tot;
  b.C = C;
  return fits(b);
}

}  // namespace

extern "C" {

size_t kda_gatedrec_scan_workspace_bytes(int64_t T_tot, int32_t C) {
  return plausible(T_tot, C, kda::gatedrec::scan_fits)
             ? kda::gatedrec::scan_workspace_bytes(T_tot, C)
             : 0;
}

size_t kda_gatedrec_starts_bytes(int64_t T_tot, int32_t C) {
  return plausible(T_tot, C, kda::gatedrec::scan_fits) ? kda::gatedrec::starts_bytes(T_tot, C) : 0;
}

kda_status kda_gatedrec_scan(const void* x, int64_t x_stride, const void* r, int64_t r_stride,
                             const void* i, int64_t i_stride, kda_dtype in_dt, const float* A_log,
                             const float* dt_bias, int32_t normalize, const int32_t* cu_seqlens,
                             const int32_t* cu_seqlens_host, int32_t N, const void* initial_state,
                             void* final_state, kda_dtype state_dt, int64_t num_slots,
                             const int32_t* state_indices, void* h, kda_dtype h_dt, float* starts,
                             int64_t T_tot, int32_t C, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const char* fn = "kda_gatedrec_scan";
  return guarded(fn, [&]() -> kda_status {
    const Inputs in{x, x_stride, r, r_stride, i, i_stride, in_dt, A_log, dt_bias, normalize, T_tot, C};
    if (const kda_status st = check_inputs(fn, in)) return st;
    if (const kda_status st = check_batch(fn, T_tot, N, cu_seqlens, cu_seqlens_host)) return st;
    kda::gatedrec::Batch b;
    b.cu = cu_seqlens;
    b.cu_host = cu_seqlens_host;
    b.N = N;
    b.T = (int)T_tot;
    b.C = C;
    if (!kda::gatedrec::scan_fits(b)) return too_large(fn, T_tot, C);
    if (!known_dtype(h_dt) || !known_dtype(state_dt))
      return fail(KDA_ERR_DTYPE, "%s: h_dt and state_dt must be KDA_F32 or KDA_BF16", fn);
    if (const kda_status st =
            check_pool(fn, initial_state || final_state, num_slots, state_indices, N, C))
      return st;
    if (T_tot > 0 && !h) return fail(KDA_ERR_INVALID_ARG, "%s: h must be non-NULL", fn);
    const size_t ss = size_of(state_dt);
    if (!aligned(h, size_of(h_dt)) || !aligned(initial_state, ss) || !aligned(final_state, ss) ||
        !aligned(starts, 4))
      return fail(KDA_ERR_ALIGNMENT, "%s: tensors must be aligned to their element size", fn);
    const size_t need = kda::gatedrec::scan_workspace_bytes(T_tot, C);
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(KDA_ERR_WORKSPACE, "%s: need a workspace of at least %zu bytes (got %zu at %p)",
                  fn, need, workspace_bytes, workspace);
    if (!aligned(workspace, 16))
      return fail(KDA_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", fn);
    const size_t st_bytes = (size_t)num_slots * C * ss;
    const Span sh{h, (size_t)T_tot * C * size_of(h_dt)}, sf{final_state, st_bytes},
        si{initial_state, st_bytes}, sw{workspace, need},
        sx{state_indices, state_indices ? (size_t)N * 4 : 0},
        sc{cu_seqlens, cu_seqlens ? ((size_t)N + 1) * 4 : 0},
        ss_{starts, kda::gatedrec::starts_bytes(T_tot, C)};
    if (const kda_status st =
            check_apart(fn, "h", sh, {in.span_x(), in.span_r(), in.span_i(), in.span_A(),
                                      in.span_b(), sf, si, sw, sx, sc, ss_}))
      return st;
    if (const kda_status st = check_apart(fn, "the final-state pool", sf,
                                          {in.span_x(), in.span_r(), in.span_i(), in.span_A(),
                                           in.span_b(), sw, sx, sc, ss_}))
      return st;
    if (final_state && final_state != initial_state && overlap(sf, si))
      return fail(KDA_ERR_INVALID_ARG, "%s: the state pools overlap without being the same", fn);
    if (const kda_status st = check_apart(fn, "starts", ss_,
                                          {in.span_x(), in.span_r(), in.span_i(), in.span_A(),
                                           in.span_b(), si, sw, sx, sc}))
      return st;
    if (const kda_status st = check_apart(fn, "the workspace", sw,
                                          {in.span_x(), in.span_r(), in.span_i(), in.span_A(),
                                           in.span_b(), si, sx, sc}))
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
          c.add_states("initial_state", initial_state, pool.bf16, state_indices, pool.slots, N, 1, C);
        },
        [&] {
          return kda::gatedrec::launch_scan(in.device(), b, pool, h, h_dt == KDA_BF16, starts,
                                            workspace, s);
        },
        [&](kda::dbg::Session& c) {
          c.add_rows("h", h, T_tot, C, C, h_dt == KDA_BF16, kFinite, of_sequences(cu_seqlens, N));
          c.add_states("final_state", final_state, pool.bf16, state_indices, pool.slots, N, 1, C);
        });
  });
}

size_t kda_gatedrec_scan_backward_workspace_bytes(int64_t T_tot, int32_t C, int32_t has_starts) {
  return plausible(T_tot, C, kda::gatedrec::backward_fits)
             ? kda::gatedrec::backward_workspace_bytes(T_tot, C, has_starts != 0)
             : 0;
}

kda_status kda_gatedrec_scan_backward(
    const void* x, int64_t x_stride, const void* r, int64_t r_stride, const void* i,
    int64_t i_stride, kda_dtype in_dt, const float* A_log, const float* dt_bias, int32_t normalize,
    const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, int32_t N,
    const float* initial_state, const float* starts, const void* dh, kda_dtype dh_dt,
    const float* d_final_state, void* dx, void* dr, void* di, kda_dtype grad_dt, float* dA_log,
    float* ddt_bias, float* d_initial_state, int64_t T_tot, int32_t C, void* workspace,
    size_t workspace_bytes, void* stream) {
  const char* fn = "kda_gatedrec_scan_backward";
  return guarded(fn, [&]() -> kda_status {
    const Inputs in{x, x_stride, r, r_stride, i, i_stride, in_dt, A_log, dt_bias, normalize, T_tot, C};
    if (const kda_status st = check_inputs(fn, in)) return st;
    if (const kda_status st = check_batch(fn, T_tot, N, cu_seqlens, cu_seqlens_host)) return st;
    if (!known_dtype(dh_dt) || !known_dtype(grad_dt))
      return fail(KDA_ERR_DTYPE, "%s: dh_dt and grad_dt must be KDA_F32 or KDA_BF16", fn);
    kda::gatedrec::Batch b;
    b.cu = cu_seqlens;
    b.cu_host = cu_seqlens_host;
    b.N = N;
    b.T = (int)T_tot;
    b.C = C;
    if (!kda::gatedrec::backward_fits(b)) return too_large(fn, T_tot, C);
    if (T_tot > 0 && (!dx || !dr || (i && !di)))
      return fail(KDA_ERR_INVALID_ARG, "%s: dx, dr and (with i) di must be non-NULL", fn);
    if (!i && di) return fail(KDA_ERR_INVALID_ARG, "%s: di without i", fn);
    if (!A_log && (dA_log || ddt_bias))
      return fail(KDA_ERR_INVALID_ARG, "%s: dA_log or ddt_bias without A_log", fn);
    const size_t ge = size_of(grad_dt);
    if (!aligned(dh, size_of(dh_dt)) || !aligned(dx, ge) || !aligned(dr, ge) || !aligned(di, ge) ||
        !aligned(initial_state, 4) || !aligned(starts, 4) || !aligned(d_final_state, 4) ||
        !aligned(dA_log, 4) || !aligned(ddt_bias, 4) || !aligned(d_initial_state, 4))
      return fail(KDA_ERR_ALIGNMENT, "%s: tensors must be aligned to their element size", fn);
    const size_t need = kda::gatedrec::backward_workspace_bytes(T_tot, C, starts != nullptr);
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(KDA_ERR_WORKSPACE, "%s: need a workspace of at least %zu bytes (got %zu at %p)",
                  fn, need, workspace_bytes, workspace);
    if (!aligned(workspace, 16))
      return fail(KDA_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", fn);
    const size_t n = (size_t)T_tot * C, st_bytes = (size_t)N * C * 4, par = (size_t)C * 4;
    const Span outs[] = {{dx, n * ge}, {dr, n * ge}, {di, n * ge}, {dA_log, par}, {ddt_bias, par},
                         {d_initial_state, st_bytes}, {workspace, workspace ? workspace_bytes : 0}};
    const Span ins[] = {in.span_x(), in.span_r(), in.span_i(), in.span_A(), in.span_b(),
                        {dh, n * size_of(dh_dt)}, {initial_state, st_bytes},
                        {starts, kda::gatedrec::starts_bytes(T_tot, C)}, {d_final_state, st_bytes},
                        {cu_seqlens, cu_seqlens ? ((size_t)N + 1) * 4 : 0}};
    for (size_t j = 0; j < sizeof(outs) / sizeof(outs[0]); ++j) {
      if (const kda_status st = check_apart(fn, "an output or the workspace", outs[j], ins))
        return st;
      for (size_t k = 0; k < j; ++k)
        if (overlap(outs[j], outs[k]))
          return fail(KDA_ERR_INVALID_ARG, "%s: two outputs, or an output and the workspace, overlap",
                      fn);
    }
    kda::gatedrec::Gradients out;
    out.dx = dx;
    out.dr = dr;
    out.di = di;
    out.bf16 = grad_dt == KDA_BF16;
    out.dA_log = dA_log;
    out.ddt_bias = ddt_bias;
    out.dS0 = d_initial_state;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const kda::dbg::Rows which = of_sequences(cu_seqlens, N);
    return run_checked(
        fn, s,
        [&](kda::dbg::Session& c) {
          in.scan(c, which);
          if (dh) c.add_rows("dh", dh, T_tot, C, C, dh_dt == KDA_BF16, kFinite, which);
          c.add_states("initial_state", initial_state, false, nullptr, N, N, 1, C);
          c.add_states("d_final_state", d_final_state, false, nullptr, N, N, 1, C);
        },
        [&] {
          return kda::gatedrec::launch_backward(in.device(), b, initial_state, starts, dh,
                                                dh_dt == KDA_BF16, d_final_state, out, workspace, s);
        },
        [&](kda::dbg::Session& c) {
          c.add_rows("dx", dx, T_tot, C, C, out.bf16, kFinite, which);
          c.add_rows("dr", dr, T_tot, C, C, out.bf16, kFinite, which);
          if (di) c.add_rows("di", di, T_tot, C, C, out.bf16, kFinite, which);
          if (dA_log) c.add("dA_log", dA_log, C, false, kFinite);
          if (ddt_bias) c.add("ddt_bias", ddt_bias, C, false, kFinite);
          c.add_states("d_initial_state", d_initial_state, false, nullptr, N, N, 1, C);
        });
  });
}

kda_status kda_gatedrec_decode(const void* x, int64_t x_stride, const void* r, int64_t r_stride,
                               const void* i, int64_t i_stride, kda_dtype in_dt,
                               const float* A_log, const float* dt_bias, int32_t normalize,
                               void* state, kda_dtype state_dt, int64_t num_slots,
                               const int32_t* state_indices, void* h, kda_dtype h_dt, int32_t N,
                               int32_t C, void* stream) {
  const char* fn = "kda_gatedrec_decode";
  return guarded(fn, [&]() -> kda_status {
    const Inputs in{x, x_stride, r, r_stride, i, i_stride, in_dt, A_log, dt_bias, normalize, N, C};
    if (const kda_status st = check_inputs(fn, in)) return st;
    if (!known_dtype(h_dt) || !known_dtype(state_dt))
      return fail(KDA_ERR_DTYPE, "%s: h_dt and state_dt must be KDA_F32 or KDA_BF16", fn);
    if (const kda_status st = check_pool(fn, true, num_slots, state_indices, N, C)) return st;
    if (N == 0) return ok();
    if (!h || (num_slots > 0 && !state))
      return fail(KDA_ERR_INVALID_ARG, "%s: state and h must be non-NULL", fn);
    if (!aligned(h, size_of(h_dt)) || !aligned(state, size_of(state_dt)))
      return fail(KDA_ERR_ALIGNMENT, "%s: tensors must be aligned to their element size", fn);
    if ((int64_t)N * (((int64_t)C + 255) / 256) > kda::gatedrec::kMaxDecodeGroups)
      return fail(KDA_ERR_UNSUPPORTED, "%s: need N * ceil(C / 256) <= %lld", fn,
                  (long long)kda::gatedrec::kMaxDecodeGroups);
    const Span sp{state, (size_t)num_slots * C * size_of(state_dt)},
        sh{h, (size_t)N * C * size_of(h_dt)},
        sx{state_indices, state_indices ? (size_t)N * 4 : 0};
    if (const kda_status st =
            check_apart(fn, "the state pool", sp, {in.span_x(), in.span_r(), in.span_i(),
                                                   in.span_A(), in.span_b(), sh, sx}))
      return st;
    if (const kda_status st = check_apart(fn, "h", sh, {in.span_x(), in.span_r(), in.span_i(),
                                                        in.span_A(), in.span_b(), sx}))
      return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool sb = state_dt == KDA_BF16;
    return run_checked(
        fn, s,
        [&](kda::dbg::Session& c) {
          in.scan(c, {nullptr, state_indices, num_slots});
          c.add_states("state", state, sb, state_indices, num_slots, N, 1, C);
        },
        [&] {
          return kda::gatedrec::launch_decode(in.device(), N, C, state, sb, num_slots,
                                              state_indices, h, h_dt == KDA_BF16, s);
        },
        [&](kda::dbg::Session& c) {
          c.add("h", h, (int64_t)N * C, h_dt == KDA_BF16, kFinite);
          c.add_states("state", state, sb, state_indices, num_slots, N, 1, C);
        });
  });
}

}  // extern "C"

namespace {

// What the RMS norm's calls have in common: rows of d in tokens of `groups`.
kda_status check_rows(const char* fn, int64_t rows, int64_t groups, int32_t d, float eps,
                      int64_t stride) {
  if (rows < 0 || groups <= 0 || d <= 0)
    return fail(KDA_ERR_INVALID_ARG, "%s: need rows >= 0, groups > 0, d > 0 (got %lld, %lld, %d)",
                fn, (long long)rows, (long long)groups, d);
  if (rows % groups)
    return fail(KDA_ERR_SHAPE, "%s: rows = %lld must be a multiple of groups = %lld", fn,
                (long long)rows, (long long)groups);
  if (d > kda::rms::kMaxD || groups > 65535)
    return fail(KDA_ERR_UNSUPPORTED, "%s: need d <= %d and groups <= 65535", fn, kda::rms::kMaxD);
  if (rows > ((int64_t)1 << 40))
    return fail(KDA_ERR_UNSUPPORTED, "%s: need rows <= 2^40", fn);
  if (stride < groups * d)
    return fail(KDA_ERR_SHAPE, "%s: the stride must be at least groups*d = %lld (got %lld)", fn,
                (long long)(groups * d), (long long)stride);
  if (stride > ((int64_t)1 << 31))
    return fail(KDA_ERR_UNSUPPORTED, "%s: the stride must be at most 2^31 elements", fn);
  if (rows / groups > ((int64_t)1 << 60) / stride)
    return fail(KDA_ERR_UNSUPPORTED, "%s: the rows are more than memory holds", fn);
  if (!(eps >= 0.0f) || eps > 3.0e38f)
    return fail(KDA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  return KDA_OK;
}

Span strided(const void* p, int64_t rows, int64_t groups, int32_t d, int64_t stride, size_t es) {
  return {p, rows > 0 ? ((size_t)(rows / groups - 1) * stride + (size_t)groups * d) * es : 0};
}

// Checks and runs both forward calls; y_bytes: of one value of y.
kda_status rmsnorm(const char* fn, kda::rms::Forward& f, kda_dtype x_dt, kda_dtype res_dt,
                   size_t y_bytes, bool y_like_x, int64_t n_scales, void* stream) {
  if (const kda_status st = check_rows(fn, f.rows, f.groups, f.d, f.eps, f.x_stride)) return st;
  if (!known_dtype(x_dt) || !known_dtype(res_dt))
    return fail(KDA_ERR_DTYPE, "%s: x_dt and res_dt must be KDA_F32 or KDA_BF16", fn);
  if (f.res && res_dt != KDA_F32 && res_dt != x_dt)
    return fail(KDA_ERR_DTYPE, "%s: the residual must have x's dtype or KDA_F32", fn);
  if (f.rows == 0) return ok();
  if (!f.x || !f.y) return fail(KDA_ERR_INVALID_ARG, "%s: x and y must be non-NULL", fn);
  if ((f.res == nullptr) != (f.s == nullptr))
    return fail(KDA_ERR_INVALID_ARG, "%s: residual and s come together", fn);
  if (n_scales > 0 && !f.scales)
    return fail(KDA_ERR_INVALID_ARG, "%s: scales must be non-NULL", fn);
  if (!aligned(f.x, size_of(x_dt)) || !aligned(f.y, y_bytes) || !aligned(f.res, size_of(res_dt)) ||
      !aligned(f.s, size_of(res_dt)) || !aligned(f.w, 4) || !aligned(f.scales, 4))
    return fail(KDA_ERR_ALIGNMENT, "%s: tensors must be aligned to their element size", fn);
  const size_t n = (size_t)f.rows * f.d;
  const Span sx = strided(f.x, f.rows, f.groups, f.d, f.x_stride, size_of(x_dt)),
             sy{f.y, n * y_bytes}, sr{f.res, n * size_of(res_dt)}, ss{f.s, n * size_of(res_dt)},
             sw{f.w, (size_t)f.groups * f.d * 4}, sc{f.scales, (size_t)n_scales * 4};
  const bool dense = f.x_stride == f.groups * f.d || f.rows == f.groups;
  if (overlap(sy, sx) && !(f.y == f.x && dense && y_like_x))
    return fail(KDA_ERR_INVALID_ARG, "%s: y overlaps x without being it", fn);
  if (overlap(ss, sx) && !(f.s == f.x && dense && res_dt == x_dt))
    return fail(KDA_ERR_INVALID_ARG, "%s: s overlaps x without being it", fn);
  if (overlap(ss, sr) && f.s != f.res)
    return fail(KDA_ERR_INVALID_ARG, "%s: s overlaps residual without being it", fn);
  if (const kda_status st = check_apart(fn, "y", sy, {sr, ss, sw, sc})) return st;
  if (const kda_status st = check_apart(fn, "s", ss, {sw, sc})) return st;
  if (const kda_status st = check_apart(fn, "scales", sc, {sx, sr, sw})) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t tokens = f.rows / f.groups, width = f.groups * f.d;
  return run_checked(
      fn, s,
      [&](kda::dbg::Session& c) {
        c.add_rows("x", f.x, tokens, width, f.x_stride, f.x_bf16, kFinite);
        if (f.res) c.add("residual", f.res, (int64_t)n, f.res_bf16, kFinite);
        c.add("weight", f.w, width, false, kFinite);
      },
      [&] { return kda::rms::launch_forward(f, s); },
      [&](kda::dbg::Session& c) {
        if (n_scales > 0) c.add("scales", f.scales, n_scales, false, kFinite);
        else c.add("y", f.y, (int64_t)n, f.y_dt == kda::rms::Out::bf16, kFinite);
        if (f.s) c.add("s", f.s, (int64_t)n, f.res_bf16, kFinite);
      });
}

kda::rms::Forward forward_of(const void* x, kda_dtype x_dt, int64_t x_stride, const void* residual,
                             void* s, kda_dtype res_dt, const float* weight, int64_t groups,
                             void* y, int64_t rows, int32_t d, float eps) {
  kda::rms::Forward f;
  f.x = x;
  f.x_bf16 = x_dt == KDA_BF16;
  f.x_stride = x_stride;
  f.res = residual;
  f.s = s;
  f.res_bf16 = res_dt == KDA_BF16;
  f.w = weight;
  f.groups = groups;
  f.y = y;
  f.rows = rows;
  f.d = d;
  f.eps = eps;
  return f;
}

}  // namespace

extern "C" {

kda_status kda_rmsnorm(const void* x, kda_dtype x_dt, int64_t x_stride, const void* residual,
                       void* s, kda_dtype res_dt, const float* weight, int64_t groups, void* y,
                       kda_dtype y_dt, int64_t rows, int32_t d, float eps, void* stream) {
  const char* fn = "kda_rmsnorm";
  return guarded(fn, [&]() -> kda_status {
    if (!known_dtype(y_dt))
      return fail(KDA_ERR_DTYPE, "%s: y_dt must be KDA_F32 or KDA_BF16", fn);
    kda::rms::Forward f =
        forward_of(x, x_dt, x_stride, residual, s, res_dt, weight, groups, y, rows, d, eps);
    f.y_dt = y_dt == KDA_BF16 ? kda::rms::Out::bf16 : kda::rms::Out::f32;
    return rmsnorm(fn, f, x_dt, res_dt, size_of(y_dt), y_dt == x_dt, 0, stream);
  });
}

kda_status kda_rmsnorm_e4m3(const void* x, kda_dtype x_dt, int64_t x_stride, const void* residual,
                            void* s, kda_dtype res_dt, const float* weight, int64_t groups,
                            uint8_t* y, float* scales, int32_t scale_group, int64_t rows,
                            int32_t d, float eps, void* stream) {
  const char* fn = "kda_rmsnorm_e4m3";
  return guarded(fn, [&]() -> kda_status {
    if (scale_group != 0 && scale_group != 128)
      return fail(KDA_ERR_UNSUPPORTED, "%s: scale_group must be 128 or 0 (a scale a row)", fn);
    kda::rms::Forward f =
        forward_of(x, x_dt, x_stride, residual, s, res_dt, weight, groups, y, rows, d, eps);
    f.y_dt = kda::rms::Out::e4m3;
    f.scales = scales;
    f.row_scale = scale_group == 0;
    const int64_t per_row = scale_group == 0 ? 1 : ((int64_t)d + 127) / 128;
    return rmsnorm(fn, f, x_dt, res_dt, 1, false, rows > 0 && rows <= ((int64_t)1 << 40) ? rows * per_row : 0,
                   stream);
  });
}

size_t kda_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t groups, int32_t d) {
  if (rows < 0 || groups <= 0 || d <= 0 || d > kda::rms::kMaxD || groups > 65535 ||
      rows % groups || rows > ((int64_t)1 << 40))
    return 0;
  return kda::rms::backward_workspace_bytes(rows, groups, d);
}

kda_status kda_rmsnorm_backward(const void* dy, kda_dtype dy_dt, const void* s, kda_dtype s_dt,
                                int64_t s_stride, const float* weight, int64_t groups,
                                const void* d_residual, void* dx, float* dweight, int64_t rows,
                                int32_t d, float eps, void* workspace, size_t workspace_bytes,
                                void* stream) {
  const char* fn = "kda_rmsnorm_backward";
  return guarded(fn, [&]() -> kda_status {
    if (const kda_status st = check_rows(fn, rows, groups, d, eps, s_stride)) return st;
    if (!known_dtype(dy_dt) || !known_dtype(s_dt))
      return fail(KDA_ERR_DTYPE, "%s: the dtypes must be KDA_F32 or KDA_BF16", fn);
    if (rows > 0 && (!dy || !s || !dx))
      return fail(KDA_ERR_INVALID_ARG, "%s: dy, s and dx must be non-NULL", fn);
    if (!aligned(dy, size_of(dy_dt)) || !aligned(s, size_of(s_dt)) || !aligned(dx, size_of(s_dt)) ||
        !aligned(d_residual, size_of(s_dt)) || !aligned(weight, 4) || !aligned(dweight, 4))
      return fail(KDA_ERR_ALIGNMENT, "%s: tensors must be aligned to their element size", fn);
    const size_t need = dweight ? kda::rms::backward_workspace_bytes(rows, groups, d) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(KDA_ERR_WORKSPACE, "%s: need a workspace of at least %zu bytes (got %zu)", fn,
                  need, workspace_bytes);
    if (!aligned(workspace, 16))
      return fail(KDA_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", fn);
    const size_t n = (size_t)rows * d, es = size_of(s_dt);
    const bool dense = s_stride == groups * d || rows == groups;
    const Span sdx{dx, n * es}, sdy{dy, n * size_of(dy_dt)},
        ss = strided(s, rows, groups, d, s_stride, es), sdr{d_residual, n * es},
        sw{weight, (size_t)groups * d * 4}, sdw{dweight, (size_t)groups * d * 4},
        sws{workspace, need};
    if ((overlap(sdx, sdy) && !(dx == dy && s_dt == dy_dt)) ||
        (overlap(sdx, ss) && !(dx == s && dense)) || (overlap(sdx, sdr) && dx != d_residual))
      return fail(KDA_ERR_INVALID_ARG, "%s: dx overlaps dy, s or d_residual without being it", fn);
    if (const kda_status st = check_apart(fn, "dx", sdx, {sw, sdw, sws})) return st;
    if (const kda_status st = check_apart(fn, "dweight", sdw, {sdy, ss, sdr, sw, sws})) return st;
    if (const kda_status st = check_apart(fn, "the workspace", sws, {sdy, ss, sdr, sw})) return st;
    kda::rms::Backward b;
    b.dy = dy;
    b.dy_bf16 = dy_dt == KDA_BF16;
    b.x = s;
    b.x_bf16 = s_dt == KDA_BF16;
    b.x_stride = s_stride;
    b.w = weight;
    b.groups = groups;
    b.dres = d_residual;
    b.dx = dx;
    b.dw = dweight;
    b.rows = rows;
    b.d = d;
    b.eps = eps;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return run_checked(
        fn, st,
        [&](kda::dbg::Session& c) {
          c.add("dy", dy, (int64_t)n, b.dy_bf16, kFinite);
          c.add_rows("s", s, rows / groups, groups * d, s_stride, b.x_bf16, kFinite);
          if (d_residual) c.add("d_residual", d_residual, (int64_t)n, b.x_bf16, kFinite);
          c.add("weight", weight, groups * d, false, kFinite);
        },
        [&] { return kda::rms::launch_backward(b, workspace, st); },
        [&](kda::dbg::Session& c) {
          c.add("dx", dx, (int64_t)n, b.x_bf16, kFinite);
          c.add("dweight", dweight, groups * d, false, kFinite);
        });
  });
}

}  // extern "C"
