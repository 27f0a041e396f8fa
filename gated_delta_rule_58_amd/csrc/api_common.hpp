// Pieces shared by the C ABI's translation units (api.hip, linattn_api.hip,
// gatedrec_api.hip): the last error's text, argument checks and the KDA_DEBUG wrapper.
#pragma once

#include <exception>
#include <mutex>
#include <string>

#include "kda_internal.hpp"

namespace kda {
namespace api {

// Sets the thread's last error and returns st.
kda_status fail(kda_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
kda_status ok();  // clears the last error

inline bool aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline bool known_dtype(kda_dtype d) { return d == KDA_F32 || d == KDA_BF16; }

inline bool finite_scale(float s) { return s == s && s <= 3.0e38f && s >= -3.0e38f; }

inline size_t size_of(kda_dtype d) { return d == KDA_BF16 ? 2 : 4; }

struct Span {
  const void* p;
  size_t n;
};
inline bool overlap(const Span& a, const Span& b) {
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

// A packed batch of N sequences: its lengths, where the host knows them.
inline kda_status check_batch(const char* fn, int64_t T_tot, int32_t N, const int32_t* cu,
                              const int32_t* cu_host) {
  if (N <= 0) return fail(KDA_ERR_INVALID_ARG, "%s: need N > 0 (got %d)", fn, N);
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

// The rows of a packed batch that belong to a sequence.
inline dbg::Rows of_sequences(const int32_t* cu, int32_t N) {
  return {cu ? cu + N : nullptr, nullptr, 0};
}

// `out` must not touch any of the others.
template <int K>
kda_status check_apart(const char* fn, const char* what, const Span& out, const Span (&others)[K]) {
  for (const Span& s : others)
    if (overlap(out, s)) return fail(KDA_ERR_INVALID_ARG, "%s: %s overlaps another tensor", fn, what);
  return KDA_OK;
}

inline kda_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(KDA_ERR_LAUNCH, "%s: launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

// Runs a call's launches (`run`).  With KDA_DEBUG=1 `pre` first adds the scans
// of its inputs (a failure returns KDA_ERR_DOMAIN before `run`), and `post`
// the scans of its outputs after it (KDA_ERR_NONFINITE); the call then waits
// for its stream.
template <class Pre, class Run, class Post>
kda_status run_checked(const char* fn, hipStream_t s, Pre pre, Run run, Post post) {
  if (!dbg::enabled()) return launched(run(), fn);
  std::lock_guard<std::mutex> lock(dbg::mutex());
  dbg::Session ses(s);
  std::string rep;
  hipError_t e = ses.begin();
  if (e == hipSuccess) {
    pre(ses);
    e = ses.finish(&rep);
  }
  if (e != hipSuccess)
    return fail(KDA_ERR_LAUNCH, "%s (KDA_DEBUG): input scan failed: %s", fn, hipGetErrorString(e));
  if (!rep.empty())
    return fail(KDA_ERR_DOMAIN, "%s (KDA_DEBUG): %s; nothing was launched", fn, rep.c_str());
  e = run();
  if (e != hipSuccess) return launched(e, fn);
  e = ses.begin();
  if (e == hipSuccess) {
    post(ses);
    e = ses.finish(&rep);
  }
  if (e != hipSuccess)
    return fail(KDA_ERR_LAUNCH, "%s (KDA_DEBUG): output scan failed: %s", fn,
                hipGetErrorString(e));
  if (!rep.empty()) return fail(KDA_ERR_NONFINITE, "%s (KDA_DEBUG): %s", fn, rep.c_str());
  return ok();
}

}  // namespace api
}  // namespace kda
