// Pieces shared by the C ABI's translation units (api.hip, linattn_api.hip):
// the last error's text, argument checks and the KDA_DEBUG wrapper.
#pragma once

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
