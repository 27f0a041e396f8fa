// Internal declarations of the per-head-decay linear attention and layer norm
// launchers (linattn_walk.hip, linattn_decode.hip, layernorm.hip).
#pragma once

#include "kda_internal.hpp"

namespace kda {
namespace linattn {

// A token tensor read by the kernels: element c of (token t, head h) is
// p[t * stride + (h / group) * d + c].
struct Operand {
  const void* p = nullptr;
  int64_t stride = 0;
  int group = 1;
  bool bf16 = false;
};

// g [T, H] (per_token) or [H]
struct Decay {
  const float* g = nullptr;
  bool per_token = false;
};

// The log-decays below this are taken as this (natural log; exp(-110) is 0 in fp32).
constexpr float kMinLogDecay = -110.0f;
__device__ __forceinline__ float clamp_log_decay(float g) {
  return g < kMinLogDecay ? kMinLogDecay : g;  // NaN stays NaN
}

// (sequence, head) pairs of a decode: 512 threads each in a launch of fewer than 2^32, in
// eights
constexpr int64_t kMaxDecodePairs = (int64_t(1) << 23) - 8;
hipError_t launch_decode(const Operand& q, const Operand& k, const Operand& v, const Decay& g,
                         void* pool, bool state_bf16, int64_t num_slots, const int32_t* slots,
                         void* o, bool o_bf16, int N, int H, int dk, int dv, float scale,
                         hipStream_t s);

// A packed batch: cu null means N sequences of T_tot / N tokens.
struct Problem {
  Decay g;
  const int32_t *cu, *cu_host;
  int N;
  int64_t T_tot;
  int H, Hk, dk, dv;
  float scale;
};
// Whether every launch of a call holds its work items (wide: an fp32 operand).
bool prefill_fits(const Problem& p, bool wide);
bool backward_fits(const Problem& p, bool wide);
size_t prefill_workspace_bytes(int64_t T_tot, int N, int H, int dk, int dv);
// ws may be null or short: sequences are then walked whole.
hipError_t launch_prefill(const Problem& p, const Operand& q, const Operand& k, const Operand& v,
                          const StatePool& st, void* o, bool o_bf16, void* ws, size_t ws_bytes,
                          hipStream_t s);
size_t backward_workspace_bytes(int64_t T_tot, int N, int H, int Hk, int dk, int dv);
hipError_t launch_backward(const Problem& p, const Operand& q, const Operand& k, const Operand& v,
                           const float* S0, const Operand& d_o, const float* dS, void* dq, void* dk,
                           void* dv, bool grad_bf16, float* dg, float* dS0, void* ws,
                           hipStream_t s);

constexpr int kMaxCleared = 4;
hipError_t launch_zero_rows_behind(const int32_t* end, int T_tot, void* const* p,
                                   const int64_t* row_bytes, int count, hipStream_t s);

}  // namespace linattn

namespace norm {

constexpr int kMaxD = 16384;

hipError_t launch_forward(const void* x, bool x_bf16, const float* w, const float* b,
                          int64_t groups, void* y, bool y_bf16, int64_t rows, int d, float eps,
                          hipStream_t s);
size_t backward_workspace_bytes(int64_t rows, int64_t groups, int d);
hipError_t launch_backward(const void* dy, bool dy_bf16, const void* x, bool x_bf16,
                           const float* w, int64_t groups, void* dx, float* dw, float* db,
                           int64_t rows, int d, float eps, void* ws, hipStream_t s);

}  // namespace norm
}  // namespace kda
