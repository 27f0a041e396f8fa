// Internal declarations of the gated linear recurrence and RMS norm launchers
// (gatedrec_scan.hip, gatedrec_backward.hip, gatedrec_decode.hip, rmsnorm.hip).
#pragma once

#include "kda_internal.hpp"

namespace kda {
namespace gatedrec {

// Rows of `C` values, `stride` values apart.
struct Rows {
  const void* p = nullptr;
  int64_t stride = 0;
};

// What a call reads of the layer: x, r and i (null: no input gate) of one
// dtype, the gate's parameters [C] (A_log null: r is the log-decay itself;
// dt_bias null: zeros) and whether m = sqrt(1 - exp(2 g)).
struct Inputs {
  Rows x, r, i;
  bool bf16 = false;
  const float *A_log = nullptr, *dt_bias = nullptr;
  bool normalize = false;
};

// A packed batch: cu null means N sequences of T / N tokens.
struct Batch {
  const int32_t *cu = nullptr, *cu_host = nullptr;
  int N = 0;
  int T = 0;
  int C = 0;
};

constexpr int kMaxC = 1 << 20;
constexpr int kStartsTokens = 32;  // tokens between two states of `starts`

// Whether the launches of a call hold its work items.
bool scan_fits(const Batch& b);
bool backward_fits(const Batch& b);
size_t starts_bytes(int64_t T, int64_t C);

size_t scan_workspace_bytes(int64_t T, int64_t C);
// h null: only starts are written.
hipError_t launch_scan(const Inputs& in, const Batch& b, const StatePool& st, void* h, bool h_bf16,
                       float* starts, void* ws, hipStream_t s);

struct Gradients {
  void *dx = nullptr, *dr = nullptr, *di = nullptr;
  bool bf16 = false;
  float *dA_log = nullptr, *ddt_bias = nullptr, *dS0 = nullptr;
};
size_t backward_workspace_bytes(int64_t T, int64_t C, bool has_starts);
hipError_t launch_backward(const Inputs& in, const Batch& b, const float* S0, const float* starts,
                           const void* dh, bool dh_bf16, const float* dS, const Gradients& out,
                           void* ws, hipStream_t s);

// workgroups of a decode: a sequence's channels, 256 threads each, fewer than 2^32 in a launch
constexpr int64_t kMaxDecodeGroups = (int64_t(1) << 24) - 1;
hipError_t launch_decode(const Inputs& in, int N, int C, void* pool, bool state_bf16,
                         int64_t num_slots, const int32_t* slots, void* h, bool h_bf16,
                         hipStream_t s);

}  // namespace gatedrec

namespace rms {

constexpr int kMaxD = 16384;

enum class Out { f32, bf16, e4m3 };
struct Forward {
  const void* x = nullptr;
  bool x_bf16 = false;
  int64_t x_stride = 0;  // between tokens (groups rows each)
  const void* res = nullptr;
  void* s = nullptr;  // res + x (written when res is there)
  bool res_bf16 = false;
  const float* w = nullptr;
  int64_t groups = 1;
  void* y = nullptr;
  Out y_dt = Out::f32;
  float* scales = nullptr;
  bool row_scale = false;  // one scale a row, not one for each 128 columns
  int64_t rows = 0;
  int d = 0;
  float eps = 0.f;
};
hipError_t launch_forward(const Forward& f, hipStream_t s);

struct Backward {
  const void* dy = nullptr;
  bool dy_bf16 = false;
  const void* x = nullptr;  // what was normalised
  bool x_bf16 = false;
  int64_t x_stride = 0;
  const float* w = nullptr;
  int64_t groups = 1;
  const void* dres = nullptr;  // gradient that the residual stream brings, of x's type
  void* dx = nullptr;          // of x's type
  float* dw = nullptr;
  int64_t rows = 0;
  int d = 0;
  float eps = 0.f;
};
size_t backward_workspace_bytes(int64_t rows, int64_t groups, int d);
hipError_t launch_backward(const Backward& b, void* ws, hipStream_t s);

}  // namespace rms
}  // namespace kda
