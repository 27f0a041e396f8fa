// kda_rmsnorm, kda_rmsnorm_e4m3 and kda_rmsnorm_backward: RMS norm over the rows of [rows, d].
//
//   forward   s = x + residual (rounded as it is stored);  y = s r w,  r = 1/sqrt(mean(s^2) + eps)
//   e4m3      scale = max |y| / 448 over 128 columns or the row;  q = y / scale
//   backward  ds = r (t - xh mean(t xh)) + d_residual,  xh = s r,  t = dy w;  dw = sum_rows dy xh
//
// HBM-bound: every tensor is read or written once, the row stays in registers between
// (norm_rows.hpp says how; as in layer norm, lanes walk down rows of one weight row, the
// next row on its way while this one is worked on).  The backward forms r again from s,
// which it reads anyway.  The sums that it makes of the rows go to memory once an owner and
// are added in a fixed order by a second kernel: the same call gives the same bits.
//
// bf16: 4,096 rows of 8,192 with the residual to 8 bits 47 us (5.0 TB/s; a scale a row the same),
// to bf16 51 us (5.3); the gradients of 4,096 x 96 rows of 128, a weight a head, 65 us (4.6); with
// the stream's gradient of 4,096 rows of 4,096 31 us (4.4), of 8,192 55 (4.9), of 12,288 88 (4.6);
// of 2,048 rows of 5,003 (nothing wider than two bytes aligned) 29 us (2.8), 4 of them the sums'
// kernel.  Above 8,192 columns the gradients' 1,024 lanes have 128 registers and spill 4 to 22 of
// them (20 to 60 B a lane).
#include "gatedrec.hpp"
#include "norm_rows.hpp"

namespace kda {
namespace rms {
namespace {

using norm::Eight;
using norm::f32x8;
using norm::lanes_of;
using norm::moved;
using norm::row_sum;
using norm::runs_of;
using norm::sum8;
using norm::threads;

constexpr float kE4m3Max = 448.0f;
// rows below this (all zeros, say) take it as their largest value: a scale that is not 0
constexpr float kLeastMax = 7.8886e-31f;  // 2^-100
constexpr int kGroup = 128;

typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

// The largest of the L lanes' bit patterns (of absolute values: a NaN is larger than any
// number, so that it stays).
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t x) {
  const uint32_t y = __float_as_uint(moved<CTRL>(__uint_as_float(x)));
  return x > y ? x : y;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
  x = max_with<0xb1>(x);
  x = max_with<0x4e>(x);
  if constexpr (L >= 8) x = max_with<0x141>(x);
  if constexpr (L >= 16) x = max_with<0x140>(x);
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = r[0] > r[1] ? r[0] : r[1];
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = r[0] > r[1] ? r[0] : r[1];
  }
  return x;
}
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t x, uint32_t* s_part) {
  x = lanes_max<(L < 64 ? L : 64)>(x);
  if constexpr (L > 64) {
    constexpr int W = L / 64;
    // (the sum of squares stands between this row's values and the last one's)
    if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = x;
    barrier_lds();
    x = lanes_max<W>(s_part[threadIdx.x & (W - 1)]);
  }
  return x;
}

__device__ __forceinline__ uint32_t max8(f32x8 x) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  return m;
}
__device__ __forceinline__ float largest(uint32_t bits) {
  const float m = __uint_as_float(bits);
  return m < kLeastMax ? kLeastMax : m;  // NaN stays NaN
}
// x / scale as e4m3, rounded to nearest even; |x| / scale is at most 448 (1 + 2^-23).  The
// quotient, not x (1 / scale), which rounds otherwise and beside the middle of two codes gives
// another code: t = x (1 / scale) is within 1.5 of its steps of the quotient, and t + (x - t scale)
// (1 / scale) within 2^-22 of one, rounded once.  fp32's own quotient could differ from that only
// where it comes so near to half a step beside a middle of two codes, which takes a scale within 8
// steps of k / 8 of a power of two; those were gone through on the CPU, and none differs.  (Where
// the largest |y| is below 2^-85 the difference is subnormal, and t + .. within 2^-6 of a step.)
// 4,096 x 8,192 bf16 with the residual: 42 us as with x (1 / scale), 49 with eight divisions;
// 393,216 x 128: 32.6, 30.5, 41.8.
__device__ __forceinline__ void store_e4m3(void* p, int64_t i, int n, f32x8 x, float scale) {
  uint8_t* d = static_cast<uint8_t*>(p) + i;
  const float inv = 1.0f / scale;
  const float s = fminf(scale, 3.4028235e38f);  // (an infinite scale leaves 0 of what is finite)
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = x[e] * inv;
    x[e] = fmaf(fmaf(-t, s, x[e]), inv, t);
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  if (n >= 8) {
    *reinterpret_cast<u32x2_a1*>(d) = u32x2_a1{(uint32_t)lo, (uint32_t)hi};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) d[e] = (uint8_t)((uint32_t)(e < 4 ? lo : hi) >> (8 * (e & 3)));
  }
}

// RES: 0 no residual, 1 bf16, 2 fp32.  Row owner q of Q walks rows q, q + Q, ... (Q a multiple
// of groups); row r is x's (token r / groups, group r % groups).
template <bool XB, int RES, int L, int M>
__global__ void __launch_bounds__(threads<L>()) forward_kernel(const Forward f, int64_t Q) {
  constexpr int RPB = threads<L>() / L;
  constexpr bool RB = RES == 1;
  __shared__ float s_part[L > 64 ? 2 * norm::kSums * (L / 64) : 1];
  __shared__ uint32_t s_max[L > 64 ? L / 64 : 1];
  const int l = threadIdx.x % L, d = f.d;
  const int64_t q = (int64_t)blockIdx.x * RPB + threadIdx.x / L;
  if (q >= Q || q >= f.rows) return;  // whole rows of lanes leave together (L > 64: the workgroup)
  int left[M];  // columns of each run that exist
  f32x8 ww[M];
  const int64_t grp = q % f.groups;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int c = (m * L + l) * 8;
    left[m] = d - c < 0 ? 0 : (d - c < 8 ? d - c : 8);
    Eight<false> t;
    ww[m] = f32x8(1.f);
    if (f.w) { t.load(f.w, grp * d + c, left[m]); ww[m] = t.get(); }
  }
  const float inv_d = 1.0f / d;
  int turn = 0;
  Eight<XB> rx[M];
  Eight<RB> rr[RES ? M : 1];
  int64_t at_x = q / f.groups * f.x_stride + grp * d;
  const int64_t step_x = Q / f.groups * f.x_stride;
  auto load = [&](int64_t r) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      rx[m].load(f.x, at_x + (m * L + l) * 8, left[m]);
      if constexpr (RES != 0) rr[m].load(f.res, r * d + (m * L + l) * 8, left[m]);
    }
    at_x += step_x;
  };
  load(q);
  for (int64_t r = q; r < f.rows; r += Q) {
    f32x8 v[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      v[m] = rx[m].get();
      if constexpr (RES != 0) {
        v[m] += rr[m].get();
        if constexpr (RB)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[m][e] = bf16_bits_to_f32(f32_to_bf16_bits(v[m][e]));
      }
    }
    if (r + Q < f.rows) load(r + Q);
    float s[1] = {0.f};
#pragma unroll
    for (int m = 0; m < M; ++m) {
      s[0] += sum8(v[m] * v[m]);
      if constexpr (RES != 0) Eight<RB>::store(f.s, r * d + (m * L + l) * 8, left[m], v[m]);
    }
    row_sum<L, 1>(s, s_part, turn);
    const float rstd = 1.0f / sqrtf(s[0] * inv_d + f.eps);
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = v[m] * rstd * ww[m];
    if (f.y_dt == Out::bf16) {
#pragma unroll
      for (int m = 0; m < M; ++m) Eight<true>::store(f.y, r * d + (m * L + l) * 8, left[m], v[m]);
    } else if (f.y_dt == Out::f32) {
#pragma unroll
      for (int m = 0; m < M; ++m) Eight<false>::store(f.y, r * d + (m * L + l) * 8, left[m], v[m]);
    } else if (f.row_scale) {
      uint32_t mx = 0;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const uint32_t b = max8(v[m]);
        mx = b > mx ? b : mx;
      }
      const float scale = largest(row_max<L>(mx, s_max)) / kE4m3Max;
      if (l == 0) f.scales[r] = scale;
#pragma unroll
      for (int m = 0; m < M; ++m) store_e4m3(f.y, r * d + (m * L + l) * 8, left[m], v[m], scale);
    } else {
      constexpr int GL = L < 16 ? L : 16;  // lanes of 128 columns
      const int64_t per_row = (d + kGroup - 1) / kGroup;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const float scale = largest(lanes_max<GL>(max8(v[m]))) / kE4m3Max;
        if (l % GL == 0 && left[m] > 0) f.scales[r * per_row + (m * L + l) / 16] = scale;
        store_e4m3(f.y, r * d + (m * L + l) * 8, left[m], v[m], scale);
      }
    }
  }
}

template <bool YB, bool XB, int L, int M>
__global__ void __launch_bounds__(threads<L>()) backward_kernel(const Backward f,
                                                                float* __restrict__ part,
                                                                int64_t Q) {
  constexpr int RPB = threads<L>() / L;
  __shared__ float s_part[L > 64 ? 2 * norm::kSums * (L / 64) : 1];
  const int l = threadIdx.x % L, d = f.d;
  const int64_t q = (int64_t)blockIdx.x * RPB + threadIdx.x / L;
  if (q >= Q || q >= f.rows) return;
  int left[M];
  f32x8 ww[M], dw[M];
  const int64_t grp = q % f.groups;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int c = (m * L + l) * 8;
    left[m] = d - c < 0 ? 0 : (d - c < 8 ? d - c : 8);
    Eight<false> t;
    ww[m] = f32x8(1.f);
    if (f.w) { t.load(f.w, grp * d + c, left[m]); ww[m] = t.get(); }
    dw[m] = f32x8(0.f);
  }
  const float inv_d = 1.0f / d;
  int turn = 0;
  constexpr bool AHEAD = L < 1024;  // 1,024 lanes have the registers of one row only
  Eight<XB> rx[M], rd[M];
  Eight<YB> ry[M];
  int64_t at_x = q / f.groups * f.x_stride + grp * d;
  const int64_t step_x = Q / f.groups * f.x_stride;
  auto load = [&](int64_t r) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      rx[m].load(f.x, at_x + (m * L + l) * 8, left[m]);
      ry[m].load(f.dy, r * d + (m * L + l) * 8, left[m]);
      if (f.dres) rd[m].load(f.dres, r * d + (m * L + l) * 8, left[m]);
    }
    at_x += step_x;
  };
  if (AHEAD) load(q);
  for (int64_t r = q; r < f.rows; r += Q) {
    if (!AHEAD) load(r);
    f32x8 v[M], g[M], more[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      v[m] = rx[m].get();
      g[m] = ry[m].get();
      more[m] = f.dres ? rd[m].get() : f32x8(0.f);
    }
    if (AHEAD && r + Q < f.rows) load(r + Q);
    float s[2] = {0.f, 0.f};  // of s^2 and of t s
#pragma unroll
    for (int m = 0; m < M; ++m) {
      s[0] += sum8(v[m] * v[m]);
      s[1] += sum8(g[m] * ww[m] * v[m]);
    }
    row_sum<L, 2>(s, s_part, turn);
    const float rstd = 1.0f / sqrtf(s[0] * inv_d + f.eps);
    const float mean = s[1] * inv_d * rstd;  // of t xh
#pragma unroll
    for (int m = 0; m < M; ++m) {
      v[m] = v[m] * rstd;
      dw[m] += g[m] * v[m];
      Eight<XB>::store(f.dx, r * d + (m * L + l) * 8, left[m],
                       rstd * (g[m] * ww[m] - v[m] * mean) + more[m]);
    }
  }
  if (part) {
#pragma unroll
    for (int m = 0; m < M; ++m) Eight<false>::store(part, q * d + (m * L + l) * 8, left[m], dw[m]);
  }
}

// dw [groups, d] from the partial rows [owners][d]: owner q belongs to weight row q % groups.
// 64 columns a workgroup, 16 owners in turn a column, added in order and in 64 bits: one after the
// other in fp32 the 8,192 owners of 65,536 rows of 128 lose 7 u (u = 2^-24) of the sum.
__global__ void __launch_bounds__(1024) partials_kernel(const float* __restrict__ part,
                                                        int64_t owners, int64_t groups, int d,
                                                        float* __restrict__ dw) {
  __shared__ double s[16][64];
  const int cl = threadIdx.x & 63, k = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + cl;
  const int64_t grp = blockIdx.y;
  double acc = 0.0;
  if (c < d)
    for (int64_t q = grp + groups * k; q < owners; q += groups * 16 * 8) {
      float x[8];  // eight loads on their way
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t at = q + groups * 16 * j;
        x[j] = at < owners ? part[at * d + c] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) hold(x[j]);  // (or each is waited for and widened where it is loaded)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc += x[j];
    }
  s[k][cl] = acc;
  __syncthreads();
  if (k == 0 && c < d) {
    for (int j = 1; j < 16; ++j) acc += s[j][cl];
    dw[grp * d + c] = (float)acc;
  }
}

int64_t forward_owners(int64_t rows, int64_t groups, int L) {
  return norm::owners(rows, groups, 256 * (L <= 512 ? 4096 : 2048) / L);
}
// An owner has at least eight rows, for it begins with its weights and ends with its sums, and
// there are no more than fill the card once.  Twice as many: 2,048 x 5,003 34 us beside 31, 4,096 x
// 96 rows of 128 66 beside 64, 4,096 x 4,096 40 beside 33.
int64_t backward_owners(int64_t rows, int64_t groups, int L, int M) {
  const int64_t one_each = 256 * (L < 256 ? 256 / L : 1);  // a workgroup a CU
  int64_t q = 256 * 1024 / (L * M);
  if (q > rows / 8) q = rows / 8;
  return norm::owners(rows, groups, q < one_each ? one_each : q);
}

}  // namespace

hipError_t launch_forward(const Forward& f, hipStream_t s) {
  if (f.rows == 0) return hipSuccess;
  const int d = f.d;
  const int64_t Q = forward_owners(f.rows, f.groups, lanes_of(d));
#define KDA_RMS_F(XB, RES, L, M)                                                               \
  forward_kernel<XB, RES, L, M><<<dim3((unsigned)((Q * L + threads<L>() - 1) / threads<L>())), \
                                  threads<L>(), 0, s>>>(f, Q)
#define KDA_RMS_CALL(L, M)                                      \
  if (f.x_bf16 && !f.res) KDA_RMS_F(true, 0, L, M);             \
  else if (f.x_bf16 && f.res_bf16) KDA_RMS_F(true, 1, L, M);    \
  else if (f.x_bf16) KDA_RMS_F(true, 2, L, M);                  \
  else if (!f.res) KDA_RMS_F(false, 0, L, M);                   \
  else KDA_RMS_F(false, 2, L, M)
  KDA_LN_DISPATCH(KDA_RMS_CALL);
#undef KDA_RMS_CALL
#undef KDA_RMS_F
  return hipGetLastError();
}

size_t backward_workspace_bytes(int64_t rows, int64_t groups, int d) {
  if (rows == 0) return 0;
  return (size_t)backward_owners(rows, groups, lanes_of(d), runs_of(d)) * d * sizeof(float);
}

hipError_t launch_backward(const Backward& f, void* ws, hipStream_t s) {
  float* part = f.dw ? static_cast<float*>(ws) : nullptr;
  const int d = f.d;
  int64_t Q = 0;
  if (f.rows > 0) {
    Q = backward_owners(f.rows, f.groups, lanes_of(d), runs_of(d));
#define KDA_RMS_B(YB, XB, L, M)                                                                 \
  backward_kernel<YB, XB, L, M><<<dim3((unsigned)((Q * L + threads<L>() - 1) / threads<L>())), \
                                  threads<L>(), 0, s>>>(f, part, Q)
#define KDA_RMS_CALL(L, M)                                \
  if (f.dy_bf16 && f.x_bf16) KDA_RMS_B(true, true, L, M); \
  else if (f.dy_bf16) KDA_RMS_B(true, false, L, M);       \
  else if (f.x_bf16) KDA_RMS_B(false, true, L, M);        \
  else KDA_RMS_B(false, false, L, M)
    KDA_LN_DISPATCH(KDA_RMS_CALL);
#undef KDA_RMS_CALL
#undef KDA_RMS_B
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (f.dw) {  // with no rows the sums are zeros
    const int64_t have = Q < f.rows ? Q : f.rows;
    partials_kernel<<<dim3((unsigned)((d + 63) / 64), (unsigned)f.groups), 1024, 0, s>>>(
        part, have, f.groups, d, f.dw);
  }
  return hipGetLastError();
}

}  // namespace rms
}  // namespace kda
