// What layer norm and RMS norm share: rows held in the registers of L lanes as runs of eight
// columns, sums over a row's lanes, and which lanes own which rows.
#pragma once

#include "kda_device.hpp"

namespace kda {
namespace norm {
namespace {

typedef u16x8 u16x8_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// Eight values at p + i of which the first n (<= 8) exist; the others are 0.
template <bool BF16>
struct Eight;
template <>
struct Eight<true> {
  u16x8 r;
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    const uint16_t* s = static_cast<const uint16_t*>(p) + i;
    if (n >= 8) {
      r = *reinterpret_cast<const u16x8_a2*>(s);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = e < n ? s[e] : uint16_t(0);
    }
  }
  __device__ __forceinline__ f32x8 get() const {
    f32x8 x;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = bf16_bits_to_f32(r[e]);
    return x;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, int n, f32x8 x) {
    uint16_t* d = static_cast<uint16_t*>(p) + i;
    u16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f32_to_bf16_bits(x[e]);
    if (n >= 8) {
      *reinterpret_cast<u16x8_a2*>(d) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) d[e] = v[e];
    }
  }
};
template <>
struct Eight<false> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    const float* s = static_cast<const float*>(p) + i;
    if (n >= 8) {
      a = *reinterpret_cast<const f32x4_a4*>(s);
      b = *reinterpret_cast<const f32x4_a4*>(s + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = e < n ? s[e] : 0.f;
        b[e] = e + 4 < n ? s[e + 4] : 0.f;
      }
    }
  }
  __device__ __forceinline__ f32x8 get() const {
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, int n, f32x8 x) {
    float* d = static_cast<float*>(p) + i;
    if (n >= 8) {
      *reinterpret_cast<f32x4_a4*>(d) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4_a4*>(d + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) d[e] = x[e];
    }
  }
};

__device__ __forceinline__ float sum8(f32x8 x) {
  return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}

template <int CTRL>
__device__ __forceinline__ float moved(float x) {  // x of the lane that CTRL names
  return __uint_as_float(
      __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
// Sum over aligned groups of L (4 .. 64) lanes, in all of them.  Moves between
// registers: an LDS permute takes some 60 clocks, and a row waits for its sums.
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
  x += moved<0xb1>(x);                                  // lane ^ 1
  x += moved<0x4e>(x);                                  // lane ^ 2
  if constexpr (L >= 8) x += moved<0x141>(x);           // 7 - lane of eight: the other four
  if constexpr (L >= 16) x += moved<0x140>(x);          // 15 - lane of sixteen: the other eight
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

constexpr int kSums = 3;  // most values of one row_sum

// Sums of NS values over the L lanes of a row; every lane gets them.  Rows of
// a whole workgroup (L = its size) go through LDS, double-buffered by `turn`
// so that one barrier a sum is enough.
template <int L, int NS>
__device__ __forceinline__ void row_sum(float (&x)[NS], float* s_part, int& turn) {
  static_assert(NS <= kSums, "size of s_part");
#pragma unroll
  for (int i = 0; i < NS; ++i) x[i] = lanes_sum<(L < 64 ? L : 64)>(x[i]);
  if constexpr (L > 64) {
    constexpr int W = L / 64;
    float* p = s_part + turn * (kSums * W);
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NS; ++i) p[i * W + (threadIdx.x >> 6)] = x[i];
    barrier_lds();
    // each lane takes one wave's part: a read and a few moves.  (W reads a lane: 512 x
    // 12288 fp32 backward 52 us against 28, 16 waves' registers run out; 8192 x 5000
    // bf16, 8 waves, 92 against 94.)
#pragma unroll
    for (int i = 0; i < NS; ++i) x[i] = lanes_sum<W>(p[i * W + (threadIdx.x & (W - 1))]);
  }
}

template <int L>
constexpr int threads() { return L > 256 ? L : 256; }

// Row owners: enough lanes for the card, at most one a row, a multiple of groups.
int64_t owners(int64_t rows, int64_t groups, int64_t most) {
  const int64_t q = most < 1 ? 1 : most > rows ? rows : most;
  return (q + groups - 1) / groups * groups;
}
int lanes_of(int d) {
  return d <= 64 ? 8 : d <= 128 ? 16 : d <= 256 ? 32 : d <= 1024 ? 64 : d <= 4096 ? 256
         : d <= 8192 ? 512 : 1024;
}
int runs_of(int d) { return (d + lanes_of(d) * 8 - 1) / (lanes_of(d) * 8); }

}  // namespace
}  // namespace norm
}  // namespace kda

#define KDA_LN_DISPATCH(CALL)                                 \
  do {                                                        \
    if (d <= 64) { CALL(8, 1); }                              \
    else if (d <= 128) { CALL(16, 1); }                       \
    else if (d <= 256) { CALL(32, 1); }                       \
    else if (d <= 512) { CALL(64, 1); }                       \
    else if (d <= 1024) { CALL(64, 2); }                      \
    else if (d <= 2048) { CALL(256, 1); }                     \
    else if (d <= 4096) { CALL(256, 2); }                     \
    else if (d <= 8192) { CALL(512, 2); }                     \
    else { CALL(1024, 2); }                                   \
  } while (0)
