// kda_layernorm and kda_layernorm_backward: layer norm over the rows of [rows, d].
//
//   forward   y  = xh w + b,  xh = (x - mu) r,  r = 1 / sqrt(var + eps)
//   backward  dx = r (t - mean(t) - xh mean(t xh)),  t = dy w
//             dw = sum_rows dy xh,  db = sum_rows dy
//
// HBM-bound: x (and dy) are read once, y (dx) is written once, the row stays
// in registers between.  Measured, bf16: forward of 393216 rows of 128 (96 weight
// rows) 39 us, 5.1 TB/s; backward 67 us, 4.5 TB/s; backward of 2048 x 5003 30 us,
// where a row's chain (loads, two sums over 512 lanes) leaves the card idle.
//
// L lanes own a row: a part of a wave up to d = 256, a wave up to 1,024, a workgroup
// beyond that; lane l holds the M runs of eight columns (m L + l) 8 .. + 7.  The
// lanes of a row then walk down rows of the SAME weight row (row % groups), so that w,
// b and the gradients' sums stay in registers: row q, q + Q, q + 2Q, ... with Q a
// multiple of groups.  Neighbouring lanes own neighbouring rows, so a wave's access is
// contiguous whatever L is.  The next row is loaded before this one is worked on.
//
// The statistics are two sums over the registers: the mean, then the differences
// from it and their squares.  The mean of fp32 sums is a few ulps off, which beside a
// spread far below the mean is not small (a row of 1000.0, d = 1000: every value 6e-5
// off, times 1 / sqrt(eps)); the sum of the differences gives that error, which comes
// off the values and off the mean square.  The backward forms the statistics again
// from x, which it reads anyway, rather than read stored ones.
//
// dw and db: each row owner adds its rows into registers in order and writes
// one partial row; a second kernel adds the partials of a weight row in a fixed
// order.  No atomics: the same call gives the same bits.
//
// Rows need only their element's alignment (d may be odd): the eight-value
// accesses are declared as such, which the hardware takes in one instruction.
#include "kda_device.hpp"
#include "linattn.hpp"

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

// x (columns past d hold 0) becomes x less its computed mean, with x rstd + shift the
// normalised value (past d something finite); rstd = 1/sqrt(var + eps).  With T = 1 the
// sums of t = dy w and of t (x - mean) come along with the two sums (t is formed where it
// is needed: the registers do not hold it too).
template <int L, int M, int T>
__device__ __forceinline__ void statistics(f32x8 (&x)[M], const f32x8 (&dy)[T ? M : 1],
                                           const f32x8 (&w)[T ? M : 1], const int (&left)[M],
                                           float inv_d, float eps, float* s_part, int& turn,
                                           float& rstd, float& shift, float& st, float& stx) {
  float s[1 + T] = {};
#pragma unroll
  for (int m = 0; m < M; ++m) {
    s[0] += sum8(x[m]);
    if constexpr (T) s[1] += sum8(dy[m] * w[m]);
  }
  row_sum<L, 1 + T>(s, s_part, turn);
  const float mu = s[0] * inv_d;
  float v[2 + T] = {};
#pragma unroll
  for (int m = 0; m < M; ++m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[m][e] = e < left[m] ? x[m][e] - mu : 0.f;
    v[0] += sum8(x[m] * x[m]);
    v[1] += sum8(x[m]);
    if constexpr (T) v[2] += sum8(dy[m] * w[m] * x[m]);
  }
  row_sum<L, 2 + T>(v, s_part, turn);
  const float off = v[1] * inv_d;  // the mean's own error
  const float var = fmaf(-off, off, v[0] * inv_d);  // (an overflow stays one: no inf - inf)
  rstd = 1.0f / sqrtf((var < 0.f ? 0.f : var) + eps);  // (a NaN stays one)
  shift = -off * rstd;
  if constexpr (T) {
    st = s[1];
    stx = v[2] - off * st;
  }
}

// Row owner q of Q walks rows q, q + Q, ... (Q a multiple of groups).  y may be x: a row
// is read before it is written and by its owner only, so neither is __restrict__ (nor are
// dy, x and dx below).
template <bool XB, bool YB, int L, int M>
__global__ void __launch_bounds__(threads<L>()) forward_kernel(
    const void* x, const float* __restrict__ w, const float* __restrict__ b, int64_t groups,
    void* y, int64_t rows, int d, float eps, int64_t Q) {
  constexpr int RPB = threads<L>() / L;
  __shared__ float s_part[L > 64 ? 2 * kSums * (L / 64) : 1];
  const int l = threadIdx.x % L;
  const int64_t q = (int64_t)blockIdx.x * RPB + threadIdx.x / L;
  if (q >= Q || q >= rows) return;  // whole rows of lanes leave together (L > 64: the workgroup)
  int left[M];  // columns of each run that exist
  f32x8 ww[M], bb[M];
  const int64_t wrow = (q % groups) * d;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int c = (m * L + l) * 8;
    left[m] = d - c < 0 ? 0 : (d - c < 8 ? d - c : 8);
    Eight<false> t;
    ww[m] = f32x8(1.f);
    bb[m] = f32x8(0.f);
    if (w) { t.load(w, wrow + c, left[m]); ww[m] = t.get(); }
    if (b) { t.load(b, wrow + c, left[m]); bb[m] = t.get(); }
  }
  const float inv_d = 1.0f / d;
  int turn = 0;
  Eight<XB> raw[M];
#pragma unroll
  for (int m = 0; m < M; ++m) raw[m].load(x, q * d + (m * L + l) * 8, left[m]);
  for (int64_t r = q; r < rows; r += Q) {
    f32x8 v[M];
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = raw[m].get();
    if (r + Q < rows)
#pragma unroll
      for (int m = 0; m < M; ++m) raw[m].load(x, (r + Q) * d + (m * L + l) * 8, left[m]);
    float rstd, shift, none;
    const f32x8 no_t[1] = {};
    statistics<L, M, 0>(v, no_t, no_t, left, inv_d, eps, s_part, turn, rstd, shift, none, none);
#pragma unroll
    for (int m = 0; m < M; ++m)
      Eight<YB>::store(y, r * d + (m * L + l) * 8, left[m],
                       (v[m] * rstd + shift) * ww[m] + bb[m]);
  }
}

template <bool YB, bool XB, int L, int M>
__global__ void __launch_bounds__(threads<L>()) backward_kernel(
    const void* dy, const void* x, const float* __restrict__ w, int64_t groups, void* dx,
    float* __restrict__ part, int64_t rows, int d, float eps, int64_t Q) {
  constexpr int RPB = threads<L>() / L;
  __shared__ float s_part[L > 64 ? 2 * kSums * (L / 64) : 1];
  const int l = threadIdx.x % L;
  const int64_t q = (int64_t)blockIdx.x * RPB + threadIdx.x / L;
  if (q >= Q || q >= rows) return;
  int left[M];
  f32x8 ww[M], dw[M], db[M];
  const int64_t wrow = (q % groups) * d;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int c = (m * L + l) * 8;
    left[m] = d - c < 0 ? 0 : (d - c < 8 ? d - c : 8);
    Eight<false> t;
    ww[m] = f32x8(1.f);
    if (w) { t.load(w, wrow + c, left[m]); ww[m] = t.get(); }
    dw[m] = db[m] = f32x8(0.f);
  }
  const float inv_d = 1.0f / d;
  int turn = 0;
  // The next row on its way while this one is worked on; 1,024 lanes have 128
  // registers each, enough for one row only (512 x 12288 fp32: with the next one,
  // spilled, 51 us, without 28).
  constexpr bool AHEAD = L < 1024;
  Eight<XB> rx[M];
  Eight<YB> ry[M];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      rx[m].load(x, r * d + (m * L + l) * 8, left[m]);
      ry[m].load(dy, r * d + (m * L + l) * 8, left[m]);
    }
  };
  if (AHEAD) load(q);
  for (int64_t r = q; r < rows; r += Q) {
    if (!AHEAD) load(r);
    f32x8 v[M], g[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      v[m] = rx[m].get();
      g[m] = ry[m].get();
    }
    if (AHEAD && r + Q < rows) load(r + Q);
    float rstd, shift, m0, m1;  // (past d dy is 0, and so is t)
    statistics<L, M, 1>(v, g, ww, left, inv_d, eps, s_part, turn, rstd, shift, m0, m1);
    m0 *= inv_d;
    m1 *= inv_d * rstd;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      v[m] = v[m] * rstd + shift;  // xh
      db[m] += g[m];
      dw[m] += g[m] * v[m];
      Eight<XB>::store(dx, r * d + (m * L + l) * 8, left[m], rstd * (g[m] * ww[m] - m0 - v[m] * m1));
    }
  }
  if (part) {
    float* pw = part + q * 2 * d;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      Eight<false>::store(pw, (m * L + l) * 8, left[m], dw[m]);
      Eight<false>::store(pw, d + (m * L + l) * 8, left[m], db[m]);
    }
  }
}

// dw, db [groups, d] from the partial rows [Q][2][d]: owner q belongs to weight
// row q % groups.  64 columns a workgroup, 16 owners in turn a column, added in order.
__global__ void __launch_bounds__(1024) partials_kernel(const float* __restrict__ part,
                                                        int64_t owners, int64_t groups, int d,
                                                        float* __restrict__ dw,
                                                        float* __restrict__ db) {
  __shared__ float s[16][64];
  const int cl = threadIdx.x & 63, k = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + cl;  // column of [2][d]
  const int64_t grp = blockIdx.y;
  float acc = 0.f;
  if (c < 2 * (int64_t)d)
    for (int64_t q = grp + groups * k; q < owners; q += groups * 16 * 8) {
      float x[8];  // eight loads on their way
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t at = q + groups * 16 * j;
        x[j] = at < owners ? part[at * 2 * d + c] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) acc += x[j];
    }
  s[k][cl] = acc;
  __syncthreads();
  if (k == 0 && c < 2 * (int64_t)d) {
    for (int j = 1; j < 16; ++j) acc += s[j][cl];
    float* out = c < d ? dw : db;
    if (out) out[grp * d + (c < d ? c : c - d)] = acc;
  }
}

// Row owners: enough lanes for the card, at most one a row, a multiple of groups.
int64_t owners(int64_t rows, int64_t groups, int64_t most) {
  const int64_t q = most < 1 ? 1 : most > rows ? rows : most;
  return (q + groups - 1) / groups * groups;
}
// lanes for the card: us at 2,048 / 4,096 a CU, bf16: 393216 x 128 37 / 36, 65536 x 1024
// 46 / 43, 16384 x 4096 46 / 43; of 512 lanes a row, 8192 x 5000 44 / 41, 2048 x 5003
// 14.1 / 14.7; of 1,024, 4096 x 12288 52 / 55
int64_t forward_owners(int64_t rows, int64_t groups, int L) {
  return owners(rows, groups, 256 * (L <= 512 ? 4096 : 2048) / L);
}
// Every owner of the backward also writes 2 d sums, which are read again: fewer
// lanes (1,024 a CU and run of eight columns; us with half of that / that / twice, bf16:
// 393216 x 128 74 / 65 / 72, 65536 x 1024 88 / 88 / 107, 16384 x 4096 95 / 86 / 99), and
// at least eight rows each (1024 x 4096: 18.5, with two rows each 20.5) unless that
// leaves CUs without a workgroup (512 x 12288: 128 owners 24.4, 256 22.7).
int64_t backward_owners(int64_t rows, int64_t groups, int L, int M) {
  const int64_t one_each = 256 * (L < 256 ? 256 / L : 1);  // a workgroup a CU
  int64_t q = 256 * 1024 / (L * M);
  if (q > rows / 8) q = rows / 8;
  return owners(rows, groups, q < one_each ? one_each : q);
}

int lanes_of(int d) {
  return d <= 64 ? 8 : d <= 128 ? 16 : d <= 256 ? 32 : d <= 1024 ? 64 : d <= 4096 ? 256
         : d <= 8192 ? 512 : 1024;
}
int runs_of(int d) { return (d + lanes_of(d) * 8 - 1) / (lanes_of(d) * 8); }

}  // namespace

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

hipError_t launch_forward(const void* x, bool x_bf16, const float* w, const float* b,
                          int64_t groups, void* y, bool y_bf16, int64_t rows, int d, float eps,
                          hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int64_t Q = forward_owners(rows, groups, lanes_of(d));
#define KDA_LN_F(XB, YB, L, M)                                                                 \
  forward_kernel<XB, YB, L, M><<<dim3((unsigned)((Q * L + threads<L>() - 1) / threads<L>())), \
                                 threads<L>(), 0, s>>>(x, w, b, groups, y, rows, d, eps, Q)
#define KDA_LN_CALL(L, M)                            \
  if (x_bf16 && y_bf16) KDA_LN_F(true, true, L, M);  \
  else if (x_bf16) KDA_LN_F(true, false, L, M);      \
  else if (y_bf16) KDA_LN_F(false, true, L, M);      \
  else KDA_LN_F(false, false, L, M)
  KDA_LN_DISPATCH(KDA_LN_CALL);
#undef KDA_LN_CALL
#undef KDA_LN_F
  return hipGetLastError();
}

size_t backward_workspace_bytes(int64_t rows, int64_t groups, int d) {
  if (rows == 0) return 0;
  return (size_t)backward_owners(rows, groups, lanes_of(d), runs_of(d)) * 2 * d * sizeof(float);
}

hipError_t launch_backward(const void* dy, bool dy_bf16, const void* x, bool x_bf16,
                           const float* w, int64_t groups, void* dx, float* dw, float* db,
                           int64_t rows, int d, float eps, void* ws, hipStream_t s) {
  const bool sums = dw || db;
  float* part = sums ? static_cast<float*>(ws) : nullptr;
  int64_t Q = 0;
  if (rows > 0) {
    Q = backward_owners(rows, groups, lanes_of(d), runs_of(d));
#define KDA_LN_B(YB, XB, L, M)                                                                  \
  backward_kernel<YB, XB, L, M><<<dim3((unsigned)((Q * L + threads<L>() - 1) / threads<L>())), \
                                  threads<L>(), 0, s>>>(dy, x, w, groups, dx, part, rows, d, eps, Q)
#define KDA_LN_CALL(L, M)                             \
  if (dy_bf16 && x_bf16) KDA_LN_B(true, true, L, M);  \
  else if (dy_bf16) KDA_LN_B(true, false, L, M);      \
  else if (x_bf16) KDA_LN_B(false, true, L, M);       \
  else KDA_LN_B(false, false, L, M)
    KDA_LN_DISPATCH(KDA_LN_CALL);
#undef KDA_LN_CALL
#undef KDA_LN_B
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (sums) {  // with no rows the sums are zeros
    const int64_t have = Q < rows ? Q : rows;
    partials_kernel<<<dim3((unsigned)((2 * (int64_t)d + 63) / 64), (unsigned)groups), 1024, 0, s>>>(
        part, have, groups, d, dw, db);
  }
  return hipGetLastError();
}

}  // namespace norm
}  // namespace kda
