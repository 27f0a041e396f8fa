// What the forward and the backward of the gated linear recurrence share on the device:
// the gate, the packed batch's borders, and the carry between tiles.
#pragma once

#include "gatedrec.hpp"
#include "kda_device.hpp"

namespace kda {
namespace gatedrec {

// ------------------------------------------------------------------ values
// V neighbouring channels of one token as they lie in memory: `rows` is a resource over a
// tensor from some row on, `row` the bytes to the token (uniform over the wave), `at` those
// to the lane's channels.  (A 64-bit address a lane and token takes two registers and three
// instructions, one of them in the vector unit.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const void* p, int64_t bytes) {
  return buffer_over(static_cast<const char*>(p) + bytes, 0xffffffffu);
}
template <bool BF16, int V>
struct Vals {
  static constexpr int BYTES = V * (BF16 ? 2 : 4), N = BYTES < 4 ? 1 : BYTES / 4;
  static_assert(BYTES == 2 || BYTES == 4 || BYTES == 8 || BYTES == 16, "one load");
  typedef uint32_t Wide __attribute__((ext_vector_type(N)));
  uint32_t w[N];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rows, uint32_t at, uint32_t row) {
    Wide x;
    if constexpr (BYTES == 2) x = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rows, at, row, 0);
    else if constexpr (BYTES == 4) x = __builtin_amdgcn_raw_buffer_load_b32(rows, at, row, 0);
    else if constexpr (BYTES == 8)
      x = __builtin_bit_cast(Wide, __builtin_amdgcn_raw_buffer_load_b64(rows, at, row, 0));
    else x = __builtin_bit_cast(Wide, __builtin_amdgcn_raw_buffer_load_b128(rows, at, row, 0));
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = x[n];
  }
  __device__ __forceinline__ float get(int v) const {
    if constexpr (BF16) return __uint_as_float(v & 1 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
    return __uint_as_float(w[BF16 ? 0 : v]);
  }
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t rows, uint32_t at,
                                               uint32_t row, const float (&x)[V]) {
    if constexpr (BYTES == 2) {
      __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16_bits(x[0]), rows, at, row, 0);
    } else {
      Wide y;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if constexpr (BF16) {
          typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
          y[n] = __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(x[2 * n]),
                                                     static_cast<__bf16>(x[2 * n + 1])});
        } else {
          y[n] = __float_as_uint(x[n]);
        }
      }
      if constexpr (BYTES == 4) __builtin_amdgcn_raw_buffer_store_b32(y[0], rows, at, row, 0);
      else if constexpr (BYTES == 8) __builtin_amdgcn_raw_buffer_store_b64(y, rows, at, row, 0);
      else __builtin_amdgcn_raw_buffer_store_b128(y, rows, at, row, 0);
    }
  }
};
template <int V>
__device__ __forceinline__ void load_state(const void* p, int64_t at, float (&x)[V], bool bf16) {
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = load1(p, at + v, bf16);
}
// states (and gradients of them) need only their element's alignment
template <int V>
__device__ __forceinline__ void store_state(void* p, int64_t at, const float (&x)[V], bool bf16) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (bf16) static_cast<uint16_t*>(p)[at + v] = f32_to_bf16_bits(x[v]);
    else static_cast<float*>(p)[at + v] = x[v];
  }
}

// Whether every row and output may be taken V values at a time.
struct Out {
  const void* p;
  bool bf16;
};
inline bool in_pieces_of(int V, const Inputs& in, int C, const Out* outs, int count) {
  const size_t es = in.bf16 ? 2 : 4;
  if (C % V) return false;
  for (const Rows* r : {&in.x, &in.r, &in.i})
    if (reinterpret_cast<uintptr_t>(r->p) % (V * es) || r->stride % V) return false;
  for (int k = 0; k < count; ++k)
    if (reinterpret_cast<uintptr_t>(outs[k].p) % (V * (outs[k].bf16 ? 2 : 4))) return false;
  return true;
}
// Values a lane takes at once in the scan and its gradients: two of bf16 (4 bytes a lane)
// where that is aligned, else one.  4,096 x 12,288, scan and training step: 110 and 323 us,
// one at a time 121 and 404; 8,192 x 4,096 from log-decays 57 and 74.  (fp32 has its 4 bytes
// with one, and two would take the registers of two workgroups a CU.)
inline int width(const Inputs& in, int C, const Out* outs, int count) {
  return in.bf16 && in_pieces_of(2, in, C, outs, count) ? 2 : 1;
}

// -------------------------------------------------------------------- gate
// Log-decays are in log2 units throughout (g2 = g log2(e), a = 2^g2): the scale goes into
// constants that are multiplied anyway.  The polynomials are minimax fits of the relative
// error over the stated ranges.
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// log2(1 + e) / e for 0 <= e <= 1, with the product 2.5 u of itself (u = 2^-24; 0.5 before its
// roundings).  A hardware log with its correction for small e (gate_math.hpp) costs half as much
// again.
__device__ __forceinline__ float log2_1p_over(float e) {
  float p = 0.007651003077626228f;
  p = fmaf(p, e, -0.04299952834844589f);
  p = fmaf(p, e, 0.11361227184534073f);
  p = fmaf(p, e, -0.19781996309757233f);
  p = fmaf(p, e, 0.276011198759079f);
  p = fmaf(p, e, -0.35851892828941345f);
  p = fmaf(p, e, 0.48071038722991943f);
  p = fmaf(p, e, -0.7213414311408997f);
  return fmaf(p, e, 1.4426950216293335f);
}
// 1 - 2^y for y <= 0, e = 2^y: the difference loses the digits of a small y, so there it is a
// polynomial (0.3 u).  Its sign is clear, for zeros of either sign too (-y p of y = +0 is -0, which
// decay_code would take for a cut): that is what the sum with +0 is for.
__device__ __forceinline__ float one_minus_exp2(float y, float e) {
  float p = 0.0011528132017701864f;
  p = fmaf(p, y, 0.009539824910461903f);
  p = fmaf(p, y, 0.055490005761384964f);
  p = fmaf(p, y, 0.24022559821605682f);
  p = fmaf(p, y, 0.6931471824645996f);
  return y > -0.5f ? fmaf(-y, p, 0.0f) : 1.0f - e;  // NaN stays NaN
}
// 1 - 4^g2 for g2 <= 0, a = 2^g2: the same up to where a^2, two digits of a off by one, leaves
// 4 u of the difference.
__device__ __forceinline__ float one_minus_square(float g2, float a) {
  float p = 0.0371021144092083f;
  p = fmaf(p, g2, 0.15275147557258606f);
  p = fmaf(p, g2, 0.4439404606819153f);
  p = fmaf(p, g2, 0.9609037637710571f);
  p = fmaf(p, g2, 1.3862943649291992f);
  return g2 > -0.25f ? -g2 * p : fmaf(-a, a, 1.0f);
}
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp2_fast(x * -kLog2e));
}

// The gate of a lane's channels: kda_gate's formula with its sums in log2 units.
template <int V, bool GATE>
struct Params {
  float neg_a[GATE ? V : 1], bias2[GATE ? V : 1];
  __device__ __forceinline__ void load(const Inputs& in, int c) {
    if constexpr (GATE) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        neg_a[v] = -exp2_fast(in.A_log[c + v] * kLog2e);
        bias2[v] = in.dt_bias ? in.dt_bias[c + v] * kLog2e : 0.0f;
      }
    }
  }
  // softplus in log2 units is max(z2, 0) + log2(1 + 2^-|z2|), z2 = z log2(e)
  __device__ __forceinline__ float log2_decay(float r, int v) const {
    if constexpr (GATE) {
      const float z2 = fmaf(r, kLog2e, bias2[v]);
      const float e = exp2_fast(-fabsf(z2));
      return neg_a[v] * fmaf(e, log2_1p_over(e), fmaxf(z2, 0.0f));  // (a NaN is in e)
    }
    return r > 0.0f ? 0.0f : r * kLog2e;  // NaN stays NaN
  }
};

// ------------------------------------------------------------ decay factors
// A stretch's decay 2^s, s the sum of its log2-decays, as one number `code`: beside 1 it is
// 1 - d with d = 1 - 2^s kept (code = d, sign clear; +0 where the stretch keeps everything), for
// 2^s itself would be rounded to 6e-8, which over the stretches of a slow channel adds up to
// 6e-8 / d of the state.  Further away it is 2^s (code = -2^s, sign set), and where that is 0,
// nothing is left of what comes before, whatever it was.
constexpr uint32_t kCut = 0x80000000u;
__device__ __forceinline__ float decay_code(float s) {
  const float e = exp2_fast(s);
  const float d = one_minus_exp2(s, e);
  return d < 0.5f ? d : -e;  // NaN stays NaN
}
__device__ __forceinline__ float decayed_onto(float code, float h, float add) {
  const float t = fmaf(-code, h, add);
  return __float_as_uint(code) == kCut ? add : __float_as_int(code) < 0 ? t : t + h;
}

// ----------------------------------------------------------- packed batch
struct Seqs {
  const int32_t* cu;
  int N, T, len;  // len: tokens of every sequence when cu is null
  __device__ __forceinline__ int clamp(int t) const { return t < 0 ? 0 : t > T ? T : t; }
  // (read through a vector load wherever the compiler sees a store before it: the value is
  // the same for the whole wave, and what follows from it belongs in scalar registers)
  __device__ __forceinline__ int at(int n) const { return __builtin_amdgcn_readfirstlane(cu[n]); }
  __device__ __forceinline__ int start(int n) const { return cu ? clamp(at(n)) : n * len; }
  __device__ __forceinline__ int live() const { return cu ? clamp(at(N)) : T; }
  // the last sequence that begins at or before t
  __device__ __forceinline__ int find(int t) const {
    if (!cu) return len > 0 ? t / len : 0;
    int lo = 0, hi = N - 1;
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (at(mid) <= t) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};
// id / blocks and the rest, by a reciprocal that the host has formed: the division of two
// numbers in scalar registers goes through the vector unit.
struct Split {
  uint32_t n = 1, inverse = 0;  // inverse: floor(2^32 / n), 0 for 1
  Split() = default;
  explicit Split(uint32_t d) : n(d), inverse(d > 1 ? (uint32_t)(((uint64_t)1 << 32) / d) : 0) {}
  __device__ __forceinline__ int operator()(int id, int& rest) const {
    uint32_t q = inverse ? __umulhi((uint32_t)id, inverse) : (uint32_t)id;  // 0 to 1 too small
    uint32_t r = (uint32_t)id - q * n;
    if (r >= n) {
      ++q;
      r -= n;
    }
    rest = (int)r;
    return (int)q;
  }
};

// The borders among the `count` (at most 32) tokens from t0: bit j of `first` (`last`) says
// that token t0 + j is the first (last) of its sequence.
// Without one (nearly always) a wave takes straight code that asks for none.
struct Borders {
  uint32_t first = 0, last = 0;
  __device__ __forceinline__ void find(const Seqs& q, int t0, int count) {
    if (count <= 0) return;
    int n = q.find(t0);
    if (q.start(n) == t0) first = 1u;
    while (n < q.N) {
      const int e = q.start(n + 1);
      int next = n + 1;
      if (e > t0) {
        if (e - t0 > count) break;
        last |= 1u << (e - t0 - 1);
        if (e - t0 == count) break;
        first |= 1u << (e - t0);
        next = q.find(e);  // past sequences without tokens
      }
      n = next > n ? next : n + 1;
    }
  }
};

// ------------------------------------------------------------------ carries
// The tiles of a channel hand their state on.  Tile k (in the order of the walk) publishes
// its own decay and contribution (code, add), looks for the nearest tile before it whose
// state is known, takes what lies between (up to kReach tiles) and publishes its own state.
// What lies between is folded one by one, forwards: wherever it begins, the bits are the same.
//
// Tiles are given out by a ticket, so whoever is waited for is running or done.  A word that
// is not there yet is all ones; what is published never is, so a word is its own proof
// of being there and nothing hangs on the order of accesses; they bypass what an XCD has to
// itself, for neighbouring tiles run on different ones.  `mark` only says where to look, one word a tile and block of
// channels, so that 64 tiles are looked at in one load.
//
// Should the words be spoilt (the workspace used by something else meanwhile), a wait
// gives up after kSpins and the tile goes on with NaN: every wait ends.  (A tile that waits
// holds its place, as does everybody before it: kSpins is about a second.)
constexpr uint32_t kEmpty = 0xffffffffu;
constexpr int kSpins = 1 << 20;
constexpr int kByOne = 4;  // so many tiles one wave looks at in one go
// (131,072 x 512 bf16, 1,024 tiles a channel: looked back over by one wave, four tiles a way to
// memory, 266 us; marks first and every wave bringing four tiles, 150 us.  Up to four tiles
// between, which is nearly always, are one wave's in one way.)

struct Chain {
  uint32_t* ticket;
  uint32_t *state, *code, *add;  // [tiles][C]
  uint32_t* mark;                // [blocks][tiles]: kEmpty, 1 (code and add), 2 (state)
};
// (blocks: at most C / 64 rounded up)
inline size_t chain_bytes(int64_t tiles, int64_t C) {
  return (256 + (size_t)tiles * C * 12 + (size_t)tiles * ((C + 63) / 64) * 4 + 255) / 256 * 256;
}
// makes every word empty, the ticket too
hipError_t launch_fill(void* ws, size_t bytes, hipStream_t s);
inline Chain chain_at(void* ws, int64_t tiles, int64_t C) {
  Chain c;
  c.ticket = static_cast<uint32_t*>(ws);
  c.state = c.ticket + 64;
  c.code = c.state + tiles * C;
  c.add = c.code + tiles * C;
  c.mark = c.add + tiles * C;
  return c;
}
__device__ __forceinline__ uint32_t peek(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void poke(uint32_t* p, uint32_t x) {
  __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// V words of a lane's channels: `rows` over some tile's row of an array on, `row` the bytes to
// the tile's, `at` those to the channels.  Coherent like an atomic access at agent scope.
constexpr int kAgent = 16;  // buffer access cache policy: sc1
template <int V>
__device__ __forceinline__ void publish(__amdgpu_buffer_rsrc_t rows, uint32_t at, const float (&x)[V]) {
  uint32_t w[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    w[v] = __float_as_uint(x[v]);
    if (w[v] == kEmpty) w[v] = 0x7fc00000u;
  }
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  if constexpr (V == 1)
    __builtin_amdgcn_raw_buffer_store_b32(w[0], rows, at, 0, kAgent);
  else
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{w[0], w[V - 1]}, rows, at, 0, kAgent);
}
template <int V>
struct Words {
  uint32_t w[V];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rows, uint32_t at, uint32_t row) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    if constexpr (V == 1) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(rows, at, row, kAgent);
    } else {
      const u32x2 x =
          __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rows, at, row, kAgent));
      w[0] = x[0];
      w[V - 1] = x[1];
    }
  }
  __device__ __forceinline__ bool there() const { return w[0] != kEmpty && w[V - 1] != kEmpty; }
  __device__ __forceinline__ float get(int v) const { return __uint_as_float(w[v]); }
};

// The nearest of the REACH tiles before k whose state is marked, with everything between
// marked too: how many tiles lie between it and k; -1 where there is none yet.  One wave; 0 < k.
template <int REACH>
__device__ __forceinline__ int marked_state(const uint32_t* mark, int k) {
  static_assert(REACH <= 64, "a lane a tile");
  const int lane = threadIdx.x & 63;
  const uint32_t m = lane < REACH && k - 1 - lane >= 0 ? peek(mark + (k - 1 - lane)) : 0u;
  const uint64_t whole = __ballot(m == 2u), part = __ballot(m == 1u);
  if (!whole) return -1;
  const int n = __builtin_ctzll(whole);
  return n == 0 || (~part & ((1ull << n) - 1)) == 0 ? n : -1;
}

// The state behind tile k - 1 where one of the N tiles before k has it and those after that one
// are there: everything is asked for at once, one way to memory and back.
template <int N, int V>
__device__ __forceinline__ bool near_state(const Chain& ch, int64_t C, int k, uint32_t at, bool on,
                                           float (&h)[V]) {
  Words<V> state[N], code[N], add[N];
  const int first = k > N ? k - N : 0;
  const __amdgpu_buffer_rsrc_t ps = rows_from(ch.state, first * C * 4),
                               pc = rows_from(ch.code, first * C * 4),
                               pa = rows_from(ch.add, first * C * 4);
#pragma unroll
  for (int j = 0; j < N; ++j) {  // tile k - 1 - j
    const uint32_t row = (uint32_t)(k - 1 - j > first ? k - 1 - j - first : 0) * (uint32_t)C * 4u;
    state[j].load(ps, at, row);
    if (j + 1 < N) {
      code[j].load(pc, at, row);
      add[j].load(pa, at, row);
    }
  }
  int q = -1;
  bool open = true;
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (open && k - 1 - j >= 0) {
      if (__all(state[j].there() || !on)) {
        q = j;
        open = false;
      } else if (j + 1 < N) {
        open = __all((code[j].there() && add[j].there()) || !on);
      }
    }
  if (q < 0) return false;
#pragma unroll
  for (int j = N - 1; j >= 0; --j) {
    if (j == q)
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = state[j].get(v);
    if (j + 1 < N && j < q)
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = decayed_onto(code[j].get(v), h[v], add[j].get(v));
  }
  return true;
}

// N tiles' words from tile `first` on (those before `end`) and, if asked for, the state before
// `first`, all on their way at once; words that are marked may still be on theirs.  (A load
// that finds none is repeated: the fence keeps the compiler from taking it for the same one.)
template <int N, int V>
__device__ __forceinline__ void fetch_tiles(const Chain& ch, int64_t C, int first, int end, uint32_t at,
                                            bool on, bool with_state, Words<V> (&code)[N],
                                            Words<V> (&add)[N], Words<V>& state) {
  const __amdgpu_buffer_rsrc_t pc = rows_from(ch.code, first * C * 4),
                               pa = rows_from(ch.add, first * C * 4),
                               ps = rows_from(ch.state, (first - 1) * C * 4);
  const int last = end - 1 - first;  // (-1: none)
  for (int spins = 0; spins < kSpins; ++spins) {
    bool there = true;
    if (with_state) {
      state.load(ps, at, 0);
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j <= last) {
        const uint32_t row = (uint32_t)j * (uint32_t)C * 4u;
        code[j].load(pc, at, row);
        add[j].load(pa, at, row);
      }
    if (with_state) there = state.there();
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j <= last) there = there && code[j].there() && add[j].there();
    if (__all(there || !on)) return;
    asm volatile("" ::: "memory");
  }  // (an empty word is a NaN)
}

// What a tile's waves do between their own tokens and those tokens' states.  Every wave has
// put (set) its decay's sum and its contribution here, and whether a border lies in it;
// waves count in the order of the walk.  Afterwards (from) there is what every wave begins with.
// All waves come to run, `order` is their place; `alone` (asked of the first one): nothing
// comes from before the tile.
template <int W, int V, int REACH>
struct Carry {
  static constexpr int CB = 64 * V;
  static_assert(REACH % kByOne == 0, "whole pieces");
  float s_sum[W][CB], s_code[W][CB], s_add[W][CB];
  // of the tiles between (at most REACH - 1; a wave brings kByOne at a time)
  float s_tcode[REACH][CB], s_tadd[REACH][CB];
  int s_cut[W];
  int s_between;

  __device__ __forceinline__ void set(int order, const float (&sum)[V], const float (&code)[V],
                                      const float (&add)[V], bool cut) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s_sum[order][lane * V + v] = sum[v];
      s_code[order][lane * V + v] = code[v];
      s_add[order][lane * V + v] = add[v];
    }
    if (lane == 0) s_cut[order] = cut;
  }
  __device__ __forceinline__ float from(int order, int v) const {
    return s_sum[order][(threadIdx.x & 63) * V + v];
  }
  __device__ __forceinline__ void run(const Chain& ch, int k, int tiles, int block, int64_t C, int c,
                                      bool on, bool alone, int order) {
    const int lane = threadIdx.x & 63, at = lane * V;
    const uint32_t cb = c * 4;
    uint32_t* const mark = ch.mark + (int64_t)block * tiles;
    float own[V], from[V], tile_code[V];  // of wave 0
    bool cut = false;
    int n = 0;
    if (order == 0) {
      float all[V];
#pragma unroll
      for (int v = 0; v < V; ++v) own[v] = all[v] = from[v] = 0.0f;
#pragma unroll 2
      for (int w = 0; w < W; ++w) {
        const bool cw = s_cut[w] != 0;
        cut |= cw;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          all[v] += s_sum[w][at + v];
          own[v] = decayed_onto(cw ? __uint_as_float(kCut) : s_code[w][at + v], own[v],
                                s_add[w][at + v]);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) tile_code[v] = cut ? __uint_as_float(kCut) : decay_code(all[v]);
      if (tiles > 1) {
        if (on) {
          if (cut) publish<V>(rows_from(ch.state, k * C * 4), cb, own);
          publish<V>(rows_from(ch.code, k * C * 4), cb, tile_code);
          publish<V>(rows_from(ch.add, k * C * 4), cb, own);
        }
        if (lane == 0) poke(mark + k, cut ? 2u : 1u);
        if (!alone) {
          for (int spins = 0;; ++spins) {
            if (near_state<kByOne, V>(ch, C, k, cb, on, from)) break;
            n = marked_state<REACH>(mark, k);
            if (n > 0) break;
            n = 0;
            if (spins > kSpins) {
              from[0] = from[V - 1] = __builtin_nanf("");
              break;
            }
            asm volatile("" ::: "memory");
          }
        }
      }
      if (lane == 0) s_between = n;
    }
    __syncthreads();
    n = __builtin_amdgcn_readfirstlane(s_between);
    if (n > 0) {  // many tiles between: every wave brings some of them to LDS
      Words<V> state;
      for (int j0 = order * kByOne; j0 < n; j0 += W * kByOne) {
        Words<V> code[kByOne], add[kByOne];
        fetch_tiles<kByOne, V>(ch, C, k - n + j0, k, cb, on, order + j0 == 0, code, add, state);
        if (order + j0 == 0)
#pragma unroll
          for (int v = 0; v < V; ++v) from[v] = state.get(v);
#pragma unroll
        for (int j = 0; j < kByOne; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) {  // (past n whatever there was)
            s_tcode[j0 + j][at + v] = code[j].get(v);
            s_tadd[j0 + j][at + v] = add[j].get(v);
          }
      }
      __syncthreads();
    }
    if (order == 0) {
#pragma unroll 4
      for (int j = 0; j < n; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v)
          from[v] = decayed_onto(s_tcode[j][at + v], from[v], s_tadd[j][at + v]);
      if (tiles > 1 && !cut) {
#pragma unroll
        for (int v = 0; v < V; ++v) own[v] = decayed_onto(tile_code[v], from[v], own[v]);
        if (on) publish<V>(rows_from(ch.state, k * C * 4), cb, own);
        if (lane == 0) poke(mark + k, 2u);
      }
#pragma unroll 2
      for (int w = 0; w < W; ++w) {
        const bool cw = s_cut[w] != 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          s_sum[w][at + v] = from[v];
          from[v] = decayed_onto(cw ? __uint_as_float(kCut) : s_code[w][at + v], from[v],
                                 s_add[w][at + v]);
        }
      }
    }
    __syncthreads();
  }
};

}  // namespace gatedrec
}  // namespace kda
