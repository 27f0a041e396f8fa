// What the forward and the backward of the gated linear recurrence share on the device:
// the gate, the packed batch's borders, and the carry between tiles.
#pragma once

#include "gatedrec.hpp"
#include "kda_device.hpp"

namespace kda {
namespace gatedrec {

// ------------------------------------------------------------------ values
// V neighbouring channels of one token as they lie in memory.
template <bool BF16, int V>
struct Vals {
  typedef uint16_t E __attribute__((ext_vector_type(V)));
  E r;
  __device__ __forceinline__ void load(const char* p) { r = *reinterpret_cast<const E*>(p); }
  __device__ __forceinline__ float get(int v) const { return bf16_bits_to_f32(r[v]); }
  static __device__ __forceinline__ void store(char* p, const float (&x)[V]) {
    E o;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = f32_to_bf16_bits(x[v]);
    *reinterpret_cast<E*>(p) = o;
  }
};
template <int V>
struct Vals<false, V> {
  typedef float E __attribute__((ext_vector_type(V)));
  E r;
  __device__ __forceinline__ void load(const char* p) { r = *reinterpret_cast<const E*>(p); }
  __device__ __forceinline__ float get(int v) const { return r[v]; }
  static __device__ __forceinline__ void store(char* p, const float (&x)[V]) {
    E o;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = x[v];
    *reinterpret_cast<E*>(p) = o;
  }
};
template <int V>
__device__ __forceinline__ void load_state(const void* p, int64_t at, float (&x)[V], bool bf16) {
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = load1(p, at + v, bf16);
}
template <int V>
__device__ __forceinline__ void store_row(void* p, int64_t at, const float (&x)[V], bool bf16) {
  if (bf16) Vals<true, V>::store(static_cast<char*>(p) + at * 2, x);
  else Vals<false, V>::store(static_cast<char*>(p) + at * 4, x);
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

// Values a lane takes at once: two of bf16 (4 bytes a lane) where every row and output is
// aligned to that, else one.
struct Out {
  const void* p;
  bool bf16;
};
inline int width(const Inputs& in, int C, const Out* outs, int count) {
  if (!in.bf16 || C % 2) return 1;
  for (const Rows* r : {&in.x, &in.r, &in.i})
    if (reinterpret_cast<uintptr_t>(r->p) % 4 || r->stride % 2) return 1;
  for (int k = 0; k < count; ++k)
    if (reinterpret_cast<uintptr_t>(outs[k].p) % (outs[k].bf16 ? 4 : 8)) return 1;
  return 2;
}

// -------------------------------------------------------------------- gate
// Log-decays are in log2 units throughout (g2 = g log2(e), a = 2^g2): the scale goes into
// constants that are multiplied anyway.  The polynomials are minimax fits of the relative
// error over the stated ranges.
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// log(1 + e) for 0 <= e <= 1: e times a polynomial, 3 u of itself (u = 2^-24).  A hardware
// log with its correction for small e (gate_math.hpp) costs half as much again.
__device__ __forceinline__ float log1p_unit(float e) {
  float p = 0.005232629366219044f;
  p = fmaf(p, e, -0.029504986479878426f);
  p = fmaf(p, e, 0.07822556048631668f);
  p = fmaf(p, e, -0.13663214445114136f);
  p = fmaf(p, e, 0.1910599321126938f);
  p = fmaf(p, e, -0.2484297901391983f);
  p = fmaf(p, e, 0.3331909775733948f);
  p = fmaf(p, e, -0.4999949336051941f);
  p = fmaf(p, e, 0.9999999403953552f);
  return e * p;
}
// 1 - 2^y for y <= 0, e = 2^y: the difference loses the digits of a small y, so there it is a
// polynomial (0.3 u).
__device__ __forceinline__ float one_minus_exp2(float y, float e) {
  float p = 0.0011528132017701864f;
  p = fmaf(p, y, 0.009539824910461903f);
  p = fmaf(p, y, 0.055490005761384964f);
  p = fmaf(p, y, 0.24022559821605682f);
  p = fmaf(p, y, 0.6931471824645996f);
  return y > -0.5f ? -y * p : 1.0f - e;  // NaN stays NaN
}
// 1 - 4^g2 for g2 <= 0, a = 2^g2: the same at y = 2 g2.
__device__ __forceinline__ float one_minus_square(float g2, float a) {
  float p = 0.036890022456645966f;
  p = fmaf(p, g2, 0.15263719856739044f);
  p = fmaf(p, g2, 0.4439200460910797f);
  p = fmaf(p, g2, 0.9609023928642273f);
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
  float neg_a[GATE ? V : 1], neg_a2[GATE ? V : 1], bias2[GATE ? V : 1];
  __device__ __forceinline__ void load(const Inputs& in, int c) {
    if constexpr (GATE) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        neg_a[v] = -expf(in.A_log[c + v]);
        neg_a2[v] = neg_a[v] * kLog2e;
        bias2[v] = in.dt_bias ? in.dt_bias[c + v] * kLog2e : 0.0f;
      }
    }
  }
  // g2; e: exp(-|z|), z2: z log2(e) (of the gate, for its slope)
  __device__ __forceinline__ float log2_decay(float r, int v, float& z2, float& e) const {
    if constexpr (GATE) {
      z2 = fmaf(r, kLog2e, bias2[v]);
      e = exp2_fast(-fabsf(z2));
      return fmaf(neg_a[v], fmaxf(z2, 0.0f), neg_a2[v] * log1p_unit(e));  // (a NaN is in e)
    }
    z2 = e = 0.0f;
    return r > 0.0f ? 0.0f : r * kLog2e;  // NaN stays NaN
  }
  __device__ __forceinline__ float log2_decay(float r, int v) const {
    float z2, e;
    return log2_decay(r, v, z2, e);
  }
};

// ------------------------------------------------------------ decay factors
// A stretch's decay 2^s, s the sum of its log2-decays, as one number `code`: beside 1 it is
// 1 - d with d = 1 - 2^s kept (code = d, sign clear), for 2^s itself would be rounded to
// 6e-8, which over the stretches of a slow channel adds up to 6e-8 / d of the state.
// Further away it is 2^s (code = -2^s, sign set).
__device__ __forceinline__ float decay_code(float s) {
  const float e = exp2_fast(s);
  const float d = one_minus_exp2(s, e);
  return d < 0.5f ? d : -e;  // NaN stays NaN
}
__device__ __forceinline__ float decayed_onto(float code, float h, float add) {
  const float t = fmaf(-code, h, add);
  return __float_as_int(code) < 0 ? t : t + h;
}

// ----------------------------------------------------------- packed batch
struct Seqs {
  const int32_t* cu;
  int N, T, len;  // len: tokens of every sequence when cu is null
  __device__ __forceinline__ int clamp(int t) const { return t < 0 ? 0 : t > T ? T : t; }
  __device__ __forceinline__ int start(int n) const { return cu ? clamp(cu[n]) : n * len; }
  __device__ __forceinline__ int live() const { return cu ? clamp(cu[N]) : T; }
  // the last sequence that begins at or before t
  __device__ __forceinline__ int find(int t) const {
    if (!cu) return len > 0 ? t / len : 0;
    int lo = 0, hi = N - 1;
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (cu[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};
// The borders among the `count` (at most 32) tokens from t0: bit j of `first` (`last`) says
// that token t0 + j is the first (last) of its sequence.
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
// The tiles of a channel hand their state on.  Tile k (in the order of the walk) first
// publishes its own decay and contribution (code, add), then waits for the state of the
// tile before it and publishes its own.  A word that is not there yet is all ones; what
// is published never is.  Nothing else is ordered by these words, so every access is a
// relaxed one, at agent scope because neighbouring tiles run on different XCDs.
//
// Tiles are given out by a ticket, so whoever is waited for is running or done.  A tile
// folds what lies between it and the nearest state one by one, forwards: whichever tile
// that is, the bits are the same.
//
// Should the words be spoilt (the workspace used by something else meanwhile), a wait
// gives up after kSpins and the tile goes on with NaN: every wait ends.
constexpr uint32_t kEmpty = 0xffffffffu;
constexpr int kSpins = 1 << 20;
constexpr int kWindow = 64;  // how far back a state is looked for

struct Chain {
  uint32_t* ticket;  // null: one workgroup walks all tiles of its channels
  uint32_t *state, *code, *add;  // [tiles][C]
};
inline size_t chain_bytes(int64_t tiles, int64_t C) {
  return (256 + (size_t)tiles * C * 12 + 255) / 256 * 256;
}
// makes every word empty, the ticket too
hipError_t launch_fill(void* ws, size_t bytes, hipStream_t s);
inline Chain chain_at(void* ws, int64_t tiles, int64_t C) {
  Chain c;
  c.ticket = static_cast<uint32_t*>(ws);
  c.state = c.ticket + 64;
  c.code = c.state + tiles * C;
  c.add = c.code + tiles * C;
  return c;
}

template <int V>
__device__ __forceinline__ void publish(uint32_t* p, const float (&x)[V]) {
  uint32_t w[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    w[v] = __float_as_uint(x[v]);
    if (w[v] == kEmpty) w[v] = 0x7fc00000u;
  }
  if constexpr (V == 1) {
    __hip_atomic_store(p, w[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2)
      __hip_atomic_store(reinterpret_cast<uint64_t*>(p + v),
                         (uint64_t)w[v] | (uint64_t)w[v + 1] << 32, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
  }
}
template <int V>
struct Words {
  uint32_t w[V];
  __device__ __forceinline__ void load(const uint32_t* p) {
    if constexpr (V == 1) {
      w[0] = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    } else {
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        const uint64_t x = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p + v),
                                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        w[v] = (uint32_t)x;
        w[v + 1] = (uint32_t)(x >> 32);
      }
    }
  }
  // whether every lane's words are there (lanes without channels: `on` false)
  __device__ __forceinline__ bool ready(bool on) const {
    bool r = true;
#pragma unroll
    for (int v = 0; v < V; ++v) r &= w[v] != kEmpty;
    return __all(r || !on);
  }
  __device__ __forceinline__ float get(int v) const { return __uint_as_float(w[v]); }
};

// The state behind tile k - 1 (k > 0) of a wave's channels c.
template <int V>
__device__ __forceinline__ void look_back(const Chain& ch, int64_t C, int k, int c, bool on,
                                          float (&h)[V]) {
  constexpr int B = 8;
  int spins = 0, q = -1;
  Words<V> st;
  while (q < 0) {  // the nearest state that is there
    for (int b = k - 1; b >= 0 && b > k - 1 - kWindow && q < 0; b -= B) {
      Words<V> w[B];
#pragma unroll
      for (int j = 0; j < B; ++j) w[j].load(ch.state + (int64_t)(b - j < 0 ? 0 : b - j) * C + c);
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (q < 0 && b - j >= 0 && w[j].ready(on)) {
          q = b - j;
          st = w[j];
        }
    }
    if (q < 0) {
      if (++spins > kSpins) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = __builtin_nanf("");
        return;
      }
      __builtin_amdgcn_s_sleep(1);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = st.get(v);
  for (int b = q + 1; b < k; b += B) {
    Words<V> code[B], add[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int64_t at = (int64_t)(b + j < k ? b + j : k - 1) * C + c;
      code[j].load(ch.code + at);
      add[j].load(ch.add + at);
    }
#pragma unroll
    for (int j = 0; j < B; ++j) {
      if (b + j < k) {
        const int64_t at = (int64_t)(b + j) * C + c;
        bool whole = false;  // the tile's state came instead
        while (!(code[j].ready(on) && add[j].ready(on))) {
          st.load(ch.state + at);
          if (st.ready(on)) {
            whole = true;
            break;
          }
          if (++spins > kSpins) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = __builtin_nanf("");
            return;
          }
          __builtin_amdgcn_s_sleep(1);
          code[j].load(ch.code + at);
          add[j].load(ch.add + at);
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
          h[v] = whole ? st.get(v) : decayed_onto(code[j].get(v), h[v], add[j].get(v));
      }
    }
  }
}

}  // namespace gatedrec
}  // namespace kda
