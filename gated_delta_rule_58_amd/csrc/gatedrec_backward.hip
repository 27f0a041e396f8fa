// kda_gatedrec_scan_backward: gradients of the gated linear recurrence, per channel
//
//   R_t = dh_t + e_{t+1},  e_t = a_t R_t    (e behind the last token: d_final_state)
//   du = m R;  dx = du s;  di = du x s (1 - s),  s = sigmoid(i)
//   dg = a h_{t-1} R - (a^2 / m) s x R      (the second part where m is normalised)
//   dr = dg dg/dr;  dA_log = sum_t dg g;  ddt_bias = sum_t dr;  d_initial_state = e_1
//
// x, r, i and dh are read once and the gradients written once.  h is formed again in fp32
// from the states that the forward saved every kStartsTokens tokens (without them the
// forward's walk runs first, for those states alone).  A tile is kTile tokens of 64 V
// channels, worked on like a tile of the forward, but the tiles hand on e, from the last
// one to the first.
//
// The parameters' gradients: every tile's sum goes to memory, a second kernel adds them in
// a fixed order.
//
// What bounds it: the vector unit and the ways of a tile to memory and back, as in the
// forward, with 1.75 times its traffic.  4,096 x 12,288 bf16: 207 us, 3.4 TB/s of the 711 MB it
// has to move (137 us at a copy's rate).  A value takes 88 instructions: 32 for the gate and m, 29
// for the products, 6 for the gradients, the rest a tile's borders, sums and carry.  What is
// formed twice (a, sigmoid(r)) is cheaper than the registers that would keep it: a wave's tokens,
// their gate's values and the products before the carry take 164 of 168.
#include <type_traits>

#include "gatedrec_device.hpp"

namespace kda {
namespace gatedrec {
namespace {

// L tokens a wave, W waves, waves a SIMD, the tiles that a look back reaches.  A longer tile has
// fewer carries, more registers a lane hold fewer waves back.  Measured, forward and backward
// of 4,096 x 12,288 bf16 (V = 2) when 8 x 4 took 336 us: 8 x 8 with 128 registers, spilt, 408;
// 6 x 8 362; 4 x 16 598.  2,999 x 1,536 fp32 (V = 1): 8 x 8 89, 8 x 4 97, 16 x 4 93.
template <int V>
struct Shape {
  static constexpr int L = 8, W = 8, OCC = 4, REACH = 60, TILE = L * W;
};
template <>
struct Shape<2> {
  static constexpr int L = 8, W = 4, OCC = 3, REACH = 40, TILE = L * W;
};
constexpr int kLeastTile = 32;
static_assert(Shape<1>::TILE % kStartsTokens == 0 && Shape<2>::TILE % kStartsTokens == 0 &&
                  Shape<1>::TILE >= kLeastTile && Shape<2>::TILE >= kLeastTile,
              "a state for every tile");

struct Args {
  Inputs in;
  Seqs q;
  int C;
  const float *S0, *starts, *dS;
  const void* dh;
  Gradients out;
  float* part;  // [tiles][2][C]
  Chain chain;
  int tiles, blocks;
  Split by_blocks;
};

// The gradient of an entry state without tokens is that of the exit state.
__device__ void copy_empty(const Args& A, int first, int step) {
  for (int n = first; n < A.q.N; n += step) {
    if (A.q.start(n + 1) > A.q.start(n)) continue;
    for (int c = threadIdx.x; c < A.C; c += blockDim.x) {
      const int64_t at = (int64_t)n * A.C + c;
      A.out.dS0[at] = A.dS ? A.dS[at] : 0.0f;
    }
  }
}

template <bool BF16, bool DB, int V, bool GATE, bool GATED, bool NORM>
__global__ void __launch_bounds__(64 * Shape<V>::W, Shape<V>::OCC)
    backward_kernel(const Args A) {
#pragma clang fp contract(off)  // (the same digits on every path: sums of products are spelt out)
  constexpr int L = Shape<V>::L, W = Shape<V>::W, CB = 64 * V, ES = BF16 ? 2 : 4;
  constexpr int kTile = Shape<V>::TILE;
  __shared__ Carry<W, V, Shape<V>::REACH> s;          // backwards: wave W - 1 comes first
  __shared__ float s_add[W][CB];           // forwards
  __shared__ int s_first[W];
  __shared__ uint32_t s_ticket;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int work = A.tiles * A.blocks;
  if ((int)blockIdx.x >= work) {
    copy_empty(A, blockIdx.x - work, gridDim.x - work);
    return;
  }
  int id = blockIdx.x;
  if (A.tiles > 1) {
    if (threadIdx.x == 0)
      s_ticket = __hip_atomic_fetch_add(A.chain.ticket, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT) + 1u;
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(s_ticket);
    if ((uint32_t)id >= (uint32_t)work) return;
  }
  int block;
  const int k = A.by_blocks(id, block);
  const int tile = A.tiles - 1 - k;
  const int tile0 = tile * kTile, live = A.q.live();
  const int c = block * CB + lane * V;
  const bool on = c < A.C;
  const int cc = on ? c : 0;
  if (tile0 >= live) {  // behind the last sequence: nothing is waited for from here
    if (A.part && wave == 0 && on)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A.part[((int64_t)tile * 2) * A.C + c + v] = 0.0f;
        A.part[((int64_t)tile * 2 + 1) * A.C + c + v] = 0.0f;
      }
    return;
  }
  const int t0 = tile0 + wave * L;

  Vals<BF16, V> rx[L], rr[L], ri[GATED ? L : 1];
  Vals<DB, V> rd[L];
  {
    const int t = t0 < live ? t0 : live - 1, most = live - 1 - t;  // (the last row again)
    const uint32_t at = cc * ES, DS = DB ? 2 : 4;
    const uint32_t sx = A.in.x.stride * ES, sr = A.in.r.stride * ES, si = A.in.i.stride * ES,
                   sd = A.C * DS;
    const __amdgpu_buffer_rsrc_t px = rows_from(A.in.x.p, (int64_t)t * sx),
                                 pr = rows_from(A.in.r.p, (int64_t)t * sr),
                                 pi = rows_from(A.in.i.p, (int64_t)t * si),
                                 // (without dh its loads give 0; the select is uniform, which
                                 // the compiler has to be told or it loops over the lanes)
                                 pd = buffer_over(
                                     static_cast<const char*>(A.dh) + (int64_t)t * sd,
                                     __builtin_amdgcn_readfirstlane(A.dh ? 0xffffffffu : 0u));
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const uint32_t row = j < most ? j : most;
      rr[j].load(pr, at, row * sr);
      if constexpr (GATED) ri[j].load(pi, at, row * si);
      rx[j].load(px, at, row * sx);
    }
#pragma unroll
    for (int j = 0; j < L; ++j) rd[j].load(pd, cc * DS, (j < most ? j : most) * sd);
  }
  auto dh = [&](int j, int v) { return rd[j].get(v); };
  float start[V];  // the state before the tile
#pragma unroll
  for (int v = 0; v < V; ++v) start[v] = A.starts[(int64_t)(tile0 / kStartsTokens) * A.C + cc + v];
  Params<V, GATE> par;
  par.load(A.in, cc);
  Borders bd;
  bd.find(A.q, t0, live - t0 < L ? live - t0 : L);
  // x of the sequence of token t0 + j, zeros without x
  auto of_sequence = [&](const float* p, int j, float (&x)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = 0.0f;
    if (p) load_state<V>(p, (int64_t)A.q.find(t0 + j) * A.C + cc, x, false);
  };

  // First every token's g, m and s, the wave's decay, what it adds to the state, and e
  // before it from what comes in: with P_t the decay from the wave's first token to t,
  // back = sum_t P_t dh_t.  (a is formed again below: 16 registers for two cycles a value.)
  // m and s stay apart: m s may be too small for its reciprocal, where s / m is not.
  float g[L][V], px[L][V], pi[L][V];
  float sum[V], add[V], back[V], P[V];
  auto chain = [&](int j, auto borders) {
#pragma clang fp contract(off)
    float dS[V] = {};
    bool in = true;
    if constexpr (borders) {
      if (bd.first >> j & 1u) of_sequence(A.S0, j, add);
      if (bd.last >> j & 1u) of_sequence(A.dS, j, dS);
      in = !(bd.last & ((1u << j) - 1));  // (back: up to the first border)
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float a = exp2_fast(g[j][v]);
      float b = rx[j].get(v);
      if constexpr (GATED) b *= pi[j][v];
      if constexpr (NORM) b *= px[j][v];
      add[v] = fmaf(a, add[v], b);
      P[v] *= a;
      float d = dh(j, v);
      if constexpr (borders) d += dS[v];
      if (in) back[v] = fmaf(P[v], d, back[v]);
    }
  };
#pragma unroll
  for (int v = 0; v < V; ++v) sum[v] = add[v] = back[v] = 0.0f, P[v] = 1.0f;
#pragma unroll
  for (int j = 0; j < L; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      g[j][v] = par.log2_decay(rr[j].get(v), v);
      px[j][v] = pi[j][v] = 1.0f;
      if constexpr (GATED) pi[j][v] = sigmoid_fast(ri[j].get(v));
      if constexpr (NORM)
        px[j][v] = __builtin_amdgcn_sqrtf(one_minus_square(g[j][v], exp2_fast(g[j][v])));
      sum[v] += g[j][v];
    }
    chain(j, std::false_type{});
  }
  // What is formed again is formed again: kept from before, it would not fit the registers.
  auto again = [&] {
#pragma unroll
    for (int j = 0; j < L; ++j) {
      hold(rx[j].w[0]);
      hold(rr[j].w[0]);
      hold(rd[j].w[0]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        hold(g[j][v]);
        if constexpr (GATED && NORM) {
          hold(px[j][v]);
          hold(pi[j][v]);
        }
      }
    }
  };
  if (bd.first | bd.last) {
    again();
#pragma unroll
    for (int v = 0; v < V; ++v) add[v] = back[v] = 0.0f, P[v] = 1.0f;
#pragma unroll
    for (int j = 0; j < L; ++j) chain(j, std::true_type{});
  }
  const int order = W - 1 - wave;
  float code[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    code[v] = decay_code(sum[v]);
    s_add[wave][lane * V + v] = add[v];
  }
  if (lane == 0) s_first[wave] = bd.first != 0;
  s.set(order, sum, code, back, bd.last != 0);
  __syncthreads();
  again();
  // forwards: the state that the wave begins with
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = start[v];
  for (int w = 0; w < wave; ++w) {
    const bool cw = s_first[w] != 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = decayed_onto(cw ? __uint_as_float(kCut) : s.s_code[W - 1 - w][lane * V + v], h[v],
                          s_add[w][lane * V + v]);
    }
  }
  // Then everything that R is multiplied with, before R is known: dx = px R, di = pi R,
  // dr = pr R, with p = m s in the place of m and a in that of g.  The parameters' sums too: R_t
  // is the sum of what comes in at s >= t (dh_s, or e behind the wave) times the decay between, so
  // with pg = q g
  //   sum_t R_t pg_t = sum_s dh_s Q_s + e Q_L,   Q_s = a_s Q_{s-1} + pg_s
  // which needs no register a token and goes forwards.
  float (&a)[L][V] = g, pr[L][V];
  float dA[V], db[V], QA[V], Qb[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dA[v] = db[v] = QA[v] = Qb[v] = 0.0f;
  auto products = [&](auto borders) {
#pragma clang fp contract(off)
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float dS[V] = {};
      if constexpr (borders) {
        if (bd.first >> j & 1u) {
          of_sequence(A.S0, j, h);
#pragma unroll
          for (int v = 0; v < V; ++v) QA[v] = Qb[v] = 0.0f;
        }
        if (bd.last >> j & 1u) of_sequence(A.dS, j, dS);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = rx[j].get(v), r = rr[j].get(v);
        const float gg = g[j][v], aa = exp2_fast(gg), m = px[j][v], s = pi[j][v];
        float u = x, p = m, before = h[v];
        if constexpr (GATED) {
          u *= s;
          p *= s;
        }
        // where m is 0 this part is 0
        if constexpr (NORM)
          before = fmaf(-aa, m > 0.0f ? u * __builtin_amdgcn_rcpf(m) : 0.0f, before);
        const float q = aa * before;
        h[v] = fmaf(aa, h[v], m * u);
        px[j][v] = p;
        if constexpr (GATED) pi[j][v] = m * u * (1.0f - s);
        a[j][v] = aa;
        if constexpr (GATE) {
          // (where g is -inf the decay is 0, and q with it)
          const float pg = q * fmaxf(gg, -3.0e38f);
          pr[j][v] = q * par.neg_a[v] *
                     __builtin_amdgcn_rcpf(1.0f + exp2_fast(-fmaf(r, kLog2e, par.bias2[v])));
          float in = dh(j, v);
          if constexpr (borders) in += dS[v];
          if (!borders || t0 + j < live) {
            QA[v] = fmaf(aa, QA[v], pg);
            Qb[v] = fmaf(aa, Qb[v], pr[j][v]);
            dA[v] = fmaf(in, QA[v], dA[v]);
            db[v] = fmaf(in, Qb[v], db[v]);
          }
        } else {
          pr[j][v] = r > 0.0f ? 0.0f : q;
        }
      }
    }
  };
  const bool plain = t0 + L <= live && !(bd.first | bd.last);
  if (plain) products(std::false_type{});
  else products(std::true_type{});
  // the tile ends with a sequence: nothing comes from behind (wave W - 1 asks)
  const bool alone = tile0 + kTile >= live || (bd.last >> (L - 1) & 1u);
  s.run(A.chain, k, A.tiles, block, A.C, cc, on, alone, order);

#pragma unroll
  for (int j = 0; j < L; ++j) hold(rd[j].w[0]);
  float e[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    e[v] = s.from(order, v);
    if (t0 + L <= live && !(bd.last >> (L - 1) & 1u)) {  // (not of another sequence)
      dA[v] = fmaf(e[v], QA[v], dA[v]);
      db[v] = fmaf(e[v], Qb[v], db[v]);
    }
  }
  const uint32_t row = A.C * (A.out.bf16 ? 2 : 4);
  const __amdgpu_buffer_rsrc_t ox = rows_from(A.out.dx, (int64_t)t0 * row),
                               orr = rows_from(A.out.dr, (int64_t)t0 * row),
                               oi = rows_from(A.out.di, (int64_t)t0 * row);
  auto gradients = [&](auto borders, auto bf) {
#pragma clang fp contract(off)
    constexpr bool OB = bf;
    constexpr int OS = OB ? 2 : 4;
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
      if constexpr (borders) {
        if (t0 + j >= live) continue;
        if (bd.last >> j & 1u) of_sequence(A.dS, j, e);
      }
      float dx[V], dr[V], di[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float R = dh(j, v) + e[v];
        e[v] = a[j][v] * R;
        dx[v] = px[j][v] * R;
        dr[v] = pr[j][v] * R;
        if constexpr (GATED) di[v] = pi[j][v] * R;
      }
      if (on) {
        Vals<OB, V>::store(ox, c * OS, j * row, dx);
        Vals<OB, V>::store(orr, c * OS, j * row, dr);
        if constexpr (GATED) Vals<OB, V>::store(oi, c * OS, j * row, di);
        if constexpr (borders)
          if (A.out.dS0 && (bd.first >> j & 1u))
            store_state<V>(A.out.dS0, (int64_t)A.q.find(t0 + j) * A.C + c, e, false);
      }
    }
  };
  if (A.out.bf16) {
    if (plain) gradients(std::false_type{}, std::true_type{});
    else gradients(std::true_type{}, std::true_type{});
  } else {
    if (plain) gradients(std::false_type{}, std::false_type{});
    else gradients(std::true_type{}, std::false_type{});
  }
  if constexpr (GATE) {
    if (A.part) {
      __syncthreads();  // what is there has been read
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s.s_add[wave][lane * V + v] = dA[v];
        s.s_code[wave][lane * V + v] = db[v];
      }
      __syncthreads();
      if (wave == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float x = 0.0f, y = 0.0f;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            x += s.s_add[w][lane * V + v];  // (of log2-decays)
            y += s.s_code[w][lane * V + v];
          }
          A.part[((int64_t)tile * 2) * A.C + c + v] = x * kLn2;
          A.part[((int64_t)tile * 2 + 1) * A.C + c + v] = y;
        }
    }
  }
}

// dA_log, ddt_bias [C] from the tiles' sums [tiles][2][C]: 64 columns a workgroup, 16 lanes
// in turn a column; in 64 bits, in a fixed order.
__global__ void __launch_bounds__(1024) partials_kernel(const float* __restrict__ part,
                                                        int64_t tiles, int64_t C,
                                                        float* __restrict__ dA,
                                                        float* __restrict__ db) {
  __shared__ double s[16][64];
  const int cl = threadIdx.x & 63, k = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + cl;  // column of [2][C]
  double acc = 0.0;
  if (c < 2 * C)
    for (int64_t t = k; t < tiles; t += 16 * 8) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = t + 16 * j < tiles ? part[(t + 16 * j) * 2 * C + c] : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc += x[j];
    }
  s[k][cl] = acc;
  __syncthreads();
  if (k == 0 && c < 2 * C) {
    for (int j = 1; j < 16; ++j) acc += s[j][cl];
    float* out = c < C ? dA : db;
    if (out) out[c < C ? c : c - C] = (float)acc;
  }
}

int64_t tiles_of(int64_t T, int tile = kLeastTile) { return (T + tile - 1) / tile; }
size_t part_bytes(int64_t T, int64_t C) {
  return ((size_t)tiles_of(T) * 2 * C * sizeof(float) + 255) / 256 * 256;
}
size_t carries_bytes(int64_t T, int64_t C, bool has_starts) {
  const size_t own = chain_bytes(tiles_of(T), C), scan = scan_workspace_bytes(T, C);
  return has_starts || own > scan ? own : scan;
}
size_t own_starts_bytes(int64_t T, int64_t C) { return (starts_bytes(T, C) + 255) / 256 * 256; }

}  // namespace

bool backward_fits(const Batch& b) {  // at most 512 threads a workgroup, fewer than 2^32 in a launch
  return tiles_of(b.T) * ((b.C + 63) / 64) < ((int64_t)1 << 23) - 1024;
}

// The tiles' carries (the forward's, without starts, have been in the same place before), the
// parameters' sums, and the states of a call without starts.
size_t backward_workspace_bytes(int64_t T, int64_t C, bool has_starts) {
  return carries_bytes(T, C, has_starts) + part_bytes(T, C) +
         (has_starts ? 0 : own_starts_bytes(T, C));
}

hipError_t launch_backward(const Inputs& in, const Batch& b, const float* S0, const float* starts,
                           const void* dh, bool dh_bf16, const float* dS, const Gradients& out,
                           void* ws, hipStream_t s) {
  char* base = static_cast<char*>(ws);
  char* const part = base + carries_bytes(b.T, b.C, starts != nullptr);
  Args A;
  A.in = in;
  A.q = Seqs{b.cu, b.N, b.T, b.N > 0 ? b.T / b.N : 0};
  A.C = b.C;
  A.S0 = S0;
  A.dS = dS;
  A.dh = dh;
  A.out = out;
  A.part = in.A_log && (out.dA_log || out.ddt_bias) ? reinterpret_cast<float*>(part) : nullptr;
  const Out outs[] = {{dh, dh_bf16}, {out.dx, out.bf16}, {out.dr, out.bf16}, {out.di, out.bf16}};
  const int V = width(in, b.C, outs, 4);
  A.tiles = (int)tiles_of(b.T, V == 2 ? Shape<2>::TILE : Shape<1>::TILE);
  A.chain = Chain{};
  if (!starts && b.T > 0) {
    float* own = reinterpret_cast<float*>(part + part_bytes(b.T, b.C));
    StatePool st;
    st.in = S0;
    st.slots = b.N;
    if (const hipError_t e = launch_scan(in, b, st, nullptr, false, own, base, s)) return e;
    starts = own;
  }
  A.starts = starts;
  if (A.tiles > 1) {
    if (const hipError_t e = launch_fill(base, chain_bytes(A.tiles, b.C), s)) return e;
    A.chain = chain_at(base, A.tiles, b.C);
  }
  A.blocks = (b.C + 64 * V - 1) / (64 * V);
  A.by_blocks = Split(A.blocks);
  bool empties = out.dS0 != nullptr;
  if (empties && b.cu_host) {
    empties = false;
    for (int n = 0; n < b.N && !empties; ++n) empties = b.cu_host[n + 1] == b.cu_host[n];
  }
  if (!b.cu && b.T > 0) empties = false;
  const int64_t work = (int64_t)A.tiles * A.blocks;
  const int64_t grid = work + (empties ? (b.N < 256 ? b.N : 256) : 0);
  if (grid > 0) {
#define KDA_GR(BF, V_, G, I, N_)                                                              \
  do {                                                                                        \
    if (dh_bf16) backward_kernel<BF, true, V_, G, I, N_><<<(unsigned)grid, 64 * Shape<V_>::W, 0, s>>>(A); \
    else backward_kernel<BF, false, V_, G, I, N_><<<(unsigned)grid, 64 * Shape<V_>::W, 0, s>>>(A);  \
  } while (0)
#define KDA_GR_N(BF, V_, G, I)                 \
  do {                                         \
    if (in.normalize) KDA_GR(BF, V_, G, I, true); \
    else KDA_GR(BF, V_, G, I, false);          \
  } while (0)
#define KDA_GR_I(BF, V_, G)                \
  do {                                     \
    if (in.i.p) KDA_GR_N(BF, V_, G, true); \
    else KDA_GR_N(BF, V_, G, false);       \
  } while (0)
#define KDA_GR_G(BF, V_)                   \
  do {                                     \
    if (in.A_log) KDA_GR_I(BF, V_, true);  \
    else KDA_GR_I(BF, V_, false);          \
  } while (0)
    if (!in.bf16) KDA_GR_G(false, 1);
    else if (V == 2) KDA_GR_G(true, 2);
    else KDA_GR_G(true, 1);
#undef KDA_GR_G
#undef KDA_GR_I
#undef KDA_GR_N
#undef KDA_GR
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (in.A_log && (out.dA_log || out.ddt_bias)) {
    partials_kernel<<<(unsigned)((2 * (int64_t)b.C + 63) / 64), 1024, 0, s>>>(
        A.part, A.tiles, b.C, out.dA_log, out.ddt_bias);
  }
  return hipGetLastError();
}

}  // namespace gatedrec
}  // namespace kda
