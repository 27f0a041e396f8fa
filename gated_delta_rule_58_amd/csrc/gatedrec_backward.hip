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
#include "gatedrec_device.hpp"

namespace kda {
namespace gatedrec {
namespace {

constexpr int kWaves = 8;
constexpr int kL = 8;
constexpr int kTile = kWaves * kL;
static_assert(kTile == kStartsTokens, "a state for every tile");

struct Args {
  Inputs in;
  Seqs q;
  int C;
  const float *S0, *starts, *dS;
  const void* dh;
  bool dh_bf16;
  Gradients out;
  float* part;  // [tiles][2][C]
  Chain chain;
  int tiles, blocks;
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

template <bool BF16, int V, bool GATE, bool GATED, bool NORM>
__global__ void __launch_bounds__(64 * kWaves, 4) backward_kernel(const Args A) {
  constexpr int L = kL, W = kWaves, CB = 64 * V, ES = BF16 ? 2 : 4;
  __shared__ Carry<W, V> s;                // backwards: wave W - 1 comes first
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
  const int k = id / A.blocks, block = id - k * A.blocks;
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
  float dh[L][V];
  {
    const int t = t0 < live ? t0 : live - 1, most = live - 1 - t;  // (the last row again)
    const uint32_t at = cc * ES;
    const uint32_t sx = A.in.x.stride * ES, sr = A.in.r.stride * ES, si = A.in.i.stride * ES;
    const __amdgpu_buffer_rsrc_t px = rows_from(A.in.x.p, (int64_t)t * sx),
                                 pr = rows_from(A.in.r.p, (int64_t)t * sr),
                                 pi = rows_from(A.in.i.p, (int64_t)t * si);
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const uint32_t row = j < most ? j : most;
      rr[j].load(pr, at, row * sr);
      if constexpr (GATED) ri[j].load(pi, at, row * si);
      rx[j].load(px, at, row * sx);
    }
    const uint32_t sd = A.C * (A.dh_bf16 ? 2 : 4);
    const __amdgpu_buffer_rsrc_t pd = rows_from(A.dh, (int64_t)t * sd);
    if (!A.dh) {
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dh[j][v] = 0.0f;
    } else if (A.dh_bf16) {
      Vals<true, V> d[L];
#pragma unroll
      for (int j = 0; j < L; ++j) d[j].load(pd, cc * 2, (j < most ? j : most) * sd);
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dh[j][v] = d[j].get(v);
    } else {
      Vals<false, V> d[L];
#pragma unroll
      for (int j = 0; j < L; ++j) d[j].load(pd, cc * 4, (j < most ? j : most) * sd);
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dh[j][v] = d[j].get(v);
    }
  }
  float start[V];  // the state before the tile
#pragma unroll
  for (int v = 0; v < V; ++v) start[v] = A.starts[(int64_t)tile * A.C + cc + v];
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

  float g[L][V], a[L][V], b[L][V], m[NORM ? L : 1][V], si[GATED ? L : 1][V];
  float sum[V], add[V], back[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sum[v] = add[v] = back[v] = 0.0f;
#pragma unroll
  for (int j = 0; j < L; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      g[j][v] = par.log2_decay(rr[j].get(v), v);
      a[j][v] = exp2_fast(g[j][v]);
      float u = rx[j].get(v);
      if constexpr (GATED) {
        si[j][v] = sigmoid_fast(ri[j].get(v));
        u *= si[j][v];
      }
      if constexpr (NORM) {
        m[j][v] = __builtin_amdgcn_sqrtf(one_minus_square(g[j][v], a[j][v]));
        u *= m[j][v];
      }
      b[j][v] = u;
      sum[v] += g[j][v];
    }
    if (bd.first >> j & 1u) of_sequence(A.S0, j, add);
#pragma unroll
    for (int v = 0; v < V; ++v) add[v] = fmaf(a[j][v], add[v], b[j][v]);
  }
#pragma unroll
  for (int j = L - 1; j >= 0; --j) {
    if (bd.last >> j & 1u) of_sequence(A.dS, j, back);
#pragma unroll
    for (int v = 0; v < V; ++v) back[v] = a[j][v] * (dh[j][v] + back[v]);
  }
  const int order = W - 1 - wave;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s.s_sum[order][lane * V + v] = sum[v];
    s.s_add[order][lane * V + v] = back[v];
    s_add[wave][lane * V + v] = add[v];
  }
  if (lane == 0) {
    s.s_cut[order] = bd.last != 0;
    s_first[wave] = bd.first != 0;
  }
  __syncthreads();
  // the tile ends with a sequence: nothing comes from behind
  const bool alone = tile0 + kTile >= live || (bd.last >> (L - 1) & 1u);  // (wave W - 1 asks)
  float h[V], e[V], dA[V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = start[v];
    dA[v] = db[v] = 0.0f;
  }
  // forwards: the state that the wave begins with
  for (int w = 0; w < wave; ++w) {
    const bool cw = s_first[w] != 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float code = cw ? __uint_as_float(kCut) : decay_code(s.s_sum[W - 1 - w][lane * V + v]);
      h[v] = decayed_onto(code, h[v], s_add[w][lane * V + v]);
    }
  }
  __syncthreads();  // (s_sum becomes the codes)
  s.run(A.chain, k, A.tiles, block, A.C, cc, on, alone, order);
#pragma unroll
  for (int v = 0; v < V; ++v) e[v] = s.s_from[order][lane * V + v];

#pragma unroll
  for (int j = 0; j < L; ++j) {  // b becomes the state before the token
    if (bd.first >> j & 1u) of_sequence(A.S0, j, h);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float add_j = b[j][v];
      b[j][v] = h[v];
      h[v] = fmaf(a[j][v], h[v], add_j);
    }
  }
  const uint32_t row = A.C * (A.out.bf16 ? 2 : 4);
  const __amdgpu_buffer_rsrc_t px = rows_from(A.out.dx, (int64_t)t0 * row),
                               pr = rows_from(A.out.dr, (int64_t)t0 * row),
                               pi = rows_from(A.out.di, (int64_t)t0 * row);
#pragma unroll
  for (int j = L - 1; j >= 0; --j) {
    if (t0 + j < live) {
      if (bd.last >> j & 1u) of_sequence(A.dS, j, e);
      float ox[V], orr[V], oi[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float R = dh[j][v] + e[v];
        e[v] = a[j][v] * R;
        const float x = rx[j].get(v);
        float u = x, du = R;
        if constexpr (GATED) u *= si[j][v];
        float dg = e[v] * b[j][v];
        if constexpr (NORM) {
          du *= m[j][v];
          const float f = a[j][v] * a[j][v] * __builtin_amdgcn_rcpf(m[j][v]) * u * R;
          dg -= m[j][v] > 0.0f ? f : 0.0f;
        }
        ox[v] = du;
        if constexpr (GATED) {
          ox[v] *= si[j][v];
          oi[v] = ox[v] * x * (1.0f - si[j][v]);
        }
        const float r = rr[j].get(v);
        if constexpr (GATE) {
          const float dr = dg * par.neg_a[v] *
                           __builtin_amdgcn_rcpf(1.0f + exp2_fast(-fmaf(r, kLog2e, par.bias2[v])));
          // (where g is -inf the decay is 0, and dg with it)
          dA[v] = fmaf(dg, fmaxf(g[j][v], -3.0e38f), dA[v]);
          db[v] += dr;
          orr[v] = dr;
        } else {
          orr[v] = r > 0.0f ? 0.0f : dg;
        }
      }
      if (on) {
        if (A.out.bf16) {
          Vals<true, V>::store(px, c * 2, j * row, ox);
          Vals<true, V>::store(pr, c * 2, j * row, orr);
          if constexpr (GATED) Vals<true, V>::store(pi, c * 2, j * row, oi);
        } else {
          Vals<false, V>::store(px, c * 4, j * row, ox);
          Vals<false, V>::store(pr, c * 4, j * row, orr);
          if constexpr (GATED) Vals<false, V>::store(pi, c * 4, j * row, oi);
        }
        if (A.out.dS0 && (bd.first >> j & 1u))
          store_state<V>(A.out.dS0, (int64_t)A.q.find(t0 + j) * A.C + c, e, false);
      }
    }
  }
  if constexpr (GATE) {
    if (A.part) {
      __syncthreads();  // s_add and s_from have been read
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s.s_add[wave][lane * V + v] = dA[v];
        s.s_from[wave][lane * V + v] = db[v];
      }
      __syncthreads();
      if (wave == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float x = 0.0f, y = 0.0f;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            x += s.s_add[w][lane * V + v];  // (of log2-decays)
            y += s.s_from[w][lane * V + v];
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

int64_t tiles_of(int64_t T) { return (T + kTile - 1) / kTile; }
size_t part_bytes(int64_t T, int64_t C) {
  return ((size_t)tiles_of(T) * 2 * C * sizeof(float) + 255) / 256 * 256;
}
size_t carries_bytes(int64_t T, int64_t C, bool has_starts) {
  const size_t own = chain_bytes(tiles_of(T), C), scan = scan_workspace_bytes(T, C);
  return has_starts || own > scan ? own : scan;
}
size_t own_starts_bytes(int64_t T, int64_t C) { return (starts_bytes(T, C) + 255) / 256 * 256; }

}  // namespace

bool backward_fits(const Batch& b) {  // 512 threads a workgroup, fewer than 2^32 in a launch
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
  const size_t chain = chain_bytes(tiles_of(b.T), b.C);
  char* const part = base + carries_bytes(b.T, b.C, starts != nullptr);
  Args A;
  A.in = in;
  A.q = Seqs{b.cu, b.N, b.T, b.N > 0 ? b.T / b.N : 0};
  A.C = b.C;
  A.S0 = S0;
  A.dS = dS;
  A.dh = dh;
  A.dh_bf16 = dh_bf16;
  A.out = out;
  A.part = in.A_log && (out.dA_log || out.ddt_bias) ? reinterpret_cast<float*>(part) : nullptr;
  A.tiles = (int)tiles_of(b.T);
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
    if (const hipError_t e = launch_fill(base, chain, s)) return e;
    A.chain = chain_at(base, A.tiles, b.C);
  }
  const Out outs[] = {{dh, dh_bf16}, {out.dx, out.bf16}, {out.dr, out.bf16}, {out.di, out.bf16}};
  const int V = width(in, b.C, outs, 4);
  A.blocks = A.tiles > 0 ? (b.C + 64 * V - 1) / (64 * V) : 0;
  bool empties = out.dS0 != nullptr;
  if (empties && b.cu_host) {
    empties = false;
    for (int n = 0; n < b.N && !empties; ++n) empties = b.cu_host[n + 1] == b.cu_host[n];
  }
  if (!b.cu && b.T > 0) empties = false;
  const int64_t work = (int64_t)A.tiles * A.blocks;
  const int64_t grid = work + (empties ? (b.N < 256 ? b.N : 256) : 0);
  if (grid > 0) {
#define KDA_GR(BF, V_, G, I, N_) \
  backward_kernel<BF, V_, G, I, N_><<<(unsigned)grid, 64 * kWaves, 0, s>>>(A)
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
