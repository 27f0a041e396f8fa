// kda_gatedrec_scan: the gated linear recurrence over a packed batch, per channel
//
//   h_t = a_t h_{t-1} + b_t,  a = exp(g),  b = m sigmoid(i) x,  m = sqrt(1 - exp(2 g))
//
// x, r and i are read once and h written once.  A tile is kTile tokens of 64 V channels; a
// wave holds L of the tokens, a lane V channels, all in registers: the gate first, then the
// wave's own decay and contribution (from h = 0), which meet in LDS; the tile's own go to
// the tiles behind it (gatedrec_device.hpp), the state before it comes, and every wave
// runs its tokens again from the state that it begins with.  The factor 1 - a^2 under the
// root is formed from g, so that slow channels keep its digits.
//
// A sequence's border inside a wave's tokens is a bit of a mask (uniform over the wave):
// the state restarts there from the sequence's entry state, which is part of b of that
// token, and is cut off from everything before.
//
// What bounds it: the vector unit, which a value with both gates takes for 40 instructions
// (five of them transcendental), and a tile's 14 us of ticket (0.7 to 1.4), loads (1.9), gate
// (4.2), barrier (2.5) and carry (4.1), of which a CU overlaps two tiles: 120 registers a lane
// and 73.8 KB of LDS a workgroup (61 of them the look back's) hold no more.  bf16: 4,096 x 12,288
// 109 us (3.7 TB/s of what it has to move; a copy reaches 5.2), 32,768 x 4,096 in eight
// sequences 277 us (3.9), 131,072 x 512 without i 136 us (3.0): there 128 tiles of a channel are
// under way at once and the carry takes 9 us of 14.6, the instructions (18 a value) little.  (Two
// of the 40 are the gate's last digits: with a degree less in both polynomials 107, 271, 136 us.)
#include "gatedrec_device.hpp"

namespace kda {
namespace gatedrec {
namespace {

constexpr int kTile = 128;
// L tokens a wave, W waves, the tiles that a look back reaches.  A longer tile has fewer carries,
// a shorter one more workgroups a CU to hide them.  Measured (us, bf16 4,096 x 12,288; 32,768 x
// 4,096 in eight sequences; 131,072 x 512) when 16 x 8 took 110, 276, 134: 8 x 8 120, 321, 288;
// 16 x 16 151, 388, 135; 16 x 4 114, 282, 374.  fp32 8,192 x 4,096 (V = 1): 16 x 8 112,
// 32 x 4 119.
template <int V>
struct Shape {
  static constexpr int L = 16, W = 8, REACH = 60, TILE = L * W;
  static_assert(TILE == kTile && kStartsTokens % L == 0, "starts at waves' tokens");
};

struct Args {
  Inputs in;
  Seqs q;
  int C;
  StatePool st;
  void* h;
  bool h_bf16;
  float* starts;
  Chain chain;
  int tiles, blocks;  // tiles along the tokens, workgroups across the channels
  Split by_blocks;
};

__device__ __forceinline__ int64_t slot_of(const StatePool& st, int n) {
  const int64_t s = st.idx ? (int64_t)__builtin_amdgcn_readfirstlane(st.idx[n]) : n;
  return s >= 0 && s < st.slots ? s : -1;
}

// The final states of sequences without tokens are their entry states.
__device__ void copy_empty(const Args& A, int first, int step) {
  for (int n = first; n < A.q.N; n += step) {
    if (A.q.start(n + 1) > A.q.start(n)) continue;
    const int64_t s = slot_of(A.st, n);
    if (s < 0) continue;
    for (int c = threadIdx.x; c < A.C; c += blockDim.x) {
      const int64_t at = s * A.C + c;
      const float x = A.st.in ? load1(A.st.in, at, A.st.bf16) : 0.0f;
      if (A.st.bf16) static_cast<uint16_t*>(A.st.out)[at] = f32_to_bf16_bits(x);
      else static_cast<float*>(A.st.out)[at] = x;
    }
  }
}

template <bool BF16, int V, bool GATE, bool GATED, bool NORM>
__global__ void __launch_bounds__(64 * Shape<V>::W, 4) scan_kernel(const Args A) {
#pragma clang fp contract(off)  // (the same digits on every path: sums of products are spelt out)
  constexpr int L = Shape<V>::L, W = Shape<V>::W, CB = 64 * V, ES = BF16 ? 2 : 4;
  __shared__ Carry<W, V, Shape<V>::REACH> s;
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
                                        __HIP_MEMORY_SCOPE_AGENT) + 1u;  // it begins at all ones
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(s_ticket);
    if ((uint32_t)id >= (uint32_t)work) return;
  }
  int block;
  const int k = A.by_blocks(id, block);
  const int tile0 = k * kTile, live = A.q.live();
  if (tile0 >= live) return;
  const int t0 = tile0 + wave * L;
  const int c = block * CB + lane * V;
  const bool on = c < A.C;
  const int cc = on ? c : 0;

  Vals<BF16, V> rx[L], rr[L], ri[GATED ? L : 1];
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
  }
  Params<V, GATE> par;
  par.load(A.in, cc);
  Borders bd;
  bd.find(A.q, t0, live - t0 < L ? live - t0 : L);

  float a[L][V], b[L][V], sum[V], add[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sum[v] = add[v] = 0.0f;
#pragma unroll
  for (int j = 0; j < L; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float g = par.log2_decay(rr[j].get(v), v);
      a[j][v] = exp2_fast(g);
      float u = rx[j].get(v);
      if constexpr (GATED) u *= sigmoid_fast(ri[j].get(v));
      if constexpr (NORM) u *= __builtin_amdgcn_sqrtf(one_minus_square(g, a[j][v]));
      b[j][v] = u;
      sum[v] += g;
      add[v] = fmaf(a[j][v], add[v], u);
    }
  // (tokens behind the last sequence are in sum and add too: nothing comes behind them)
  if (bd.first) {  // entry states become part of b, and add begins there
    if (A.st.in) {
      for (uint32_t f = bd.first; f; f &= f - 1) {
        const int k0 = __builtin_ctz(f);
        const int64_t slot = slot_of(A.st, A.q.find(t0 + k0));
        float s0[V] = {};
        if (slot >= 0) load_state<V>(A.st.in, slot * A.C + cc, s0, A.st.bf16);
#pragma unroll
        for (int j = 0; j < L; ++j)
          if (j == k0)
#pragma unroll
            for (int v = 0; v < V; ++v) b[j][v] = fmaf(a[j][v], s0[v], b[j][v]);
      }
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
      if (bd.first >> j & 1u)
#pragma unroll
        for (int v = 0; v < V; ++v) add[v] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) add[v] = fmaf(a[j][v], add[v], b[j][v]);
    }
  }
  float code[V];
#pragma unroll
  for (int v = 0; v < V; ++v) code[v] = decay_code(sum[v]);
  s.set(wave, sum, code, add, bd.first != 0);
  __syncthreads();
  s.run(A.chain, k, A.tiles, block, A.C, cc, on, k == 0 || (bd.first & 1u), wave);

  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = s.from(wave, v);
  if (!on || t0 >= live) return;
  if (A.starts && t0 % kStartsTokens == 0)
#pragma unroll
    for (int v = 0; v < V; ++v) A.starts[(int64_t)(t0 / kStartsTokens) * A.C + c + v] = h[v];
  if (!A.h) return;
  const uint32_t row = A.C * (A.h_bf16 ? 2 : 4);
  const __amdgpu_buffer_rsrc_t ph = rows_from(A.h, (int64_t)t0 * row);
  if (t0 + L <= live && !(bd.first | bd.last)) {
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) b[j][v] = h[v] = fmaf(a[j][v], h[v], b[j][v]);
    if (A.h_bf16) {
#pragma unroll
      for (int j = 0; j < L; ++j) Vals<true, V>::store(ph, c * 2, j * row, b[j]);
    } else {
#pragma unroll
      for (int j = 0; j < L; ++j) Vals<false, V>::store(ph, c * 4, j * row, b[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < L; ++j) {
      if (t0 + j < live) {
        if (bd.first >> j & 1u)
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) b[j][v] = h[v] = fmaf(a[j][v], h[v], b[j][v]);
        if (A.h_bf16) Vals<true, V>::store(ph, c * 2, j * row, h);
        else Vals<false, V>::store(ph, c * 4, j * row, h);
      }
    }
    if (A.st.out) {
      for (uint32_t f = bd.last; f; f &= f - 1) {
        const int k0 = __builtin_ctz(f);
        const int64_t slot = slot_of(A.st, A.q.find(t0 + k0));
        if (slot < 0) continue;
        float x[V];
#pragma unroll
        for (int j = 0; j < L; ++j)
          if (j == k0)
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = b[j][v];
        store_state<V>(A.st.out, slot * A.C + c, x, A.st.bf16);
      }
    }
  }
}

__global__ void __launch_bounds__(256) fill_kernel(u32x4* p, int64_t n) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step)
    p[i] = u32x4{kEmpty, kEmpty, kEmpty, kEmpty};
}

int64_t tiles_of(int64_t T) { return (T + kTile - 1) / kTile; }

}  // namespace

bool scan_fits(const Batch& b) {
  // 512 threads a workgroup, a workgroup for a tile of 64 channels, fewer than 2^32 in a launch
  return tiles_of(b.T) * ((b.C + 63) / 64) < ((int64_t)1 << 23) - 1024;
}
size_t starts_bytes(int64_t T, int64_t C) {
  return (size_t)((T + kStartsTokens - 1) / kStartsTokens) * C * sizeof(float);
}
hipError_t launch_fill(void* ws, size_t bytes, hipStream_t s) {
  const int64_t n = (int64_t)(bytes / 16);
  const int64_t blocks = (n + 1023) / 1024;
  fill_kernel<<<(unsigned)(blocks < 1024 ? blocks : 1024), 256, 0, s>>>(static_cast<u32x4*>(ws), n);
  return hipGetLastError();
}

size_t scan_workspace_bytes(int64_t T, int64_t C) {
  const int64_t tiles = tiles_of(T);
  return tiles > 1 ? chain_bytes(tiles, C) : 0;
}

hipError_t launch_scan(const Inputs& in, const Batch& b, const StatePool& st, void* h, bool h_bf16,
                       float* starts, void* ws, hipStream_t s) {
  Args A;
  A.in = in;
  A.q = Seqs{b.cu, b.N, b.T, b.N > 0 ? b.T / b.N : 0};
  A.C = b.C;
  A.st = st;
  A.h = h;
  A.h_bf16 = h_bf16;
  A.starts = starts;
  A.tiles = (int)tiles_of(b.T);
  A.chain = Chain{};
  if (A.tiles > 1) {
    if (const hipError_t e = launch_fill(ws, scan_workspace_bytes(b.T, b.C), s)) return e;
    A.chain = chain_at(ws, A.tiles, b.C);
  }
  const Out outs[] = {{h, h_bf16}};
  const int V = width(in, b.C, outs, 1);
  A.blocks = (b.C + 64 * V - 1) / (64 * V);
  A.by_blocks = Split(A.blocks);
  // Sequences without tokens: workgroups of their own behind the tiles', unless the host
  // knows that there are none or their states stay where they are.
  bool empties = st.out && st.out != st.in;
  if (empties && b.cu_host) {
    empties = false;
    for (int n = 0; n < b.N && !empties; ++n) empties = b.cu_host[n + 1] == b.cu_host[n];
  }
  if (!b.cu && b.T > 0) empties = false;
  const int64_t work = (int64_t)A.tiles * A.blocks;
  const int64_t grid = work + (empties ? (b.N < 256 ? b.N : 256) : 0);
  if (grid == 0) return hipSuccess;
#define KDA_GR(BF, V_, G, I, N_) \
  scan_kernel<BF, V_, G, I, N_><<<(unsigned)grid, 64 * Shape<V_>::W, 0, s>>>(A)
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
  return hipGetLastError();
}

}  // namespace gatedrec
}  // namespace kda
