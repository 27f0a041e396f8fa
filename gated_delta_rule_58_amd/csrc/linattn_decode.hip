// kda_linattn_recurrent_decode: one token per sequence over a pool of states.
//
// Per (sequence n, head h) with S = pool[slot(n), h] (dk x dv, S[c][j]):
//   S'[c][j] = exp(g) S[c][j] + k_c v_j        o_j = scale sum_c q_c S'[c][j]
//
// HBM-bound: each state is read and written once, everything else is small.
// The new state needs no sum over the old one (there is no delta correction),
// so a thread's elements go out as soon as they have come in; only o waits for
// the sums over the rows.  Every column is independent of the others, so a
// (sequence, head) may be cut into column tiles without any exchange.
#include "kda_device.hpp"
#include "linattn.hpp"

namespace kda {
namespace linattn {
namespace {

// One workgroup: columns [CT * tile, + CT) of one (sequence, head) state.  A
// thread holds 16 bytes (CPT columns) of RPT rows.
template <bool S_BF16, int DK, int DV, int CT, int NTHR>
__global__ void __launch_bounds__(NTHR) decode_kernel(
    Operand q, Operand k, Operand v, Decay gd, void* __restrict__ pool,
    const int32_t* __restrict__ slots, int64_t num_slots, void* __restrict__ o, bool o_bf16,
    int H, int64_t blocks, float scale) {
  constexpr int ES = S_BF16 ? 2 : 4;
  constexpr int CPT = 16 / ES;
  constexpr int NV = CPT / 4;
  constexpr int NCG = CT / CPT;
  constexpr int NRS = NTHR / NCG;
  constexpr int RPT = DK / NRS;
  constexpr int NT = DV / CT;
  constexpr int NW = NTHR / 64;
  static_assert(RPT >= 1 && NRS * RPT == DK && NCG <= 64, "state tile split");

  __shared__ float s_q[DK], s_k[DK];
  __shared__ f32x4 s_red[NW][CT / 4];

  const int t = threadIdx.x;
  const int cg = t % NCG, rs = t / NCG;
  // Workgroups go to the XCDs in turn: each XCD walks a range of the states of its
  // own (256 x 96 states of 64 KB: 554 us, 5.8 TB/s; in the order of the states
  // 581).
  const int64_t per_xcd = gridDim.x >> 3;
  const int64_t id = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if (id >= blocks) return;
  const int64_t pair = id / NT;
  const int tile = id % NT;
  const int64_t n = pair / H;
  const int h = static_cast<int>(pair - n * H);
  const int64_t slot = slots ? static_cast<int64_t>(slots[n]) : n;
  const bool live = slot >= 0 && slot < num_slots;
  // an empty range for a slot outside the pool: loads give 0, stores are dropped
  const char* base = static_cast<const char*>(pool) +
                     (live ? (slot * H + h) * (int64_t)(DK * DV * ES) : 0);
  const __amdgpu_buffer_rsrc_t r = buffer_over(base, live ? DK * DV * ES : 0);
  const int col = tile * CT + cg * CPT;  // first column of the thread

  u32x4 raw[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    raw[i] = __builtin_bit_cast(
        u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, ((rs + NRS * i) * DV + col) * ES, 0, kBufNT));
  const float a = expf(clamp_log_decay(gd.g[gd.per_token ? pair : h]));
  for (int c = t; c < DK; c += NTHR) {
    s_q[c] = load1(q.p, n * q.stride + (int64_t)(h / q.group) * DK + c, q.bf16);
    s_k[c] = load1(k.p, n * k.stride + (int64_t)(h / k.group) * DK + c, k.bf16);
  }
  f32x4 vv[NV], acc[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    vv[u] = load4(v.p, n * v.stride + (int64_t)h * DV + col + 4 * u, v.bf16);
    acc[u] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  barrier_lds();
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int c = rs + NRS * i;
    const float kc = s_k[c], qc = s_q[c];
    f32x4 st[NV];
    if constexpr (S_BF16) {
      const u16x8 b = __builtin_bit_cast(u16x8, raw[i]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        st[u] = f32x4{bf16_bits_to_f32(b[4 * u]), bf16_bits_to_f32(b[4 * u + 1]),
                      bf16_bits_to_f32(b[4 * u + 2]), bf16_bits_to_f32(b[4 * u + 3])};
    } else {
      st[0] = __builtin_bit_cast(f32x4, raw[i]);
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      st[u] = a * st[u] + kc * vv[u];
      acc[u] += qc * st[u];
    }
    u32x4 w;
    if constexpr (S_BF16) {
      u16x8 b;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) b[4 * u + e] = f32_to_bf16_bits(st[u][e]);
      w = __builtin_bit_cast(u32x4, b);
    } else {
      w = __builtin_bit_cast(u32x4, st[0]);
    }
    __builtin_amdgcn_raw_buffer_store_b128(w, r, (c * DV + col) * ES, 0, kBufNT);
  }
  // o: the lanes of a wave that share columns, then the waves
#pragma unroll
  for (int off = NCG; off < 64; off <<= 1)
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[u][e] += __shfl_xor(acc[u][e], off);
  if ((t & 63) < NCG) {
#pragma unroll
    for (int u = 0; u < NV; ++u) s_red[t >> 6][cg * NV + u] = acc[u];
  }
  barrier_lds();
  if (t < CT / 4) {
    f32x4 sum = s_red[0][t];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += s_red[w][t];
    store4(o, pair * DV + tile * CT + 4 * t, live ? scale * sum : f32x4{0.f, 0.f, 0.f, 0.f},
           o_bf16);
  }
}

template <bool S_BF16, int DK, int DV>
hipError_t launch(const Operand& q, const Operand& k, const Operand& v, const Decay& g, void* pool,
                  int64_t num_slots, const int32_t* slots, void* o, bool o_bf16, int N, int H,
                  float scale, hipStream_t s) {
  const int64_t pairs = (int64_t)N * H;
  // Few states: 32 columns a workgroup, so that more CUs take part; many: a whole
  // state each.  us whole / tiled, fp32 at dk x dv = 128 x 128: 96 states 4.9 / 4.5, 256
  // 7.1 / 7.0, 512 12.4 / 13.2, 768 17.7 / 20.3; 128 x 64: 512 7.9 / 7.3, 1,024 14.0 /
  // 12.5; 64 x 128: 512 8.0 / 7.4, 768 10.0 / 11.9; 64 x 64 within 5 % from 96 to 2,048.
  // bf16, where 32 columns are half a cache line: 128 x 128: 64 states 4.4 / 3.9, 96 4.5 /
  // 4.6, 384 6.5 / 8.2; 128 x 64: 96 4.0 / 3.8, 192 4.4 / 4.5, 768 7.0 / 7.9; 64 x 64: 96
  // 3.8 / 3.5, 256 4.2 / 4.2, 768 5.9 / 6.4.
  const bool tiled = pairs < (S_BF16 ? 96 : 512);
  const int64_t blocks = pairs * (tiled ? DV / 32 : 1);
  const dim3 grid(static_cast<unsigned>((blocks + 7) / 8 * 8));
  if (tiled)
    decode_kernel<S_BF16, DK, DV, 32, 256><<<grid, 256, 0, s>>>(q, k, v, g, pool, slots, num_slots,
                                                              o, o_bf16, H, blocks, scale);
  else
    decode_kernel<S_BF16, DK, DV, DV, 512><<<grid, 512, 0, s>>>(q, k, v, g, pool, slots, num_slots,
                                                              o, o_bf16, H, blocks, scale);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_decode(const Operand& q, const Operand& k, const Operand& v, const Decay& g,
                         void* pool, bool state_bf16, int64_t num_slots, const int32_t* slots,
                         void* o, bool o_bf16, int N, int H, int dk, int dv, float scale,
                         hipStream_t s) {
  if (N == 0) return hipSuccess;
#define KDA_LD(SB, DK, DV) \
  return launch<SB, DK, DV>(q, k, v, g, pool, num_slots, slots, o, o_bf16, N, H, scale, s)
#define KDA_LD_D(SB)                           \
  do {                                         \
    if (dk == 128 && dv == 128) KDA_LD(SB, 128, 128); \
    if (dk == 128 && dv == 64) KDA_LD(SB, 128, 64);   \
    if (dk == 64 && dv == 128) KDA_LD(SB, 64, 128);   \
    KDA_LD(SB, 64, 64);                        \
  } while (0)
  if (state_bf16) KDA_LD_D(true);
  KDA_LD_D(false);
#undef KDA_LD_D
#undef KDA_LD
}

}  // namespace linattn
}  // namespace kda
