// kda_gatedrec_decode: one token per sequence over a pool of states [slots, C].
//
// Per (sequence n, channel c): h = exp(g) S[slot(n), c] + m sigmoid(i) x, which is the
// output and, rounded to the pool's type, the new state.  A value reads and writes its
// state and reads x, r and i: HBM-bound, and by the launch where there are few.  256 x 12,288
// over fp32 states: 11.4 us, 4.4 TB/s; 1,024 x 4,096 13.7 us, 4.9 TB/s; one or two sequences 2.7.
//
// Beside 1 the decay is taken as 1 - d with d kept (gatedrec_device.hpp): a state that
// decays by 1e-5 a step would otherwise drift by 6e-3 of itself from what a scan gives.
#include "gatedrec_device.hpp"

namespace kda {
namespace gatedrec {
namespace {

// A workgroup's channels belong to one sequence, so that rows are uniform.
template <bool BF16, bool SB, int V, bool GATE, bool GATED, bool NORM>
__global__ void __launch_bounds__(256) decode_kernel(
    const Inputs in, int N, int C, void* pool, int64_t num_slots,
    const int32_t* __restrict__ slots, void* __restrict__ h, bool h_bf16) {
  constexpr int ES = BF16 ? 2 : 4, SS = SB ? 2 : 4;
  const int per = (C + 256 * V - 1) / (256 * V);
  const int n = blockIdx.x / per;
  const int c = ((blockIdx.x - n * per) * 256 + threadIdx.x) * V;
  if (c >= C) return;
  Vals<BF16, V> rx, rr, ri;  // on their way before the slot is known
  rr.load(rows_from(in.r.p, n * in.r.stride * ES), c * ES, 0);
  rx.load(rows_from(in.x.p, n * in.x.stride * ES), c * ES, 0);
  if constexpr (GATED) ri.load(rows_from(in.i.p, n * in.i.stride * ES), c * ES, 0);
  Params<V, GATE> par;
  par.load(in, c);
  const int64_t slot = slots ? (int64_t)__builtin_amdgcn_readfirstlane(slots[n]) : n;
  const __amdgpu_buffer_rsrc_t ph = rows_from(h, (int64_t)n * C * (h_bf16 ? 2 : 4));
  float out[V];
  if (slot < 0 || slot >= num_slots) {
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.0f;
  } else {
    const __amdgpu_buffer_rsrc_t ps = rows_from(pool, slot * C * SS);
    Vals<SB, V> st;
    st.load(ps, c * SS, 0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float g = par.log2_decay(rr.get(v), v);
      const float a = exp2_fast(g);
      float u = rx.get(v);
      if constexpr (GATED) u *= sigmoid_fast(ri.get(v));
      if constexpr (NORM) u *= __builtin_amdgcn_sqrtf(one_minus_square(g, a));
      out[v] = decayed_onto(decay_code(g), st.get(v), u);
    }
    Vals<SB, V>::store(ps, c * SS, 0, out);
  }
  if (h_bf16) Vals<true, V>::store(ph, c * 2, 0, out);
  else Vals<false, V>::store(ph, c * 4, 0, out);
}

}  // namespace

hipError_t launch_decode(const Inputs& in, int N, int C, void* pool, bool state_bf16,
                         int64_t num_slots, const int32_t* slots, void* h, bool h_bf16,
                         hipStream_t s) {
  if (N == 0) return hipSuccess;
  const Out outs[] = {{h, h_bf16}, {pool, state_bf16}};
  // Two channels a lane where that is aligned.  bf16, fp32 states, 256 x 12,288 and 1,024 x
  // 4,096: 11.4 and 13.7 us; one channel 13.9 and 17.2, four 13.1 and 15.8 (bf16 states, 1,024 x
  // 8,192: 22.9, 30.0, 27.4): four have half the waves, each with twice the gates in a row.
  const int V = in_pieces_of(2, in, C, outs, 2) ? 2 : 1;
  const int64_t grid = (int64_t)N * ((C + 256 * V - 1) / (256 * V));
#define KDA_GR(BF, SB, V_, G, I, N_)                                                               \
  decode_kernel<BF, SB, V_, G, I, N_><<<(unsigned)grid, 256, 0, s>>>(in, N, C, pool, num_slots, slots, \
                                                                   h, h_bf16)
#define KDA_GR_N(BF, SB, V_, G, I)                    \
  do {                                                \
    if (in.normalize) KDA_GR(BF, SB, V_, G, I, true); \
    else KDA_GR(BF, SB, V_, G, I, false);             \
  } while (0)
#define KDA_GR_I(BF, SB, V_, G)                \
  do {                                         \
    if (in.i.p) KDA_GR_N(BF, SB, V_, G, true); \
    else KDA_GR_N(BF, SB, V_, G, false);       \
  } while (0)
#define KDA_GR_G(BF, SB, V_)                   \
  do {                                         \
    if (in.A_log) KDA_GR_I(BF, SB, V_, true);  \
    else KDA_GR_I(BF, SB, V_, false);          \
  } while (0)
#define KDA_GR_V(BF, SB)              \
  do {                                \
    if (V == 2) KDA_GR_G(BF, SB, 2);  \
    else KDA_GR_G(BF, SB, 1);         \
  } while (0)
  if (in.bf16 && state_bf16) KDA_GR_V(true, true);
  else if (in.bf16) KDA_GR_V(true, false);
  else if (state_bf16) KDA_GR_V(false, true);
  else KDA_GR_V(false, false);
#undef KDA_GR_V
#undef KDA_GR_G
#undef KDA_GR_I
#undef KDA_GR_N
#undef KDA_GR
  return hipGetLastError();
}

}  // namespace gatedrec
}  // namespace kda
