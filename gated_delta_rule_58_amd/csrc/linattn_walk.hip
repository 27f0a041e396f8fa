// kda_linattn_chunk_prefill and its backward: the chunked form of
//
//   S_t = exp(g_t) S_{t-1} + b_t c_t^T          out_t = scale S_t^T a_t
//
// with (a, b, c) = (q, k, v).  Per chunk of 64 tokens with entry state S and
// gamma_r = sum_{s <= r} g_s inside the chunk:
//   P[r,s]  = (a_r . b_s) e^(gamma_r - gamma_s)       (s <= r)
//   out     = scale (e^gamma (A S) + P C)
//   S      <- e^gamma_end S + B^T (e^(gamma_end - gamma) C)
// Every factor is at most 1, so nothing overflows however strong the decay is.
//
// The gradients are the same recurrence.  With D_t = dL/dS_t,
//   D_t = scale q_t do_t^T + e^{g_{t+1}} D_{t+1},   dq_t = scale S_t do_t,
//   dk_t = D_t v_t,  dv_t = D_t^T k_t,
// so dq is the walk of (a, b, c) = (do, v, k) with the state S^T, and dv and dk
// are walks from the last token to the first of (k, q, do) with state D and of
// (v, do, q) with state D^T; there token t's decay is g_{t+1} and the state
// carries scale.  One kernel runs the three walks at once (blockIdx.y).
//
// dg: with G[j,i] = P[j,i] dP[j,i] the part of the loss's derivative that token
// i's key and token j's query share (i = before the first token: the initial
// state; j = after the last: the final state), the decay of t lies between i
// and j when i < t <= j, so
//   dg_t = sum_{i < t <= j} G[j,i] = sum_{j >= t} q_j.dq_j - sum_{i >= t} k_i.dk_i
// The pairs i = j cancel in that difference; they are left out of both dots, in
// which they would be the largest terms when the decay is strong.  To keep the
// sums short, <S, dL/dS> at the end of every segment of tokens takes the place
// of the sums over all later tokens (dg_kernel).
//
// Workgroup: 64 columns of c (and so of S and out) of one (sequence, head),
// waves of four kinds, each with a loop of its own over the chunks:
//   state waves   wave w owns columns 16w .. 16w+15 of S in MFMA accumulators.
//                 Per chunk it adds b^T (decayed c) and leaves the new state's
//                 bf16 values in LDS as the operands of the next readout.
//   output waves  wave i owns the chunk's rows 16i .. 16i+15: scores against the
//                 tokens up to its rows, S^T a^T, c^T P^T and the stores.  a goes
//                 from global memory straight to its registers, and the scores
//                 never leave them.
//   copy wave     brings b and c of the chunk after the next into LDS
//                 (three buffers) and touches nothing else, so that its loads
//                 are waited for in the copy wave alone.
//   decay wave    the next chunk's decays.
// S is the only thing handed between the kinds, so one barrier a chunk is
// enough.  (fp32 operands: the state waves copy, because each value is split
// into three, with one buffer and a second barrier.)
// What bounds it: the sequential walk.  A layer of 96 heads gives 192
// workgroups for 256 CUs, each with T / 64 chunks to go through, so the time is
// chunks x the latency of one chunk until HBM is reached.  LDS carries the most
// per chunk (240 to 350 KB a workgroup at 128 B a cycle), which is why the output
// waves split rows and not columns: a and the scores then need no LDS.
//
// Fragments (16x16x32: lane = (lr, lg), lr the row or column, k = 8 lg + e):
//   scores     computed transposed, b a^T: the accumulators of two row tiles of
//              tokens s are, unchanged, the right operand of c^T P^T, with the
//              token order 16(e >> 2) + 4 lg + (e & 3); c^T is read from LDS in
//              that order with the transposing LDS read (four tokens of one
//              column a lane)
//   state      tile t = 2kk + h holds channels 32kk + 8lg + 4h + i in its rows
//              4lg + i, so that the tile pair is the left operand S^T of S^T a^T
//              in natural channel order; b^T is read transposed to match
// LDS rows are 64 or 128 channels; the 16-byte blocks of a row are swizzled so
// that both kinds of read spread over the banks.
//
// Precision: a, b, c in bf16 enter as they are (fp32 ones as three bf16 values
// that add up to them), P as NPP, S as NPS and the decayed c as NPC bf16 values;
// accumulators, decays and the state are fp32, gamma is summed in 64 bits and
// kept as two fp32 values, so that a strong decay early in a chunk costs the
// weak ones behind it no digits.
#include "chunk_common.hpp"
#include "linattn.hpp"

namespace kda {
namespace linattn {

using chunk::ex2;
using chunk::mma_bf16;
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

namespace {

constexpr int C = 64;        // tokens a chunk
constexpr int CT = 64;       // columns a workgroup
constexpr int NTHR = 256;    // threads of the small kernels, and of the state waves
constexpr int kMinSegChunks = 8;   // shortest segment of a cut sequence
constexpr int kBorderChunks = 32;  // segments of dg's sums when sequences are walked whole

// swizzle of the 16-byte block index of a row (rows of 128 / 64 channels)
template <int W>
__device__ __forceinline__ int swz(int row) {
  if constexpr (W == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
  else return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
}

__device__ __forceinline__ f32x8 widen8(bf16x8 x) { return __builtin_convertvector(x, f32x8); }

// x as the sum of NP bf16 values (each the rounding of what is left)
template <int NP>
__device__ __forceinline__ void split8(f32x8 x, bf16x8 (&out)[NP]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    out[p] = __builtin_convertvector(x, bf16x8);
    if (p + 1 < NP) x -= widen8(out[p]);
  }
}

// acc += A B over the planes of A and B that matter (i + j < the larger count)
template <int NA, int NB>
__device__ __forceinline__ void mma_planes(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB],
                                           f32x4& acc) {
  constexpr int NMAX = NA > NB ? NA : NB;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < NMAX) acc = mma_bf16(a[i], b[j], acc);
}

__device__ __forceinline__ s16x4 read_tr(const char* p) {
  typedef __attribute__((address_space(3))) s16x4* P;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
}
// tokens 4lg .. +3 of two token tiles, one column a lane
__device__ __forceinline__ bf16x8 read_tr2(const char* p0, const char* p1) {
  const s16x4 a = read_tr(p0), b = read_tr(p1);
  return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

struct Walk {
  Operand a, b, c, x;       // x: the tensor of the dots (with dots)
  const void* s_in;         // entry states, or null (zeros)
  void* s_out;              // exit states, or null
  int64_t s_row, s_col;     // element strides of the states' channel and column
  int64_t s_elems;          // elements of one state
  const int32_t* in_idx;    // slot per sequence, or null
  const int32_t* out_idx;
  int64_t in_slots, out_slots;
  void* out;                // [T, H, CD]
  float* dots;              // [T, H, 2]: x_t . out_t without the pair (t, t), per column tile
  float* ends;              // states at the segments' ends (dg), slot-major, or null
  float* seg_state;         // cut sequences: each segment's own state, then its entry state
  float* seg_decay;         // cut sequences: each segment's summed log2-decay [slot, H]
  bool in_bf16, out_state_bf16, out_bf16, reverse;
};

struct Args {
  Walk walk[3];
  Decay g;
  const int32_t* cu;   // null: equal lengths
  int N, T_tot, H, eq_len;
  int seg_chunks;      // chunks a segment (cut sequences and the dg borders)
  int nseg;            // segments a workgroup grid covers (1: sequences walked whole)
  float scale;
};

// Token range of sequence n.
__device__ __forceinline__ void seq_range(const Args& A, int n, int& bos, int& len) {
  if (A.cu) {
    const int T = A.T_tot;
    int b = A.cu[n], e = A.cu[n + 1];
    b = b < 0 ? 0 : (b > T ? T : b);
    e = e < b ? b : (e > T ? T : e);
    bos = b;
    len = e - b;
  } else {
    bos = n * A.eq_len;
    len = A.eq_len;
  }
}
// First slot of sequence n's segments: unique, below T_tot / (64 seg_chunks) + N.
__device__ __forceinline__ int64_t seg_slot(const Args& A, int n, int bos) {
  return bos / (C * A.seg_chunks) + n;
}

template <bool WIDE, int KD>
struct Lds {
  static constexpr int NPL = WIDE ? 3 : 1;          // planes of an operand
  static constexpr int NPS = WIDE ? 3 : 2;          // planes of the state
  static constexpr int NBUF = WIDE ? 1 : 3;         // chunks of b and c
  static constexpr int NSB = WIDE ? 1 : 2;          // states
  static constexpr int BB = C * KD * 2;             // one plane of b
  static constexpr int CC = C * CT * 2;             // one plane of c
  static constexpr int SS = KD * CT * 2;            // one plane of the state
  static constexpr int buf = NPL * (BB + CC);
  static constexpr int off_c = NPL * BB;
  static constexpr int off_s = NBUF * buf;
  static constexpr int total = off_s + NSB * NPS * SS;
};
// Waves of a workgroup: state waves 0 .. 3, then (FULL) output waves, then helpers.
template <bool WIDE, bool FULL>
struct Waves {
  static constexpr int out = 4;                        // first output wave
  static constexpr int decay = FULL ? 8 : 4;
  static constexpr int copy = WIDE ? -1 : decay + 1;
  static constexpr int threads = 64 * (decay + (WIDE ? 1 : 2));
};

// The eight values of a block as NP bf16 planes.
template <bool WIDE>
__device__ __forceinline__ void planes_of(const u32x4 (&r)[WIDE ? 2 : 1], bool bf16,
                                          bf16x8 (&pl)[WIDE ? 3 : 1]) {
  if constexpr (WIDE) {
    f32x8 x;
    if (bf16) {
      x = widen8(__builtin_bit_cast(bf16x8, r[0]));
    } else {
      const f32x4 lo = __builtin_bit_cast(f32x4, r[0]), hi = __builtin_bit_cast(f32x4, r[1]);
      x = f32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
    split8<3>(x, pl);
  } else {
    pl[0] = __builtin_bit_cast(bf16x8, r[0]);
  }
}
constexpr int kOutside = 0x7fffff00;  // an offset past every chunk: reads 0, stores nothing
template <bool WIDE>
__device__ __forceinline__ void load_block(__amdgpu_buffer_rsrc_t rsrc, int off, bool bf16,
                                           u32x4 (&r)[WIDE ? 2 : 1]) {
  r[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, 0));
  if constexpr (WIDE) {
    r[1] = u32x4{0, 0, 0, 0};
    if (!bf16)
      r[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off + 16, 0, 0));
  }
}

// One operand's chunk, global memory -> registers -> LDS planes.  Thread t of
// TH moves blocks of 8 channels u = t + TH i: row u / (W / 8), block u % (W / 8).
template <bool WIDE, int W, int TH>
struct Stage {
  static constexpr int NB = C * W / 8 / TH;   // blocks of 8 channels a thread
  u32x4 r[NB][WIDE ? 2 : 1];
  // rsrc covers the chunk's rows of this head; a row past the chunk reads zeros
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rsrc, int stride_bytes, bool bf16,
                                       int rows, bool reverse) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int u = threadIdx.x + TH * i;
      const int row = u / (W / 8), blk = u % (W / 8);
      const int tok = reverse ? rows - 1 - row : row;
      load_block<WIDE>(rsrc, row < rows ? tok * stride_bytes + blk * (bf16 ? 16 : 32) : kOutside,
                       bf16, r[i]);
    }
  }
  __device__ __forceinline__ void write(char* lds, bool bf16) const {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int u = threadIdx.x + TH * i;
      const int row = u / (W / 8), blk = u % (W / 8);
      char* p = lds + row * (W * 2) + ((blk ^ swz<W>(row)) << 4);
      bf16x8 pl[WIDE ? 3 : 1];
      planes_of<WIDE>(r[i], bf16, pl);
#pragma unroll
      for (int k = 0; k < (WIDE ? 3 : 1); ++k)
        *reinterpret_cast<bf16x8*>(p + k * (C * W * 2)) = pl[k];
    }
  }
};

// Buffer over the chunk's rows [tok0, tok0 + rows) of head h (a null tensor is zeros).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const Operand& o, bool bf16,
                                                          int64_t tok0, int rows, int h, int d,
                                                          int col0, int cols) {
  const int es = bf16 ? 2 : 4;
  const char* p = static_cast<const char*>(o.p) +
                  (tok0 * o.stride + (int64_t)(h / o.group) * d + col0) * es;
  return buffer_over(p, rows > 0 && o.p ? (uint32_t)(((rows - 1) * o.stride + cols) * es) : 0);
}

// Copies 64 rows of W channels of bf16 straight into LDS: 1 KiB an instruction,
// lane l writes 16 bytes at 16 l, so the swizzle is in which block a lane asks for.
template <int W>
__device__ __forceinline__ void copy_rows(__amdgpu_buffer_rsrc_t r, char* dst, int stride_bytes,
                                          int rows, bool reverse, int lane) {
  constexpr int BPR = W / 8, RPI = 64 / BPR;  // blocks a row, rows an instruction
#pragma unroll
  for (int u = 0; u < C / RPI; ++u) {
    const int row = u * RPI + lane / BPR;
    const int blk = (lane % BPR) ^ swz<W>(row);
    const int tok = reverse ? rows - 1 - row : row;
    chunk::buf_to_lds16(r, (chunk::lds_ptr_t)(dst + u * 1024),
                        row < rows ? tok * stride_bytes + blk * 16 : kOutside, 0);
  }
}
// waits until at most N vector-memory operations of this wave are outstanding
template <int N>
__device__ __forceinline__ void wait_vm_le() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
  asm volatile("" ::: "memory");
}

// FULL: out, dots and the states; else (no output waves) the segment's own
// state and decay.  DOTS: the backward's walks.
template <bool WIDE, int KD, bool FULL, bool DOTS>
__global__ void __launch_bounds__((Waves<WIDE, FULL>::threads), 1) walk_kernel(Args A) {
  using L = Lds<WIDE, KD>;
  using WV = Waves<WIDE, FULL>;
  constexpr int NPL = L::NPL, NPS = L::NPS;
  constexpr int NPP = WIDE ? 3 : 2, NPC = 3;
  constexpr int KK = KD / 32;   // contraction steps over the channels
  constexpr int NT = KD / 16;   // state tiles a wave
  constexpr int JT = CT / 16;   // column tiles
  __shared__ __attribute__((aligned(16))) char lds[FULL ? L::total : L::off_s];
  __shared__ __attribute__((aligned(16))) float s_gh[2][C], s_gl[2][C], s_row[2][C], s_col[2][C];
  __shared__ float s_end[2];
  __shared__ int s_seq[1];

  const Walk& W = A.walk[blockIdx.y];
  const int tid = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const bool rev = W.reverse;
  const bool a_bf = !WIDE || W.a.bf16, b_bf = !WIDE || W.b.bf16, c_bf = !WIDE || W.c.bf16;

  // ---- blockIdx.x -> (sequence, segment, head, tile): the tiles of a head on one XCD
  const int CD = static_cast<int>(W.s_elems / KD);
  const int ntile = CD / CT;
  const int id = blockIdx.x >> 3;
  const int tile = id % ntile;
  const int64_t pair = (int64_t)(id / ntile) * 8 + (blockIdx.x & 7);
  if (pair >= (int64_t)A.N * A.nseg * A.H) return;
  const int h = static_cast<int>(pair % A.H);
  const int seg = static_cast<int>((pair / A.H) % A.nseg);
  int n = static_cast<int>(pair / A.H / A.nseg);
  if (A.cu) n = chunk::lpt_sequence(A.cu, A.N, A.T_tot, n, s_seq);
  n = __builtin_amdgcn_readfirstlane(n);
  int bos, len;
  seq_range(A, n, bos, len);
  const int nch_all = (len + C - 1) / C;
  int c_lo = 0, c_hi = nch_all;
  if (A.nseg > 1) {
    c_lo = seg * A.seg_chunks;
    c_hi = c_lo + A.seg_chunks < nch_all ? c_lo + A.seg_chunks : nch_all;
    if (c_lo >= c_hi) return;  // nothing here (scan_kernel hands empty sequences' states on)
  }
  const int nch = c_hi - c_lo;
  auto chunk_of = [&](int it) { return rev ? c_hi - 1 - it : c_lo + it; };
  auto rows_in = [&](int c) { return len - c * C < C ? len - c * C : C; };
  // chunk `it` is in buffer it % NBUF
  auto buf_of = [&](int it) -> char* {
    return lds + (L::NBUF == 1 ? 0 : (it % L::NBUF) * L::buf);
  };
  // lane constants of the transposed reads: row of a token tile, its swizzles, piece
  const int tj = 4 * lg + (lr >> 2);
  const int twB = swz<KD>(tj), twC = swz<CT>(tj);
  const int pc = lr & 3;
  // c^T of column tile j, tokens of step ks
  auto read_c = [&](const char* bc, int j, int ks, bf16x8 (&f)[NPL]) {
    const int r0 = 32 * ks + tj, r1 = r0 + 16;
    const int cb = (((2 * j + (pc >> 1)) ^ twC) << 4) + ((pc & 1) << 3);
#pragma unroll
    for (int p = 0; p < NPL; ++p)
      f[p] = read_tr2(bc + p * L::CC + r0 * (CT * 2) + cb, bc + p * L::CC + r1 * (CT * 2) + cb);
  };
  // Every wave passes the same barriers: one a chunk, when the chunk and its
  // entry state are in LDS; with one buffer a second one when it has been read.

  if (w < 4) {
    // =================================================== state waves
    const int64_t slot0 = seg_slot(A, n, bos);
    const int col = tile * CT + 16 * w + lr;  // this lane's column of S
    auto channel = [&](int t) { return 32 * (t >> 1) + 8 * lg + 4 * (t & 1); };
    // a segment's states in the workspace: fp32, tile by tile in this lane's order
    auto seg_at = [&](float* base, int64_t slot) {
      return base + ((slot * A.H + h) * ntile + tile) * (int64_t)(KD * CT) + (w * 64 + lane) * 4;
    };
    f32x4 S[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (FULL) {
      if (A.nseg > 1) {
        const float* p = seg_at(W.seg_state, slot0 + seg);
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] = *reinterpret_cast<const f32x4*>(p + t * (NTHR * 4));
      } else if (W.s_in) {
        const int64_t sl = W.in_idx ? (int64_t)W.in_idx[n] : n;
        if (sl >= 0 && sl < W.in_slots) {
          const int64_t base = (sl * A.H + h) * W.s_elems + col * W.s_col;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              S[t][i] = load1(W.s_in, base + (channel(t) + i) * W.s_row, W.in_bf16);
        }
      }
    }
    // the state's planes, as the left operands of S^T a^T: unit (column tile, kk), 16 bytes a lane
    auto write_state = [&](int sbuf) {
      if constexpr (FULL) {
        char* p = lds + L::off_s + sbuf * (NPS * L::SS) + w * (KK * 1024) + lane * 16;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          const f32x4 t0 = S[2 * kk], t1 = S[2 * kk + 1];
          bf16x8 f[NPS];
          split8<NPS>(f32x8{t0[0], t0[1], t0[2], t0[3], t1[0], t1[1], t1[2], t1[3]}, f);
#pragma unroll
          for (int k = 0; k < NPS; ++k) *reinterpret_cast<bf16x8*>(p + k * L::SS + kk * 1024) = f[k];
        }
      }
    };
    auto dump = [&](int c) {  // S at a segment's end, for dg
      float* p = seg_at(W.ends, slot0 + c / A.seg_chunks);
#pragma unroll
      for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4*>(p + t * (NTHR * 4)) = S[t];
    };
    // fp32 operands: these waves also copy
    Stage<WIDE, KD, NTHR> rb;
    Stage<WIDE, CT, NTHR> rc;
    auto load_chunk = [&](int c) {
      const int rows = rows_in(c);
      const int64_t tok0 = (int64_t)bos + c * C;
      rb.load(rows_of(W.b, b_bf, tok0, rows, h, KD, 0, KD), (int)(W.b.stride * (b_bf ? 2 : 4)), b_bf,
              rows, rev);
      rc.load(rows_of(W.c, c_bf, tok0, rows, h, CD, tile * CT, CT),
              (int)(W.c.stride * (c_bf ? 2 : 4)), c_bf, rows, rev);
    };
    auto write_chunk = [&](char* p) {
      rb.write(p, b_bf);
      rc.write(p + L::off_c, c_bf);
    };
    if (nch > 0) {
      if constexpr (WIDE) {
        load_chunk(chunk_of(0));
        write_chunk(lds);
        if (nch > 1) load_chunk(chunk_of(1));
      }
      write_state(0);
    }
    for (int it = 0; it < nch; ++it) {
      const int c = chunk_of(it);
      const int gb = it & 1;
      const char* bb = buf_of(it);
      const char* bc = bb + L::off_c;
      const bool ends = DOTS && W.ends && ((c + 1) % A.seg_chunks == 0 || c + 1 == nch_all);
      barrier_lds();
      // the backward walks have the state at the segment's end before its last chunk
      if (ends && rev) dump(c);
      // ---- S <- e^gamma_end S + b^T (decayed c)
      const float dec = s_end[gb];
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t] *= dec;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        bf16x8 fc[NPL];
        read_c(bc, w, ks, fc);
        f32x8 x = widen8(fc[0]);
#pragma unroll
        for (int p = 1; p < NPL; ++p) x += widen8(fc[p]);
        const f32x4 e0 = *reinterpret_cast<const f32x4*>(&s_col[gb][32 * ks + 4 * lg]);
        const f32x4 e1 = *reinterpret_cast<const f32x4*>(&s_col[gb][32 * ks + 16 + 4 * lg]);
        x *= f32x8{e0[0], e0[1], e0[2], e0[3], e1[0], e1[1], e1[2], e1[3]};
        bf16x8 fx[NPC];
        split8<NPC>(x, fx);
        const int r0 = 32 * ks + tj, r1 = r0 + 16;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int at = (((4 * (t >> 1) + pc) ^ twB) << 4) + ((t & 1) << 3);
          bf16x8 fb[NPL];
#pragma unroll
          for (int p = 0; p < NPL; ++p)
            fb[p] = read_tr2(bb + p * L::BB + r0 * (KD * 2) + at, bb + p * L::BB + r1 * (KD * 2) + at);
          mma_planes<NPL, NPC>(fb, fx, S[t]);
        }
      }
      if (ends && !rev) dump(c);
      if constexpr (L::NBUF == 1) barrier_lds();
      if (it + 1 < nch) {
        write_state(L::NSB == 1 ? 0 : gb ^ 1);
        if constexpr (WIDE) {
          write_chunk(lds);
          if (it + 2 < nch) load_chunk(chunk_of(it + 2));
        }
      }
    }
    if constexpr (!FULL) {
      float* p = seg_at(W.seg_state, slot0 + seg);
#pragma unroll
      for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4*>(p + t * (NTHR * 4)) = S[t];
    } else if (A.nseg == 1 && W.s_out) {
      const int64_t sl = W.out_idx ? (int64_t)W.out_idx[n] : n;
      if (sl >= 0 && sl < W.out_slots) {
        // walking backwards, the state before the first token has its decay too
        float first = 1.0f;
        if (rev && len > 0)
          first = ex2(clamp_log_decay(A.g.g[A.g.per_token ? (int64_t)bos * A.H + h : h]) *
                      1.4426950408889634f);
        const int64_t base = (sl * A.H + h) * W.s_elems + col * W.s_col;
        const bool sbf = W.out_state_bf16;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t at = base + (channel(t) + i) * W.s_row;
            const float x = S[t][i] * first;
            if (sbf) static_cast<uint16_t*>(W.s_out)[at] = f32_to_bf16_bits(x);
            else static_cast<float*>(W.s_out)[at] = x;
          }
      }
    }
    return;
  }

  if (w == WV::decay) {
    // =================================================== decay wave
    // log2-decay of row `lane` of chunk c (rows past the chunk: 0).  Walking
    // backwards, token t's decay is that of t + 1 and the last token's is 0.
    auto load_decay = [&](int c) -> float {
      const int rows = rows_in(c);
      if (lane >= rows) return 0.f;
      const int t = c * C + (rev ? rows - lane : lane);
      if (t >= len) return 0.f;
      return clamp_log_decay(A.g.g[A.g.per_token ? ((int64_t)bos + t) * A.H + h : h]);
    };
    double sum = 0.0;
    // gamma as two floats, row and column factors
    auto decays = [&](float g, int buf) {
      double x = (double)g * 1.4426950408889634;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_up(x, off);
        if (lane >= off) x += y;
      }
      const double end = __shfl(x, 63);
      const float hi = (float)x;
      s_gh[buf][lane] = hi;
      s_gl[buf][lane] = (float)(x - (double)hi);
      s_row[buf][lane] = ex2(hi) * (rev ? 1.0f : A.scale);
      s_col[buf][lane] = ex2((float)(end - x)) * (rev ? A.scale : 1.0f);
      if (lane == 0) s_end[buf] = ex2((float)end);
      sum += end;
    };
    float g1 = 0.f, g2 = 0.f;  // the next two chunks'
    if (nch > 0) decays(load_decay(chunk_of(0)), 0);
    if (nch > 1) g1 = load_decay(chunk_of(1));
    if (nch > 2) g2 = load_decay(chunk_of(2));
    for (int it = 0; it < nch; ++it) {
      barrier_lds();
      if (it + 1 < nch) {
        const float g = g1;
        g1 = g2;
        if (it + 3 < nch) g2 = load_decay(chunk_of(it + 3));
        decays(g, (it & 1) ^ 1);
      }
      if constexpr (L::NBUF == 1) barrier_lds();
    }
    if (!FULL && lane == 0 && tile == 0)
      W.seg_decay[(seg_slot(A, n, bos) + seg) * A.H + h] = (float)sum;
    return;
  }

  if constexpr (!WIDE) {
    if (w == WV::copy) {
      // ================================================= copy wave
      constexpr int OPS = L::buf / 1024;  // instructions a chunk
      static_assert(L::NBUF == 3 && 2 * OPS < 64, "two chunks in flight");
      const int sb = (int)(W.b.stride * 2), sc = (int)(W.c.stride * 2);
      auto issue = [&](int it) {
        const int c = chunk_of(it);
        const int rows = rows_in(c);
        const int64_t tok0 = (int64_t)bos + c * C;
        char* p = buf_of(it);
        copy_rows<KD>(rows_of(W.b, true, tok0, rows, h, KD, 0, KD), p, sb, rows, rev, lane);
        copy_rows<CT>(rows_of(W.c, true, tok0, rows, h, CD, tile * CT, CT), p + L::off_c, sc, rows,
                      rev, lane);
      };
      if (nch > 0) issue(0);
      if (nch > 1) issue(1);
      for (int it = 0; it < nch; ++it) {
        // chunk `it` has arrived; the one behind it may be on its way
        if (it + 1 < nch) wait_vm_le<OPS>();
        else wait_vm_le<0>();
        chunk::barrier_nofence();
        if (it + 2 < nch) issue(it + 2);  // into the buffer of chunk it - 1, which has been read
      }
      return;
    }
  }

  if constexpr (FULL) {
    // =================================================== output waves
    const int i = w - WV::out;          // row tile
    const int orow = 16 * i + lr;       // this lane's row
    const int swB = swz<KD>(lr);        // row reads: rows 16 x + lr
    const int sa = (int)(W.a.stride * (a_bf ? 2 : 4));
    const bool x_bf = !WIDE || W.x.bf16, o_bf = W.out_bf16;
    float* const dots = DOTS ? W.dots : nullptr;
    u32x4 ra[KK][WIDE ? 2 : 1], ra_next[KK][WIDE ? 2 : 1];
    auto load_a = [&](int c, u32x4 (&r4)[KK][WIDE ? 2 : 1]) {
      const int rows = rows_in(c);
      const __amdgpu_buffer_rsrc_t r = rows_of(W.a, a_bf, (int64_t)bos + c * C, rows, h, KD, 0, KD);
      const int tok = rev ? rows - 1 - orow : orow;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
        load_block<WIDE>(r, orow < rows ? tok * sa + (4 * kk + lg) * (a_bf ? 16 : 32) : kOutside,
                         a_bf, r4[kk]);
    };
    if (nch > 0) load_a(chunk_of(0), ra);
    for (int it = 0; it < nch; ++it) {
      const int c = chunk_of(it);
      const int rows = rows_in(c);
      const int gb = it & 1;
      const char* bb = buf_of(it);
      const char* bc = bb + L::off_c;
      const int64_t tok0 = (int64_t)bos + c * C;
      const int tok = rev ? rows - 1 - orow : orow;
      bf16x8 fa[KK][NPL];
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) planes_of<WIDE>(ra[kk], a_bf, fa[kk]);
      if (it + 1 < nch) load_a(chunk_of(it + 1), ra_next);
      u32x4 xr[JT];  // x of this lane's row, for the dots
      if constexpr (DOTS) {
        if (dots) {
          const __amdgpu_buffer_rsrc_t r = rows_of(W.x, x_bf, tok0, rows, h, CD, tile * CT, CT);
          const int xs = (int)(W.x.stride * (x_bf ? 2 : 4));
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            if (x_bf) {
              const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                  r, orow < rows ? tok * xs + (16 * j + 4 * lg) * 2 : kOutside, 0, 0));
              xr[j] = u32x4{v[0], v[1], 0, 0};
            } else {
              xr[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                  r, orow < rows ? tok * xs + (16 * j + 4 * lg) * 4 : kOutside, 0, 0));
            }
          }
        }
      }
      barrier_lds();
      // ---- scores of row tile i against the tokens 0 .. 16i + 15, transposed
      bf16x8 fp[2][NPP];
      float diag = 0.f;
      const float rh = s_gh[gb][orow], rl = s_gl[gb][orow];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (2 * ks > i) continue;
        f32x4 p0 = {0.f, 0.f, 0.f, 0.f}, p1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          const int blk = ((4 * kk + lg) ^ swB) << 4;
          bf16x8 f0[NPL], f1[NPL];
#pragma unroll
          for (int p = 0; p < NPL; ++p) {
            f0[p] = *reinterpret_cast<const bf16x8*>(bb + p * L::BB + (32 * ks + lr) * (KD * 2) + blk);
            f1[p] = *reinterpret_cast<const bf16x8*>(bb + p * L::BB + (32 * ks + 16 + lr) * (KD * 2) + blk);
          }
          mma_planes<NPL, NPL>(f0, fa[kk], p0);
          mma_planes<NPL, NPL>(f1, fa[kk], p1);  // masked where it lies behind the rows
        }
        f32x8 pv;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int s0 = 32 * ks + 16 * half + 4 * lg;
          const f32x4 sh = *reinterpret_cast<const f32x4*>(&s_gh[gb][s0]);
          const f32x4 sl = *reinterpret_cast<const f32x4*>(&s_gl[gb][s0]);
          const f32x4 v = half ? p1 : p0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = v[e] * A.scale * ex2((rh - sh[e]) + (rl - sl[e]));
            if constexpr (DOTS) {
              if (s0 + e == orow) diag = x;
              pv[4 * half + e] = (dots ? s0 + e < orow : s0 + e <= orow) ? x : 0.f;
            } else {
              pv[4 * half + e] = s0 + e <= orow ? x : 0.f;
            }
          }
        }
        split8<NPP>(pv, fp[ks]);
      }
      // ---- out^T = S^T a^T, the rows' decay, + c^T P^T
      f32x4 acc[JT];
      const float rowf = s_row[gb][orow];
      const char* sp = lds + L::off_s + (L::NSB == 1 ? 0 : gb) * (NPS * L::SS) + lane * 16;
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          bf16x8 fs[NPS];
#pragma unroll
          for (int k = 0; k < NPS; ++k)
            fs[k] = *reinterpret_cast<const bf16x8*>(sp + k * L::SS + (j * KK + kk) * 1024);
          mma_planes<NPS, NPL>(fs, fa[kk], acc[j]);
        }
        acc[j] *= rowf;
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (2 * ks > i) continue;
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          bf16x8 fc[NPL];
          read_c(bc, j, ks, fc);
          mma_planes<NPL, NPP>(fc, fp[ks], acc[j]);
        }
      }
      if constexpr (DOTS) {
        if (dots) {
          // x_t . out_t over the tile's columns, then the pair (t, t)
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            f32x4 xv = __builtin_bit_cast(f32x4, xr[j]);
            if (x_bf) {
              xv = f32x4{__uint_as_float(xr[j][0] << 16), __uint_as_float(xr[j][0] & 0xffff0000u),
                         __uint_as_float(xr[j][1] << 16), __uint_as_float(xr[j][1] & 0xffff0000u)};
            }
            dot += (xv[0] * acc[j][0] + xv[1] * acc[j][1]) + (xv[2] * acc[j][2] + xv[3] * acc[j][3]);
          }
          dot += __shfl_xor(dot, 16);
          dot += __shfl_xor(dot, 32);
          if (lg == 0 && orow < rows) dots[((tok0 + tok) * A.H + h) * 2 + tile] = dot;
          // + P[t,t] c_t: the lane that holds the pair hands it to the others of its row
          const float pd = __shfl(diag, lr + 16 * (lr >> 2));
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            const int cc = 16 * j + 4 * lg;
            const char* cp = bc + orow * (CT * 2) + (((cc >> 3) ^ swz<CT>(orow)) << 4) + ((cc & 7) << 1);
#pragma unroll
            for (int p = 0; p < NPL; ++p) {
              const u16x4 b = *reinterpret_cast<const u16x4*>(cp + p * L::CC);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[j][e] += pd * bf16_bits_to_f32(b[e]);
            }
          }
        }
      }
      if constexpr (L::NBUF == 1) barrier_lds();
      const int64_t ld = (int64_t)A.H * CD;
      const int out_es = o_bf ? 2 : 4;
      const __amdgpu_buffer_rsrc_t ow =
          buffer_over(static_cast<char*>(W.out) + (tok0 * ld + (int64_t)h * CD + tile * CT) * out_es,
                      (uint32_t)(((rows - 1) * ld + CT) * out_es));
      const int off = orow < rows ? (int)((tok * ld + 4 * lg) * out_es) : kOutside;
      if (o_bf) {
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const u16x4 b = {f32_to_bf16_bits(acc[j][0]), f32_to_bf16_bits(acc[j][1]),
                           f32_to_bf16_bits(acc[j][2]), f32_to_bf16_bits(acc[j][3])};
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, b), ow, off + 32 * j, 0, 0);
        }
      } else {
#pragma unroll
        for (int j = 0; j < JT; ++j)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[j]), ow, off + 64 * j,
                                                 0, 0);
      }
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int e = 0; e < (WIDE ? 2 : 1); ++e) ra[kk][e] = ra_next[kk][e];
    }
  }
}

// Cut sequences: the segments' own states become their entry states, and the
// exit state is written.  One workgroup per (sequence, head, tile) and walk;
// the threads own the elements in the walk kernel's order.
template <int KD>
__global__ void __launch_bounds__(NTHR) scan_kernel(Args A) {
  constexpr int NT = KD / 16;
  const Walk& W = A.walk[blockIdx.y];
  const int CD = static_cast<int>(W.s_elems / KD);
  const int ntile = CD / CT;
  const int t = blockIdx.x % NT;          // state tile
  int id = blockIdx.x / NT;
  const int tile = id % ntile;
  id /= ntile;
  const int h = id % A.H, n = id / A.H;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  int bos, len;
  seq_range(A, n, bos, len);
  const int nch = (len + C - 1) / C;
  const int nseg = (nch + A.seg_chunks - 1) / A.seg_chunks;
  const int64_t slot0 = seg_slot(A, n, bos);
  const int ch = 32 * (t >> 1) + 8 * lg + 4 * (t & 1);
  const int col = tile * CT + 16 * w + lr;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (W.s_in) {
    const int64_t sl = W.in_idx ? (int64_t)W.in_idx[n] : n;
    if (sl >= 0 && sl < W.in_slots) {
      const int64_t base = (sl * A.H + h) * W.s_elems + col * W.s_col;
#pragma unroll
      for (int i = 0; i < 4; ++i) S[i] = load1(W.s_in, base + (ch + i) * W.s_row, W.in_bf16);
    }
  }
  auto at = [&](int j) {
    const int64_t slot = slot0 + (W.reverse ? nseg - 1 - j : j);
    return W.seg_state + ((slot * A.H + h) * ntile + tile) * (int64_t)(KD * CT) +
           (w * 64 + lane) * 4 + t * (NTHR * 4);
  };
  f32x4 next = S;
  if (nseg > 0) next = *reinterpret_cast<const f32x4*>(at(0));
  for (int j = 0; j < nseg; ++j) {
    const f32x4 own = next;
    if (j + 1 < nseg) next = *reinterpret_cast<const f32x4*>(at(j + 1));
    const int64_t slot = slot0 + (W.reverse ? nseg - 1 - j : j);
    *reinterpret_cast<f32x4*>(at(j)) = S;
    S = S * ex2(W.seg_decay[slot * A.H + h]) + own;
  }
  if (W.s_out) {
    const int64_t sl = W.out_idx ? (int64_t)W.out_idx[n] : n;
    if (sl >= 0 && sl < W.out_slots) {
      float first = 1.0f;
      if (W.reverse && len > 0)
        first = ex2(clamp_log_decay(A.g.g[A.g.per_token ? (int64_t)bos * A.H + h : h]) *
                    1.4426950408889634f);
      const int64_t base = (sl * A.H + h) * W.s_elems + col * W.s_col;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t e = base + (ch + i) * W.s_row;
        if (W.out_state_bf16) static_cast<uint16_t*>(W.s_out)[e] = f32_to_bf16_bits(S[i] * first);
        else static_cast<float*>(W.s_out)[e] = S[i] * first;
      }
    }
  }
}

// dg of one segment of one (sequence, head): suffix sums of q.dq - k.dk, plus
// <S, dL/dS> at the segment's end.  In 64 bits (a few thousand terms).
__global__ void __launch_bounds__(NTHR) dg_kernel(Args A, const float* dotq, const float* dotk,
                                                  const float* ends_s, const float* ends_d,
                                                  int dk, int dv, bool has_final, float* dg,
                                                  float* dg_part, int nseg_max) {
  __shared__ double s_w[4];
  const int h = blockIdx.x % A.H;
  const int seg = (blockIdx.x / A.H) % nseg_max;
  const int n = blockIdx.x / A.H / nseg_max;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int bos, len;
  seq_range(A, n, bos, len);
  const int nch = (len + C - 1) / C;
  const int nseg = (nch + A.seg_chunks - 1) / A.seg_chunks;
  if (seg >= nseg) return;
  const int64_t slot = seg_slot(A, n, bos) + seg;
  const bool last = seg == nseg - 1;
  // <S, D> over the state, both in the walks' order
  double m = 0.0;
  if (!last || has_final) {
    const int64_t elems = (int64_t)dk * dv;
    const f32x4* a = reinterpret_cast<const f32x4*>(ends_s + (slot * A.H + h) * elems);
    const f32x4* b = reinterpret_cast<const f32x4*>(ends_d + (slot * A.H + h) * elems);
    f32x4 p = {0.f, 0.f, 0.f, 0.f};
    for (int i = tid; i < elems / 4; i += NTHR) p += a[i] * b[i];
    m = ((double)p[0] + (double)p[1]) + ((double)p[2] + (double)p[3]);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m += __shfl_xor(m, off);
  if (lane == 0) s_w[w] = m;
  __syncthreads();
  const double border = (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
  __syncthreads();
  const int t_lo = seg * A.seg_chunks * C;
  const int t_hi = t_lo + A.seg_chunks * C < len ? t_lo + A.seg_chunks * C : len;
  double run = border;
  if (!last) {  // the gradient walks keep dL/dS_t of the token behind the border
    const float g = A.g.g[A.g.per_token ? ((int64_t)bos + t_hi) * A.H + h : h];
    run *= exp((double)clamp_log_decay(g));
  }
  double total = 0.0;
  for (int hi = t_hi; hi > t_lo; hi -= NTHR) {
    const int t = hi - 1 - tid;
    double x = 0.0;
    if (t >= t_lo) {  // one partial dot a column tile of 64 channels
      const int64_t at = (((int64_t)bos + t) * A.H + h) * 2;
      x = (double)dotq[at] - (double)dotk[at];
      if (dk > CT) x += (double)dotq[at + 1] - (double)dotk[at + 1];
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    if (lane == 63) s_w[w] = x;
    __syncthreads();
    double before = run;
    for (int j = 0; j < w; ++j) before += s_w[j];
    x += before;
    run += (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
    __syncthreads();
    if (t >= t_lo) {
      if (A.g.per_token) dg[((int64_t)bos + t) * A.H + h] = (float)x;
      else total += x;
    }
  }
  if (!A.g.per_token) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) total += __shfl_xor(total, off);
    if (lane == 0) s_w[w] = total;
    __syncthreads();
    if (tid == 0) {
      const double s = (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
      dg_part[2 * (slot * A.H + h)] = (float)s;
      dg_part[2 * (slot * A.H + h) + 1] = (float)(s - (double)(float)s);
    }
  }
}

// dg [H] from the segments' sums, in order.  One workgroup per head.
__global__ void __launch_bounds__(64) dg_heads_kernel(Args A, const float* part, float* dg) {
  const int h = blockIdx.x;
  double sum = 0.0;
  for (int n = 0; n < A.N; ++n) {
    int bos, len;
    seq_range(A, n, bos, len);
    const int nch = (len + C - 1) / C;
    const int nseg = (nch + A.seg_chunks - 1) / A.seg_chunks;
    const int64_t slot0 = seg_slot(A, n, bos);
    for (int j = threadIdx.x; j < nseg; j += 64) {
      const int64_t at = 2 * ((slot0 + j) * A.H + h);
      sum += (double)part[at] + (double)part[at + 1];
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  if (threadIdx.x == 0) dg[h] = (float)sum;
}

// dq, dk of shared heads: the sum over the group's heads of the tokens that
// belong to a sequence.  One thread per 4 channels.
__global__ void __launch_bounds__(NTHR) group_sum_kernel(Args A, const float* hq, const float* hk,
                                                         int d, int group, void* dq, void* dk,
                                                         bool bf16) {
  const int Hk = A.H / group;
  const int64_t per = (int64_t)Hk * (d / 4);
  const int64_t i = (int64_t)blockIdx.x * NTHR + threadIdx.x;
  // rows behind the last sequence stay as they are
  int64_t T = A.T_tot;
  if (A.cu) {
    const int e = A.cu[A.N];
    T = e < 0 ? 0 : (e > A.T_tot ? A.T_tot : e);
  }
  if (i >= T * per) return;
  const int64_t t = i / per;
  const int rest = static_cast<int>(i - t * per);
  const int hk_i = rest / (d / 4), c = (rest % (d / 4)) * 4;
  const float* src = blockIdx.y ? hk : hq;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < group; ++j)
    s += *reinterpret_cast<const f32x4*>(src + (t * A.H + hk_i * group + j) * (int64_t)d + c);
  store4(blockIdx.y ? dk : dq, (t * Hk + hk_i) * (int64_t)d + c, s, bf16);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <bool WIDE, int KD, bool FULL, bool DOTS>
hipError_t launch_walk_kd(const Args& A, int walks, hipStream_t s) {
  const int64_t blocks =
      cdiv((int64_t)A.N * A.nseg * A.H, 8) * 8 * (A.walk[0].s_elems / KD / CT);
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  walk_kernel<WIDE, KD, FULL, DOTS><<<dim3((unsigned)blocks, walks),
                                      Waves<WIDE, FULL>::threads, 0, s>>>(A);
  return hipGetLastError();
}
// `walks` walks of one contraction width kd
template <bool DOTS>
hipError_t launch_walk(const Args& A, int walks, bool wide, int kd, bool full, hipStream_t s) {
#define KDA_LW(WD, KDV)                                             \
  return full ? launch_walk_kd<WD, KDV, true, DOTS>(A, walks, s)    \
              : launch_walk_kd<WD, KDV, false, false>(A, walks, s)
  if (wide && kd == 128) KDA_LW(true, 128);
  if (wide) KDA_LW(true, 64);
  if (kd == 128) KDA_LW(false, 128);
  KDA_LW(false, 64);
#undef KDA_LW
}

hipError_t launch_scan(const Args& A, int walks, int kd, hipStream_t s) {
  const int64_t blocks = (int64_t)A.N * A.H * (A.walk[0].s_elems / kd / CT) * (kd / 16);
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks, walks);
  if (kd == 128) scan_kernel<128><<<grid, NTHR, 0, s>>>(A);
  else scan_kernel<64><<<grid, NTHR, 0, s>>>(A);
  return hipGetLastError();
}

// Chunks a segment when sequences are cut, 0 when they are walked whole: with
// `walkers` workgroups a segment, cut when whole sequences are too few for the
// card and long enough; segments then give about two workgroups a CU.
int cut_chunks(int64_t T_tot, int64_t N, int64_t walkers) {
  if (N * walkers >= 192) return 0;
  const int64_t chunks = cdiv(T_tot, C);
  if (chunks < N * 2 * kMinSegChunks) return 0;
  const int64_t sc = cdiv(chunks * walkers, 512);
  return static_cast<int>(sc > kMinSegChunks ? sc : kMinSegChunks);
}

int64_t slots_of(int64_t T_tot, int64_t N, int seg_chunks) {
  return T_tot / (C * (int64_t)seg_chunks) + N;
}

struct Carve {  // 256-byte aligned pieces of a workspace
  char* p;
  size_t used = 0;
  float* take(int64_t floats) {
    float* r = p ? reinterpret_cast<float*>(p + used) : nullptr;
    used += ((size_t)floats * 4 + 255) / 256 * 256;
    return r;
  }
};

struct ForwardWs {
  float *state, *decay;
  size_t bytes;
  ForwardWs(void* ws, int64_t T_tot, int N, int H, int dk, int dv, int seg) {
    Carve c{static_cast<char*>(ws)};
    const int64_t slots = seg ? slots_of(T_tot, N, seg) : 0;
    state = c.take(slots * H * dk * dv);
    decay = c.take(slots * H);
    bytes = c.used;
  }
};

struct BackwardWs {
  float *dotq, *dotk, *ends_s, *ends_d, *dg_part, *hq, *hk, *state[3], *decay[3];
  size_t bytes;
  BackwardWs(void* ws, int64_t T_tot, int N, int H, int Hk, int dk, int dv, int seg, bool cut) {
    Carve c{static_cast<char*>(ws)};
    const int64_t slots = slots_of(T_tot, N, seg), st = slots * H * dk * dv;
    dotq = c.take(T_tot * H * 2);
    dotk = c.take(T_tot * H * 2);
    ends_s = c.take(st);
    ends_d = c.take(st);
    dg_part = c.take(slots * H * 2);
    const int64_t heads = Hk < H ? T_tot * H * dk : 0;
    hq = c.take(heads);
    hk = c.take(heads);
    for (int i = 0; i < 3; ++i) {
      state[i] = c.take(cut ? st : 0);
      decay[i] = c.take(cut ? slots * H : 0);
    }
    bytes = c.used;
  }
};

// longest sequence: from the host copy, or the most it can be
int64_t longest(const Args& A, const int32_t* cu_host) {
  if (!A.cu) return A.eq_len;
  if (!cu_host) return A.T_tot;
  int64_t m = 0;
  for (int n = 0; n < A.N; ++n)
    m = cu_host[n + 1] - cu_host[n] > m ? cu_host[n + 1] - cu_host[n] : m;
  return m;
}

}  // namespace

size_t prefill_workspace_bytes(int64_t T_tot, int N, int H, int dk, int dv) {
  const int seg = cut_chunks(T_tot, N, (int64_t)H * (dv / CT));
  return seg ? ForwardWs(nullptr, T_tot, N, H, dk, dv, seg).bytes : 0;
}

hipError_t launch_prefill(const Problem& p, const Operand& q, const Operand& k, const Operand& v,
                          const StatePool& st, void* o, bool o_bf16, void* ws, size_t ws_bytes,
                          hipStream_t s) {
  Args A{};
  A.g = p.g;
  A.cu = p.cu;
  A.N = p.N;
  A.T_tot = static_cast<int>(p.T_tot);
  A.H = p.H;
  A.eq_len = p.cu ? 0 : static_cast<int>(p.T_tot / p.N);
  A.scale = p.scale;
  A.nseg = 1;
  A.seg_chunks = kBorderChunks;
  Walk& W = A.walk[0];
  W.a = q;
  W.b = k;
  W.c = v;
  W.s_in = st.in;
  W.s_out = st.out;
  W.in_idx = W.out_idx = st.idx;
  W.in_slots = W.out_slots = st.slots;
  W.in_bf16 = W.out_state_bf16 = st.bf16;
  W.s_row = p.dv;
  W.s_col = 1;
  W.s_elems = (int64_t)p.dk * p.dv;
  W.out = o;
  W.out_bf16 = o_bf16;
  const bool wide = !(q.bf16 && k.bf16 && v.bf16);
  const int seg = cut_chunks(p.T_tot, p.N, (int64_t)p.H * (p.dv / CT));
  const ForwardWs f(ws, p.T_tot, p.N, p.H, p.dk, p.dv, seg);
  if (seg && ws && ws_bytes >= f.bytes) {
    A.seg_chunks = seg;
    A.nseg = static_cast<int>(cdiv(cdiv(longest(A, p.cu_host), C), seg));
    if (A.nseg < 1) A.nseg = 1;
    W.seg_state = f.state;
    W.seg_decay = f.decay;
  }
  if (A.nseg > 1) {
    hipError_t e = launch_walk<false>(A, 1, wide, p.dk, false, s);
    if (e == hipSuccess) e = launch_scan(A, 1, p.dk, s);
    if (e != hipSuccess) return e;
  }
  return launch_walk<false>(A, 1, wide, p.dk, true, s);
}

namespace {
int border_chunks(int64_t T_tot, int N, int H, int dk, int dv, bool* cut) {
  const int seg = cut_chunks(T_tot, N, (int64_t)H * (2 * (dk / CT) + dv / CT));
  *cut = seg > 0;
  return seg ? seg : kBorderChunks;
}
}  // namespace

size_t backward_workspace_bytes(int64_t T_tot, int N, int H, int Hk, int dk, int dv) {
  bool cut;
  const int seg = border_chunks(T_tot, N, H, dk, dv, &cut);
  return BackwardWs(nullptr, T_tot, N, H, Hk, dk, dv, seg, cut).bytes;
}

hipError_t launch_backward(const Problem& p, const Operand& q, const Operand& k, const Operand& v,
                           const float* S0, const Operand& d_o, const float* dS, void* dq, void* dk,
                           void* dv, bool grad_bf16, float* dg, float* dS0, void* ws,
                           hipStream_t s) {
  const int DK = p.dk, DV = p.dv, group = p.H / p.Hk;
  bool cut;
  const int seg = border_chunks(p.T_tot, p.N, p.H, DK, DV, &cut);
  const BackwardWs b(ws, p.T_tot, p.N, p.H, p.Hk, DK, DV, seg, cut);
  Args A{};
  A.g = p.g;
  A.cu = p.cu;
  A.N = p.N;
  A.T_tot = static_cast<int>(p.T_tot);
  A.H = p.H;
  A.eq_len = p.cu ? 0 : static_cast<int>(p.T_tot / p.N);
  A.scale = p.scale;
  A.seg_chunks = seg;
  const int64_t max_chunks = cdiv(longest(A, p.cu_host), C);
  const int nseg = static_cast<int>(max_chunks ? cdiv(max_chunks, seg) : 1);
  A.nseg = cut ? nseg : 1;

  Walk wq{}, wk{}, wv{};
  wq.a = d_o; wq.b = v; wq.c = k; wq.x = q;
  wk.a = v; wk.b = d_o; wk.c = q; wk.x = k;
  wv.a = k; wv.b = q; wv.c = d_o;
  wk.reverse = wv.reverse = true;
  Walk* ws3[3] = {&wq, &wk, &wv};
  for (int i = 0; i < 3; ++i) {
    ws3[i]->s_elems = (int64_t)DK * DV;
    ws3[i]->in_slots = ws3[i]->out_slots = p.N;
    ws3[i]->seg_state = b.state[i];
    ws3[i]->seg_decay = b.decay[i];
    ws3[i]->out_bf16 = grad_bf16;
  }
  wq.s_in = S0;
  wk.s_in = wv.s_in = dS;
  wv.s_out = dS0;
  wq.s_row = wk.s_row = 1;      // the transposed states of dq and dk
  wq.s_col = wk.s_col = DV;
  wv.s_row = DV;
  wv.s_col = 1;
  wq.dots = b.dotq;
  wk.dots = b.dotk;
  wq.ends = b.ends_s;
  wk.ends = b.ends_d;
  wq.out = dq;
  wk.out = dk;
  wv.out = dv;
  if (group > 1) {
    wq.out = b.hq;
    wk.out = b.hk;
    wq.out_bf16 = wk.out_bf16 = false;
  }
  const bool wide = !(q.bf16 && k.bf16 && v.bf16 && (d_o.bf16 || !d_o.p));
  A.walk[0] = wq;
  A.walk[1] = wk;
  A.walk[2] = wv;
  Args B = A;  // dk != dv: the walk of dv contracts over another width
  B.walk[0] = wv;
  const bool same = DK == DV;
  for (int phase = A.nseg > 1 ? 0 : 2; phase < 3; ++phase) {
    hipError_t e;
    if (phase == 1) {
      e = launch_scan(A, same ? 3 : 2, DV, s);
      if (e == hipSuccess && !same) e = launch_scan(B, 1, DK, s);
    } else {
      const bool full = phase == 2;
      e = launch_walk<true>(A, same ? 3 : 2, wide, DV, full, s);
      if (e == hipSuccess && !same) e = launch_walk<true>(B, 1, wide, DK, full, s);
    }
    if (e != hipSuccess) return e;
  }
  const int64_t blocks = (int64_t)p.N * nseg * p.H;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  dg_kernel<<<dim3((unsigned)blocks), NTHR, 0, s>>>(A, b.dotq, b.dotk, b.ends_s, b.ends_d, DK, DV,
                                                    dS != nullptr, dg, b.dg_part, nseg);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!A.g.per_token) {
    dg_heads_kernel<<<dim3(p.H), 64, 0, s>>>(A, b.dg_part, dg);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (group > 1 && p.T_tot > 0) {
    const int64_t n = cdiv(p.T_tot * p.Hk * (DK / 4), NTHR);
    if (n > 0x7fffffff) return hipErrorInvalidValue;
    group_sum_kernel<<<dim3((unsigned)n, 2), NTHR, 0, s>>>(A, b.hq, b.hk, DK, group, dq, dk,
                                                         grad_bf16);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace linattn
}  // namespace kda
