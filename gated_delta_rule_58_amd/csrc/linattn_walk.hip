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
// carries scale.  (blockIdx.y: the walks of dq and dk share a launch.)
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
// waves of four kinds, each kind with a loop of its own over the chunks:
//   state waves   wave w owns 16 columns of S in MFMA accumulators.  Per chunk it
//                 adds b^T (decayed c) and leaves the new state's bf16 values in
//                 LDS as the operands of the next readout.
//   output waves  two row tiles (0 and 3, or 1 and 2: the same work) and two
//                 column tiles each: scores against the tokens up to the rows,
//                 S^T a^T, c^T P^T and the stores.  The scores never leave the
//                 registers.
//   copy waves    bring a, b and c of coming chunks straight into LDS and do
//                 nothing else: under load a wave spends thousands of cycles in
//                 the issue of its loads, which no other wave then waits for.
//   decay wave    the next chunk's decays.
// S is the only thing handed between the kinds, so with two of its buffers one
// barrier a chunk is enough.  The walks with dots keep S as three values, and two
// buffers of those do not fit: there the output waves read S first, and a second
// barrier lets the state waves overwrite it while the scores are made (a second
// buffer in the place of a's, which then goes straight to registers: backward of
// T = 4096 x 96 679 against 545 us).  fp32 operands, three values each: the state
// waves copy, with one buffer and a second barrier.
// What bounds it: a layer of 96 heads gives 192 workgroups for 256 CUs, each with
// T / 64 chunks to go through one after the other, about 4,000 cycles each.  Of
// those LDS is busy for 1,600 (16-byte reads at 256 B a cycle, transposing ones at
// 128, stores at 80 to 128) and the matrix units of a SIMD for 1,400; the rest is
// the chain scores -> decays -> c^T P^T of an output wave.  Measured, dk = dv = 128, bf16:
// T = 4096 x 96 heads 116 us (1.65 us a chunk of a lone workgroup; 3.5 TB/s of what
// has to be read and written), 8 sequences of 32,768 tokens together x 96 831 us
// (4.0 TB/s), one of 131,072 x 16 heads, in segments, 751 us; backward of T = 4096 x
// 96 427 us.  On the way there: scores and readout in the state's waves 302 us, waves
// of two kinds 253, copies and decays in waves of their own 167, one value of S and P
// and eight output columns a store 119.
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
// that add up to them).  The decayed c, of which the fp32 state is made, enters as
// three bf16 values; S and P, of which out is made, as one where out is bf16 (each
// element is then off by at most 2^-8 of itself, as the rounding of out is), as
// two where out is fp32 or the sequence is one chunk, as three where it makes dg
// (launch_walk).  Accumulators, decays and the state are fp32; gamma is summed in 64
// bits and kept as two fp32 values, so that a strong decay early in a chunk costs the
// weak ones behind it no digits.
#include <type_traits>

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
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

namespace {

constexpr int C = 64;        // tokens a chunk
constexpr int CT = 64;       // columns a workgroup
constexpr int NTHR = 256;    // threads of the small kernels, and of the state waves
constexpr int kMinSegChunks = 4;   // shortest segment of a cut sequence
constexpr int64_t kCus = 256;
constexpr int kBorderChunks = 32;  // segments of dg's sums when sequences are walked whole

// Swizzle of the 16-byte block index of a row (rows of 128 / 64 channels).  A read
// of 16 bytes a lane goes through 64 banks in four steps, and a step takes rows 0-3
// and 12-15 of one k block with rows 4-11 of the next: the low bits of rows 0-3 and
// 12-15 are therefore made to differ in bit 0 only, so that a step's 16 blocks are
// all different.  (Low bits row >> 2: every such read took twice as long.)
template <int W>
__device__ __forceinline__ int swz(int row) {
  const int x = (row >> 2) & 3, low = ((x & 1) << 1) ^ ((x >> 1) * 3);  // 0, 2, 3, 1
  if constexpr (W == 128) return ((row & 3) << 2) | low;
  else return (((row >> 1) & 1) << 2) | low;
}

__device__ __forceinline__ f32x8 widen8(bf16x8 x) { return __builtin_convertvector(x, f32x8); }

// x as the sum of NP bf16 values (each the rounding of what is left).  Two
// values a conversion: the empty asm keeps the pair in one register, or the
// compiler converts each value by itself to widen it again.
template <int NP>
__device__ __forceinline__ void split8(f32x8 x, bf16x8 (&out)[NP]) {
  u32x4 w[NP];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a = x[2 * k], b = x[2 * k + 1];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      uint32_t u = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
      if (p + 1 < NP) {
        asm("" : "+v"(u));
        a -= __uint_as_float(u << 16);
        b -= __uint_as_float(u & 0xffff0000u);
      }
      w[p][k] = u;
    }
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) out[p] = __builtin_bit_cast(bf16x8, w[p]);
}

// Calls f(i, j) for the products of plane i of A and plane j of B that matter
// (i + j < the larger count), the smallest first.  The products of several
// accumulators go inside f: an MFMA that waits for the one before it takes more
// than twice as long as one that does not (44 against 20 clocks here).
template <int NA, int NB, class F>
__device__ __forceinline__ void for_planes(F f) {
  constexpr int NMAX = NA > NB ? NA : NB;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < NMAX) f(i, j);
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

// x of another lane of the wave, by data-parallel move (0 where there is none)
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Inclusive sums over the 64 lanes.  Moves between registers and no LDS
// permutes: under the other waves' LDS traffic a chain of permutes took longer
// than the rest of the chunk's work.
__device__ __forceinline__ double wave_scan(double x) {
  x += moved<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8: within 16 lanes
  x += moved<0x112, 0xf>(x);
  x += moved<0x114, 0xf>(x);
  x += moved<0x118, 0xf>(x);
  x += moved<0x142, 0xa>(x);  // lane 15 of a row to the next row (rows 1, 3)
  x += moved<0x143, 0xc>(x);  // lane 31 to rows 2, 3
  return x;
}
__device__ __forceinline__ double of_lane(double x, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, l);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// sum of x over the lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ __forceinline__ float sum_rows(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
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
  float* dots;              // [H, T, 4]: x_t . out_t without the pair (t, t), per 32 columns
  float* ends;              // states at the segments' ends (dg), slot-major, or null
  float* seg_state;         // cut sequences: each segment's own state, then its entry state
  float* seg_decay;         // cut sequences: each segment's summed log2-decay [slot, H]
  bool in_bf16, out_state_bf16, out_bf16, reverse;
};

__host__ __device__ __forceinline__ int heads_per_xcd(int H) { return H < 16 ? 1 : H / 8; }

struct Args {
  Walk walk[3];
  int first;           // walk of blockIdx.y = 0
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

// The sequence whose segments begin at or below `slot` (the last such): each step asks
// for 64 sequences at once, one a lane.
__device__ __forceinline__ int seq_of_slot(const Args& A, int64_t slot) {
  int lo = 0, cnt = A.N;  // it is one of lo .. lo + cnt - 1
  while (cnt > 1) {
    const int step = (cnt + 63) / 64, off = (int)(threadIdx.x & 63) * step;
    bool le = false;
    if (off < cnt) {
      int bos, len;
      seq_range(A, lo + off, bos, len);
      le = seg_slot(A, lo + off, bos) <= slot;
    }
    const int k = __popcll(__ballot(le));
    const int at = k > 0 ? (k - 1) * step : 0;
    lo += at;
    cnt = cnt - at < step ? cnt - at : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// PS: bf16 values of a state's element (see walk)
template <bool WIDE, int KD, bool FULL, bool DOTS, int PS>
struct Lds {
  static constexpr int NPL = WIDE ? 3 : 1;          // planes of an operand
  static constexpr int NBUF = WIDE ? 1 : PS == 1 ? 3 : 2;  // chunks of a, b and c
  static constexpr int NSB = PS == 3 ? 1 : 2;       // states
  static constexpr int AB = C * KD * 2;             // one plane of a or b
  static constexpr int CC = C * CT * 2;             // one plane of c
  static constexpr int SS = KD * CT * 2;            // one plane of the state
  static constexpr int off_b = FULL && !WIDE ? AB : 0;  // (fp32: a goes straight to registers)
  static constexpr int off_c = off_b + NPL * AB;
  static constexpr int off_x = off_c + NPL * CC;    // x of the dots (fp32: straight to registers)
  static constexpr int buf = off_x + (DOTS && !WIDE ? CC : 0);
  static constexpr int off_s = NBUF * buf;
  static constexpr int total = off_s + NSB * PS * SS;
};
// Decays of a chunk (of two, in turn), with gamma_i the sum up to row tile i's
// first row; behind everything else in LDS.
struct alignas(16) Decays {
  float gh[2][C], gl[2][C];  // gamma as two floats
  float row[2][C];           // e^(gamma_r - gamma_i), r in tile i
  float tok[2][3][C];        // scale e^(gamma_i - gamma_s), tile i = 1 ..
  float col[2][C];           // e^(gamma_end - gamma_s)
  float tile[2][4];          // e^gamma_i
  float end[2];              // e^gamma_end
};
// Waves of a workgroup: state waves 0 .. 3, output waves 4 .. 7, then the helpers.
template <bool WIDE, bool FULL>
struct Waves {
  static constexpr int decay = FULL ? 8 : 4;
  static constexpr int copy = decay + 1;  // and copy + 1
  static constexpr int threads = 64 * (WIDE ? decay : copy + 2);
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
// Rows past a chunk's end need no test: their offsets lie behind the buffer's
// range (or, walking backwards, below 0, which is behind it as an unsigned
// offset), where loads read 0 and stores are dropped.  A test here becomes a
// branch around each load, and the loads then wait for each other.
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
      const int u = threadIdx.x % TH + TH * i;
      const int row = u / (W / 8), blk = u % (W / 8);
      const int tok = reverse ? rows - 1 - row : row;
      load_block<WIDE>(rsrc, tok * stride_bytes + blk * (bf16 ? 16 : 32), bf16, r[i]);
    }
  }
  __device__ __forceinline__ void write(char* lds, bool bf16) const {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int u = threadIdx.x % TH + TH * i;
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

// The rows of one operand (or of out) that a workgroup walks over: one head's
// `cols` channels from col0 of every token of its sequence.  Everything here is
// the same for all lanes; the division by the group is done once.
struct Rows {
  const char* base;   // first token of the sequence
  int64_t chunk;      // bytes a chunk
  int stride, width;  // bytes between tokens, bytes of a row
  __device__ __forceinline__ Rows(const Operand& o, bool bf16, int bos, int h, int d, int col0,
                                  int cols) {
    const int es = bf16 ? 2 : 4;
    stride = (int)o.stride * es;
    chunk = (int64_t)C * stride;
    width = o.p ? cols * es : 0;  // a null tensor: nothing in range, which is zeros
    base = static_cast<const char*>(o.p) +
           (bos * o.stride + (int64_t)(h / o.group) * d + col0) * es;
  }
  // Buffer over `rows` rows of chunk c (none: everything reads zeros).
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t of(int c, int rows) const {
    const int n = rows > 0 && width > 0 ? (rows - 1) * stride + width : 0;
    return buffer_over(base + c * chunk, (uint32_t)n);
  }
};

// Copies rows [row0, row0 + 64 / PARTS) of 64 rows of W channels of bf16 straight
// into LDS: 1 KiB an instruction, lane l writes 16 bytes at 16 l, so the swizzle
// is in which block a lane asks for.
template <int W, int PARTS>
__device__ __forceinline__ void copy_rows(__amdgpu_buffer_rsrc_t r, char* dst, int stride_bytes,
                                          int rows, bool reverse, int lane, int row0) {
  constexpr int BPR = W / 8, RPI = 64 / BPR;  // blocks a row, rows an instruction
#pragma unroll
  for (int u = 0; u < C / RPI / PARTS; ++u) {
    const int row = row0 + u * RPI + lane / BPR;
    const int blk = (lane % BPR) ^ swz<W>(row);
    const int tok = reverse ? rows - 1 - row : row;
    chunk::buf_to_lds16(r, (chunk::lds_ptr_t)(dst + row0 * (W * 2) + u * 1024),
                        tok * stride_bytes + blk * 16, 0);
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

// FULL: out, dots and the states; else (no output waves) the segment's own state
// and decay.  DOTS: the backward's walks.  PL: bf16 values that stand for an
// element of S and P in the products for out.
template <bool WIDE, int KD, bool FULL, bool DOTS, int PL>
constexpr int lds_bytes() {
  using L = Lds<WIDE, KD, FULL, DOTS, PL>;
  return (FULL ? L::total : L::off_s) + (int)sizeof(Decays);
}
// What a workgroup walks: column tile `tile` of head h of segment seg of sequence n.
struct Place {
  int n, bos, len, seg, h, tile;
};
// False: nothing (the grid is rounded up).  Every thread of the workgroup calls it.
//
// Workgroups go to the XCDs in turn; an XCD gets hb = H / 8 consecutive heads (of 8 hb in
// the list of all segments' heads) with their tiles, which are neighbours in a token's row
// and share q and k where those are shared.  It makes little difference; us like this /
// with every eighth head on an XCD: 131,072 tokens x 16 heads (2 of q/k) 728 / 745, eight
// sequences of 4,096 x 96 790 / 779, T = 4096 x 96 123 / 122, backward of T = 4096 x 64
// 314 / 318.
template <int KD>
__device__ __forceinline__ bool locate(const Args& A, const Walk& W, int block, int* s_seq,
                                       Place& at) {
  const int ntile = static_cast<int>(W.s_elems / KD) / CT;
  const int hb = heads_per_xcd(A.H);
  int id = block >> 3;
  at.tile = id % ntile;
  id /= ntile;
  id = (id / hb * 8 + (block & 7)) * hb + id % hb;
  at.h = id % A.H;
  id /= A.H;
  at.seg = id % A.nseg;
  int n = id / A.nseg;
  if (n >= A.N) return false;
  if (A.cu) n = chunk::lpt_sequence(A.cu, A.N, A.T_tot, n, s_seq);
  at.n = __builtin_amdgcn_readfirstlane(n);
  seq_range(A, at.n, at.bos, at.len);
  return true;
}

template <bool WIDE, int KD, bool FULL, bool DOTS, int PL>
__device__ __forceinline__ void walk(const Args& A, const Walk& W, const Place& at, char* lds) {
  using L = Lds<WIDE, KD, FULL, DOTS, PL>;
  using WV = Waves<WIDE, FULL>;
  constexpr int NPL = L::NPL, NBUF = L::NBUF;
  constexpr int NPS = PL, NPP = PL, NPC = 3;
  constexpr int KK = KD / 32;   // contraction steps over the channels
  constexpr int NT = KD / 16;   // state tiles a wave
  Decays& D = *reinterpret_cast<Decays*>(lds + (FULL ? L::total : L::off_s));
  auto& s_gh = D.gh;
  auto& s_gl = D.gl;
  auto& s_row = D.row;
  auto& s_tok = D.tok;
  auto& s_col = D.col;
  auto& s_tile = D.tile;
  auto& s_end = D.end;
  const int tid = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const bool rev = W.reverse;
  const bool a_bf = !WIDE || W.a.bf16, b_bf = !WIDE || W.b.bf16, c_bf = !WIDE || W.c.bf16;

  const int n = at.n, bos = at.bos, len = at.len, seg = at.seg, h = at.h, tile = at.tile;
  const int CD = static_cast<int>(W.s_elems / KD);
  const int ntile = CD / CT;
  const int nch_all = (len + C - 1) / C;
  int c_lo = 0, c_hi = nch_all;
  if (A.nseg > 1) {
    c_lo = seg * A.seg_chunks;
    c_hi = c_lo + A.seg_chunks < nch_all ? c_lo + A.seg_chunks : nch_all;
    if (c_lo >= c_hi) return;  // nothing here (scan_kernel hands empty sequences' states on)
  }
  const int nch = c_hi - c_lo;
  auto chunk_of = [&](int it) { return rev ? c_hi - 1 - it : c_lo + it; };
  // rows of the walk's `it`-th chunk; none behind the last one, where the loads
  // run all the same and read nothing (a branch around them would make every
  // wait one for all of them)
  auto rows_in = [&](int it) {
    const int left = len - chunk_of(it) * C;
    return it >= nch ? 0 : left < C ? left : C;
  };
  const int tj = 4 * lg + (lr >> 2);  // transposed reads: row of a token tile, piece
  const int pc = lr & 3;
  // Column tile 2 jh + j of the workgroup's columns: its column m is column
  // 32 jh + 8 (m >> 2) + 4 j + (m & 3), so that a lane's rows 4 lg + i of a tile
  // pair are eight consecutive columns of out.
  auto column_of = [](int tl, int m) { return 32 * (tl >> 1) + 8 * (m >> 2) + 4 * (tl & 1) + (m & 3); };
  // the lane's part of the reads of c^T, column tile tl
  auto lane_c = [&](int tl) {
    return L::off_c + tj * (CT * 2) + (((4 * (tl >> 1) + pc) ^ swz<CT>(tj)) << 4) + ((tl & 1) << 3);
  };
  auto read_c = [&](const char* bc, int ks, bf16x8 (&f)[NPL]) {
#pragma unroll
    for (int p = 0; p < NPL; ++p)
      f[p] = read_tr2(bc + p * L::CC + 32 * ks * (CT * 2), bc + p * L::CC + (32 * ks + 16) * (CT * 2));
  };
  // All kinds pass the same barriers: one a chunk, when the chunk and its entry
  // state are in LDS; with one buffer a second one when it has been read.

  // ---- decays: the decay wave's (fp32 operands: state wave 3's)
  // Log-decay of row `lane` of a chunk as loaded, by every state wave (a load
  // that only one of them makes would make the others' waits inexact).  Walking
  // backwards, token t's decay is that of t + 1.
  const float* const g0 = A.g.g + (A.g.per_token ? (int64_t)bos * A.H + h : h);
  const int g_step = A.g.per_token ? A.H * 4 : 0;
  auto load_decay = [&](int it) -> float {
    const int c = chunk_of(it), rows = rows_in(it);
    const int last = len - c * C < rows + 1 ? rows - 1 : rows;  // last token a lane may ask for
    const __amdgpu_buffer_rsrc_t r =
        buffer_over(reinterpret_cast<const char*>(g0) + (int64_t)c * C * g_step,
                    rows > 0 ? (uint32_t)(last * g_step + 4) : 0);
    return __uint_as_float(
        __builtin_amdgcn_raw_buffer_load_b32(r, (rev ? rows - lane : lane) * g_step, 0, 0));
  };
  double sum = 0.0;
  // of chunk `it` from its loaded g; rows past its end and, walking backwards, the
  // last token have none
  auto decays = [&](int it, float g, int buf) {
    const int c = chunk_of(it), rows = rows_in(it);
    const int t = c * C + (rev ? rows - lane : lane);
    g = lane < rows && t < len ? clamp_log_decay(g) : 0.f;
    const double x = wave_scan((double)g * 1.4426950408889634);
    const double end = of_lane(x, 63);
    const double e1 = of_lane(x, 15), e2 = of_lane(x, 31), e3 = of_lane(x, 47);
    const float hi = (float)x;
    // walking backwards the state carries scale, so the readout does not
    s_col[buf][lane] = ex2((float)(end - x)) * (rev ? A.scale : 1.0f);
    if constexpr (FULL) {
      s_gh[buf][lane] = hi;
      s_gl[buf][lane] = (float)(x - (double)hi);
      const double mine = lane < 16 ? 0.0 : lane < 32 ? e1 : lane < 48 ? e2 : e3;
      s_row[buf][lane] = ex2((float)(x - mine));
      s_tok[buf][0][lane] = A.scale * ex2((float)(e1 - x));  // read for s before the tile only
      s_tok[buf][1][lane] = A.scale * ex2((float)(e2 - x));
      s_tok[buf][2][lane] = A.scale * ex2((float)(e3 - x));
      if ((lane & 15) == 0) s_tile[buf][lane >> 4] = ex2((float)mine) * (rev ? 1.0f : A.scale);
    }
    if (lane == 0) s_end[buf] = ex2((float)end);
    sum += end;
  };

  if (w < 4) {
    // =================================================== state waves
    const int64_t slot0 = seg_slot(A, n, bos);
    const int col = tile * CT + column_of(w, lr);  // this lane's column of S
    auto channel = [&](int t) { return 32 * (t >> 1) + 8 * lg + 4 * (t & 1); };
    // a segment's states in the workspace: fp32, tile by tile in this lane's order
    auto seg_at = [&](float* base, int64_t slot) {
      return base + ((slot * A.H + h) * ntile + tile) * (int64_t)(KD * CT) + (w * 64 + lane) * 4;
    };
    // fp32 operands: b and c of the next chunk on their way
    Stage<WIDE, KD, NTHR> rb[1];
    Stage<WIDE, CT, NTHR> rc[1];
    const Rows b_rows(W.b, b_bf, bos, h, KD, 0, KD), c_rows(W.c, c_bf, bos, h, CD, tile * CT, CT);
    auto load_chunk = [&](int it, auto& sb, auto& sc) {
      const int c = chunk_of(it), rows = rows_in(it);
      sb.load(b_rows.of(c, rows), b_rows.stride, b_bf, rows, rev);
      sc.load(c_rows.of(c, rows), c_rows.stride, c_bf, rows, rev);
    };
    auto write_chunk = [&](char* p, const auto& sb, const auto& sc) {
      sb.write(p + L::off_b, b_bf);
      sc.write(p + L::off_c, c_bf);
    };
    float g_next = 0.f;  // of the next chunk
    if constexpr (WIDE) {
      if (nch > 0) {
        const float g_first = load_decay(0);
        load_chunk(0, rb[0], rc[0]);
        g_next = load_decay(1);
        if (w == 3) decays(0, g_first, 0);
      }
    }
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
    // the lane's part of the transposed reads
    const int my_c = lane_c(w);
    int my_b[KK];
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
      my_b[kk] = L::off_b + tj * (KD * 2) + (((4 * kk + pc) ^ swz<KD>(tj)) << 4);

    if (nch > 0) {
      if constexpr (WIDE) {
        write_chunk(lds, rb[0], rc[0]);
        load_chunk(1, rb[0], rc[0]);
      }
      write_state(0);
    }
    int slot = 0;  // it % NBUF
    for (int it = 0; it < nch; ++it) {
      const int c = chunk_of(it);
      const int gb = it & 1;
      const char* const buf = lds + slot * L::buf;
      const bool ends = DOTS && W.ends && ((c + 1) % A.seg_chunks == 0 || c + 1 == nch_all);
      barrier_lds();
      // the backward walks have the state at the segment's end before its last chunk
      if (ends && rev) dump(c);
      // ---- S <- e^gamma_end S + b^T (decayed c), G tiles at a time: the fragments
      // of b^T of the next tiles are read while these are multiplied.
      constexpr int G = WIDE ? 2 : 4;
      bf16x8 fc[2][NPL], fb[2][G][NPL];
      auto read_b = [&](int grp, bf16x8 (&f)[G][NPL]) {  // grp = (step ks, tiles)
#pragma unroll
        for (int x = 0; x < G; ++x) {
          const int idx = grp * G + x, t = idx % NT, r0 = 32 * (idx / NT);
#pragma unroll
          for (int p = 0; p < NPL; ++p) {
            const char* q = buf + my_b[t >> 1] + (p * L::AB + r0 * (KD * 2) + 8 * (t & 1));
            f[x][p] = read_tr2(q, q + 16 * (KD * 2));
          }
        }
      };
      f32x4 ec[4];
      const float dec = s_end[gb];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        read_c(buf + my_c, ks, fc[ks]);
        ec[2 * ks] = *reinterpret_cast<const f32x4*>(&s_col[gb][32 * ks + 4 * lg]);
        ec[2 * ks + 1] = *reinterpret_cast<const f32x4*>(&s_col[gb][32 * ks + 16 + 4 * lg]);
      }
      read_b(0, fb[0]);
      if constexpr (WIDE) {
        if (w == 3 && it + 1 < nch) decays(it + 1, g_next, gb ^ 1);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t] *= dec;
      bf16x8 fx[2][NPC];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        f32x8 x = widen8(fc[ks][0]);
#pragma unroll
        for (int p = 1; p < NPL; ++p) x += widen8(fc[ks][p]);
        const f32x4 e0 = ec[2 * ks], e1 = ec[2 * ks + 1];
        x *= f32x8{e0[0], e0[1], e0[2], e0[3], e1[0], e1[1], e1[2], e1[3]};
        split8<NPC>(x, fx[ks]);
      }
#pragma unroll
      for (int grp = 0; grp < 2 * NT / G; ++grp) {
        if (grp + 1 < 2 * NT / G) read_b(grp + 1, fb[(grp + 1) & 1]);
          for_planes<NPL, NPC>([&](int i, int j) {
#pragma unroll
          for (int x = 0; x < G; ++x) {
            f32x4& acc = S[(grp * G + x) % NT];
            acc = mma_bf16(fb[grp & 1][x][i], fx[grp * G / NT][j], acc);
          }
        });
        }
      if (ends && !rev) dump(c);
      if constexpr (WIDE || (FULL && L::NSB == 1)) barrier_lds();
      write_state(L::NSB == 2 ? gb ^ 1 : 0);
      if constexpr (WIDE) {
        write_chunk(lds, rb[0], rc[0]);
        g_next = load_decay(it + 2);
        load_chunk(it + 2, rb[0], rc[0]);
      }
      slot = slot + 1 == NBUF ? 0 : slot + 1;
    }

    if constexpr (!FULL) {
      float* p = seg_at(W.seg_state, slot0 + seg);
#pragma unroll
      for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4*>(p + t * (NTHR * 4)) = S[t];
      if (WIDE && w == 3 && lane == 0 && tile == 0)
        W.seg_decay[(slot0 + seg) * A.H + h] = (float)sum;
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

  if constexpr (!WIDE) {
    if (w == WV::decay) {
      // ================================================= decay wave
      float g1 = load_decay(0), g2 = load_decay(1);
      if (nch > 0) decays(0, g1, 0);
      g1 = g2;
      g2 = load_decay(2);
      for (int it = 0; it < nch; ++it) {
        barrier_lds();
        if constexpr (FULL && L::NSB == 1) barrier_lds();
        const float g = g1;
        g1 = g2;
        g2 = load_decay(it + 3);
        if (it + 1 < nch) decays(it + 1, g, (it & 1) ^ 1);
      }
      if (!FULL && lane == 0 && tile == 0)
        W.seg_decay[(seg_slot(A, n, bos) + seg) * A.H + h] = (float)sum;
      return;
    }
    if (w >= WV::copy) {
      // ================================================= copy waves: a and b, half of c each
      const int half = w - WV::copy;
      constexpr int OPS = (FULL ? L::AB : L::AB / 2) / 1024 + L::CC / 2048 * (DOTS ? 2 : 1);
      static_assert(2 * OPS < 64, "two chunks in flight");
      const Operand& ab = FULL && half == 0 ? W.a : W.b;
      const Rows ab_rows(ab, true, bos, h, KD, 0, KD), c_rows(W.c, true, bos, h, CD, tile * CT, CT);
      const Rows x_rows(W.x, true, bos, h, CD, tile * CT, CT);
      auto issue = [&](int it, int slot) {
        const int c = chunk_of(it), rows = rows_in(it);
        char* p = lds + slot * L::buf;
        if constexpr (FULL)
          copy_rows<KD, 1>(ab_rows.of(c, rows), p + half * L::off_b, ab_rows.stride, rows, rev, lane, 0);
        else
          copy_rows<KD, 2>(ab_rows.of(c, rows), p + L::off_b, ab_rows.stride, rows, rev, lane, 32 * half);
        copy_rows<CT, 2>(c_rows.of(c, rows), p + L::off_c, c_rows.stride, rows, rev, lane, 32 * half);
        if constexpr (DOTS)
          copy_rows<CT, 2>(x_rows.of(c, rows), p + L::off_x, x_rows.stride, rows, rev, lane, 32 * half);
      };
      // chunks it .. it + NBUF - 2 are asked for before barrier `it`; the buffer of
      // chunk it - 1 is free behind it
      if (nch > 0) issue(0, 0);
      if (NBUF == 3 && nch > 0) issue(1, 1);
      int slot = NBUF - 1;  // (it + NBUF - 1) % NBUF
      for (int it = 0; it < nch; ++it) {
        wait_vm_le<(NBUF - 2) * OPS>();  // chunk `it` has arrived
        chunk::barrier_nofence();
        issue(it + NBUF - 1, slot);      // (none behind the last chunk: reads zeros)
        if constexpr (FULL && L::NSB == 1) chunk::barrier_nofence();
        slot = slot + 1 == NBUF ? 0 : slot + 1;
      }
      wait_vm_le<0>();
      return;
    }
  }

  if constexpr (FULL) {
    // =================================================== output waves
    // row tiles T0 and T1 (fixed at compile time: no branches inside, so that the
    // loads of one product can be placed among the arithmetic of another),
    // column tiles 2 jh and 2 jh + 1
    // the longest chain of a chunk is theirs: before the state waves of their SIMDs
    // (without: 8 sequences x 96 heads 882 against 865 us on one card, T = 4096 126
    // against 120)
    __builtin_amdgcn_s_setprio(2);
    const int jh = w & 1;
    const bool x_bf = !WIDE || W.x.bf16, o_bf = W.out_bf16;
    const Rows a_rows(W.a, a_bf, bos, h, KD, 0, KD);
    const Rows x_rows(W.x, x_bf, bos, h, CD, tile * CT + 32 * jh, 32);
    Operand out_op;
    out_op.p = W.out;
    out_op.stride = (int64_t)A.H * CD;
    const Rows o_rows(out_op, o_bf, bos, h, CD, tile * CT + 32 * jh, 32);
    int my_k[KK], my_c[2];              // the lane's part of the reads of b and of c^T
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) my_k[kk] = lr * (KD * 2) + (((4 * kk + lg) ^ swz<KD>(lr)) << 4);
#pragma unroll
    for (int j = 0; j < 2; ++j) my_c[j] = lane_c(2 * jh + j);

    auto output = [&](auto half_of) {
      constexpr int T[2] = {decltype(half_of)::value, 3 - decltype(half_of)::value};
      constexpr int NU = T[1] + 1;      // token tiles up to the rows
      u32x4 ra[2][KK][WIDE ? 2 : 1], ra_next[2][KK][WIDE ? 2 : 1];
      auto load_a = [&](int it, u32x4 (&r4)[2][KK][WIDE ? 2 : 1]) {
        const int rows = rows_in(it);
        const __amdgpu_buffer_rsrc_t r = a_rows.of(chunk_of(it), rows);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = 16 * T[t] + lr;
          const int tok = rev ? rows - 1 - row : row;
#pragma unroll
          for (int kk = 0; kk < KK; ++kk)
            load_block<WIDE>(r, tok * a_rows.stride + (4 * kk + lg) * (a_bf ? 16 : 32), a_bf,
                             r4[t][kk]);
        }
      };
      if (nch > 0) {
        if constexpr (WIDE) load_a(0, ra);
      }
      int slot = 0;  // it % NBUF
      for (int it = 0; it < nch; ++it) {
        const int c = chunk_of(it);
        const int rows = rows_in(it);
        const int gb = it & 1;
        const char* const ba = lds + slot * L::buf;
        const char* const bb = ba + L::off_b;
        const char* const sp =
            lds + L::off_s + (L::NSB == 2 ? gb : 0) * (NPS * L::SS) + jh * (2 * KK * 1024) + lane * 16;
        bf16x8 fa[2][KK][NPL];
        if constexpr (WIDE) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) planes_of<WIDE>(ra[t][kk], a_bf, fa[t][kk]);
          load_a(it + 1, ra_next);
        }
        u32x4 xr[2][2];  // x of this lane's rows, for the dots
        if constexpr (DOTS && WIDE) {
          const __amdgpu_buffer_rsrc_t r = x_rows.of(c, rows);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int row = 16 * T[t] + lr;
            const int tok = rev ? rows - 1 - row : row;
            for (int j = 0; j < 2; ++j) {  // eight bf16, or four of eight fp32
              xr[t][j] = u32x4{0, 0, 0, 0};
              if (j == 0 || !x_bf)
                xr[t][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                    r, tok * x_rows.stride + (x_bf ? 16 * lg : 32 * lg + 16 * j), 0, 0));
            }
          }
        }
        barrier_lds();

        // ---- scores against token tile u, transposed
        bf16x8 fk[NU][KK][NPL], fs[2][KK][NPS], fc[2][2][NPL], fp[2][2][NPP];
        f32x4 p[2][NU], acc[2][2];
        auto read_k = [&](int u) {
#pragma unroll
          for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int q = 0; q < NPL; ++q)
              fk[u][kk][q] = *reinterpret_cast<const bf16x8*>(
                  bb + my_k[kk] + (q * L::AB + 16 * u * (KD * 2)));
        };
        // token tiles u0 and u0 + 1
        auto mul_k = [&](int u0) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = u0; u < u0 + 2; ++u)
              if (u <= T[t]) p[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kk = 0; kk < KK; ++kk)
            for_planes<NPL, NPL>([&](int i, int j) {
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int u = u0; u < u0 + 2; ++u)
                  if (u <= T[t])  // not behind the rows
                    p[t][u] = mma_bf16(fk[u][kk][i], fa[t][kk][j], p[t][u]);
            });
        };
        auto read_s = [&](int kk0, int kk1) {
#pragma unroll
          for (int kk = kk0; kk < kk1; ++kk)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int k = 0; k < NPS; ++k)
                fs[j][kk][k] =
                    *reinterpret_cast<const bf16x8*>(sp + k * L::SS + (j * KK + kk) * 1024);
        };
        auto mul_s = [&](int kk0, int kk1) {
#pragma unroll
          for (int kk = kk0; kk < kk1; ++kk)
            for_planes<NPS, NPL>([&](int i, int k) {
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  acc[t][j] = mma_bf16(fs[j][kk][i], fa[t][kk][k], acc[t][j]);
            });
        };
        // Decays of the scores.  Tokens before row tile i: e^(gamma_r - gamma_i)
        // e^(gamma_i - gamma_s), both at most 1; tokens of the tile itself: the
        // difference of the sums, masked.
        float rowf[2], tilef[2], rh[2], rl[2];
        bf16x8 fd[2][NPP];  // with dots: the pairs (t, t), which the dots leave out
        f32x4 tokf[2][3], sh[2], sl[2];
        auto read_w = [&](int t) {
          const int row = 16 * T[t] + lr, own = 16 * T[t] + 4 * lg;
          rowf[t] = s_row[gb][row];
          tilef[t] = s_tile[gb][T[t]];
          rh[t] = s_gh[gb][row];
          rl[t] = s_gl[gb][row];
          sh[t] = *reinterpret_cast<const f32x4*>(&s_gh[gb][own]);
          sl[t] = *reinterpret_cast<const f32x4*>(&s_gl[gb][own]);
#pragma unroll
          for (int u = 0; u < T[t]; ++u)
            tokf[t][u] = *reinterpret_cast<const f32x4*>(&s_tok[gb][T[t] - 1][16 * u + 4 * lg]);
        };
        auto weigh = [&](int t) {
          const int row = 16 * T[t] + lr;
#pragma unroll
          for (int u = 0; u <= T[t]; ++u) {
            const int s0 = 16 * u + 4 * lg;
            if (u < T[t]) {
              p[t][u] *= tokf[t][u < 3 ? u : 0] * rowf[t];
            } else {
              f32x8 own = {};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float x = p[t][u][e] * A.scale * ex2((rh[t] - sh[t][e]) + (rl[t] - sl[t][e]));
                if constexpr (DOTS) {
                  own[4 * (u & 1) + e] = s0 + e == row ? x : 0.f;
                  p[t][u][e] = s0 + e < row ? x : 0.f;
                } else {
                  p[t][u][e] = s0 + e <= row ? x : 0.f;
                }
              }
              if constexpr (DOTS) split8<NPP>(own, fd[t]);
            }
          }
#pragma unroll
          for (int ks = 0; 2 * ks <= T[t]; ++ks) {
            const f32x4 lo = p[t][2 * ks];
            f32x4 hi = {0.f, 0.f, 0.f, 0.f};
            if (2 * ks + 1 <= T[t]) hi = p[t][2 * ks + 1];
            split8<NPP>(f32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}, fp[t][ks]);
          }
        };
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (!WIDE) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
              fa[t][kk][0] = *reinterpret_cast<const bf16x8*>(ba + my_k[kk] + 16 * T[t] * (KD * 2));
        }
        auto read_c2 = [&] {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) read_c(ba + my_c[j], ks, fc[j][ks]);
        };
        if constexpr (PL == 1) {
          read_k(0);
          read_k(1);
          read_k(2);
          if constexpr (NU == 4) read_k(3);
          read_s(0, KK);
          read_w(0);
          read_w(1);
          mul_k(0);
          mul_k(2);
          read_c2();
          weigh(0);
          weigh(1);
          mul_s(0, KK);
        } else if constexpr (L::NSB == 1 && !WIDE) {
          // the products with the state first: behind the second barrier the state
          // waves overwrite it
          read_s(0, KK / 2);
          mul_s(0, KK / 2);
          read_s(KK / 2, KK);
          mul_s(KK / 2, KK);
          barrier_lds();
          read_k(0);
          read_k(1);
          read_w(0);
          read_w(1);
          mul_k(0);
          read_k(2);
          if constexpr (NU == 4) read_k(3);
          weigh(0);
          mul_k(2);
          read_c2();
          weigh(1);
        } else {
          // one group of operands after the other: all at once they do not fit the registers
          read_k(0);
          read_k(1);
          read_w(0);
          read_w(1);
          mul_k(0);
          read_k(2);
          if constexpr (NU == 4) read_k(3);
          weigh(0);
          mul_k(2);
          read_s(0, KK / 2);
          weigh(1);
          mul_s(0, KK / 2);
          read_s(KK / 2, KK);
          read_c2();
          mul_s(KK / 2, KK);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float f = rowf[t] * tilef[t];
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[t][j] *= f;
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          for_planes<NPL, NPP>([&](int i, int k) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (2 * ks <= T[t]) acc[t][j] = mma_bf16(fc[j][ks][i], fp[t][ks][k], acc[t][j]);
          });
        if constexpr (DOTS) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int row = 16 * T[t] + lr;
            const int tok = rev ? rows - 1 - row : row;
            // x_t . out_t over the wave's columns
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              f32x4 xv = __builtin_bit_cast(f32x4, xr[t][j]);
              if (x_bf) {
                if constexpr (!WIDE)
                  xr[t][0] = *reinterpret_cast<const u32x4*>(
                      ba + L::off_x + row * (CT * 2) + (((4 * jh + lg) ^ swz<CT>(row)) << 4));
                const uint32_t x0 = xr[t][0][2 * j], x1 = xr[t][0][2 * j + 1];
                xv = f32x4{__uint_as_float(x0 << 16), __uint_as_float(x0 & 0xffff0000u),
                           __uint_as_float(x1 << 16), __uint_as_float(x1 & 0xffff0000u)};
              }
              dot += (xv[0] * acc[t][j][0] + xv[1] * acc[t][j][1]) +
                     (xv[2] * acc[t][j][2] + xv[3] * acc[t][j][3]);
            }
            dot = sum_rows(dot);
            if (lg == 0 && row < rows)
              W.dots[((int64_t)h * A.T_tot + bos + c * C + tok) * 4 + 2 * tile + jh] = dot;
          }
          for_planes<NPL, NPP>([&](int i, int k) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                acc[t][j] = mma_bf16(fc[j][T[t] >> 1][i], fd[t][k], acc[t][j]);
          });
        }
        if constexpr (WIDE) barrier_lds();
        // the next a before the stores: loads behind them would be waited for with them
        if constexpr (WIDE) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                ra[t][kk][e] = ra_next[t][kk][e];
                hold(ra[t][kk][e]);
              }
        }
        slot = slot + 1 == NBUF ? 0 : slot + 1;
        const __amdgpu_buffer_rsrc_t ow = o_rows.of(c, rows);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = 16 * T[t] + lr;
          const int off = (rev ? rows - 1 - row : row) * o_rows.stride + 8 * lg * (o_bf ? 2 : 4);
          if (o_bf) {
            u16x8 b;
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = f32_to_bf16_bits(acc[t][e >> 2][e & 3]);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, b), ow, off, 0, 0);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[t][j]), ow,
                                                     off + 16 * j, 0, 0);
          }
        }
      }
    };
    if (w & 2) output(std::integral_constant<int, 1>{});
    else output(std::integral_constant<int, 0>{});
  }
}

// S and P as one bf16 value each in the products for out, as two for a sequence of one
// chunk (kByLength; see launch_walk).
constexpr int kByLength = 0;
template <bool WIDE, int KD, bool FULL, bool DOTS, int PL>
constexpr int lds_of() {
  if constexpr (PL != kByLength) {
    return lds_bytes<WIDE, KD, FULL, DOTS, PL>();
  } else {
    constexpr int a = lds_bytes<WIDE, KD, FULL, DOTS, 1>(), b = lds_bytes<WIDE, KD, FULL, DOTS, 2>();
    return a > b ? a : b;
  }
}
template <bool WIDE, int KD, bool FULL, bool DOTS, int PL>
__device__ __forceinline__ void walk_block(const Args& A, const Walk& W, int block, int* s_seq,
                                           char* lds) {
  Place at;
  if (!locate<KD>(A, W, block, s_seq, at)) return;
  if constexpr (PL != kByLength) walk<WIDE, KD, FULL, DOTS, PL>(A, W, at, lds);
  else if (at.len <= C) walk<WIDE, KD, FULL, DOTS, 2>(A, W, at, lds);
  else walk<WIDE, KD, FULL, DOTS, 1>(A, W, at, lds);
}

template <bool WIDE, int KD, bool FULL, bool DOTS, int PL>
__global__ void __launch_bounds__((Waves<WIDE, FULL>::threads), 1) walk_kernel(Args A) {
  __shared__ __attribute__((aligned(16))) char lds[lds_of<WIDE, KD, FULL, DOTS, PL>()];
  __shared__ int s_seq;
  walk_block<WIDE, KD, FULL, DOTS, PL>(A, A.walk[A.first + blockIdx.y], blockIdx.x, &s_seq, lds);
}

// The three walks of the backward in one launch, at one workgroup a CU: dq, the
// first v1 workgroups of dv, dk, the rest of dv.  n_qk, n_v: workgroups of dq's and
// of dv's walk; they and v1 are multiples of 8.
template <int DK, int DV, int PLV>
__global__ void __launch_bounds__((Waves<false, true>::threads), 1)
    gradient_kernel(Args A, int n_qk, int v1) {
  constexpr int a = lds_of<false, DV, true, true, 3>(), b = lds_of<false, DK, true, false, PLV>();
  __shared__ __attribute__((aligned(16))) char lds[a > b ? a : b];
  __shared__ int s_seq;
  const int block = blockIdx.x;
  if (block < n_qk || (block >= n_qk + v1 && block < 2 * n_qk + v1)) {
    const int y = block >= n_qk;
    walk_block<false, DV, true, true, 3>(A, A.walk[y], block - (y ? n_qk + v1 : 0), &s_seq, lds);
  } else {
    walk_block<false, DK, true, false, PLV>(A, A.walk[2],
                                            block - (block < n_qk + v1 ? 1 : 2) * n_qk, &s_seq, lds);
  }
}

// Cut sequences: the segments' own states become their entry states, and the
// exit state is written.  One workgroup per (sequence, head, tile) and walk;
// the threads own the elements in the walk kernel's order.
template <int KD>
__global__ void __launch_bounds__(NTHR) scan_kernel(Args A) {
  constexpr int NT = KD / 16;
  const Walk& W = A.walk[A.first + blockIdx.y];
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
  const int col = tile * CT + 32 * (w >> 1) + 8 * (lr >> 2) + 4 * (w & 1) + (lr & 3);  // as in the walk
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
  // AHEAD segments' loads at a time: the chain itself is short
  constexpr int AHEAD = 8;
  for (int j0 = 0; j0 < nseg; j0 += AHEAD) {
    f32x4 own[AHEAD];
    float decay[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int j = j0 + i < nseg ? j0 + i : nseg - 1;
      own[i] = *reinterpret_cast<const f32x4*>(at(j));
      decay[i] = W.seg_decay[(slot0 + (W.reverse ? nseg - 1 - j : j)) * A.H + h];
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (j0 + i < nseg) {
        *reinterpret_cast<f32x4*>(at(j0 + i)) = S;
        S = S * ex2(decay[i]) + own[i];
      }
    }
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
// <S, dL/dS> at the segment's end.  In 64 bits (a few thousand terms).  One workgroup
// per segment slot and head, so that the grid follows the tokens and the sequences and
// not their product, whatever the host knows of the lengths.  512 lanes:
// a segment of 2,048 tokens is few trips to memory (the whole backward of T = 4096
// x 96 with 256 / 512 / 1,024: 436 / 431 / 433 us; of T = 128 x 4, 12.9 / 13.6 / 14.6).
constexpr int DGT = 512;
__global__ void __launch_bounds__(DGT) dg_kernel(Args A, const float* dotq, const float* dotk,
                                                  const float* ends_s, const float* ends_d,
                                                  int dk, int dv, bool has_final, float* dg,
                                                  float* dg_part) {
  __shared__ double s_w[DGT / 64];
  const int h = blockIdx.x % A.H;
  const int64_t slot = blockIdx.x / A.H;
  const int n = seq_of_slot(A, slot);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int bos, len;
  seq_range(A, n, bos, len);
  const int nch = (len + C - 1) / C;
  const int nseg = (nch + A.seg_chunks - 1) / A.seg_chunks;
  const int seg = static_cast<int>(slot - seg_slot(A, n, bos));
  if (seg < 0 || seg >= nseg) {  // no segment's slot
    if (!A.g.per_token && tid == 0)
      dg_part[2 * (slot * A.H + h)] = dg_part[2 * (slot * A.H + h) + 1] = 0.f;
    return;
  }
  const bool last = seg == nseg - 1;
  // <S, D> over the state, both in the walks' order
  double m = 0.0;
  if (!last || has_final) {
    const int64_t elems = (int64_t)dk * dv;
    const f32x4* a = reinterpret_cast<const f32x4*>(ends_s + (slot * A.H + h) * elems);
    const f32x4* b = reinterpret_cast<const f32x4*>(ends_d + (slot * A.H + h) * elems);
    f32x4 p = {0.f, 0.f, 0.f, 0.f};
    for (int i = tid; i < elems / 4; i += DGT) p += a[i] * b[i];
    m = ((double)p[0] + (double)p[1]) + ((double)p[2] + (double)p[3]);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m += __shfl_xor(m, off);
  if (lane == 0) s_w[w] = m;
  __syncthreads();
  auto all_waves = [&] {
    double x = 0.0;
#pragma unroll
    for (int j = 0; j < DGT / 64; ++j) x += s_w[j];
    return x;
  };
  const double border = all_waves();
  __syncthreads();
  const int t_lo = seg * A.seg_chunks * C;
  const int t_hi = t_lo + A.seg_chunks * C < len ? t_lo + A.seg_chunks * C : len;
  double run = border;
  if (!last) {  // the gradient walks keep dL/dS_t of the token behind the border
    const float g = A.g.g[A.g.per_token ? ((int64_t)bos + t_hi) * A.H + h : h];
    run *= exp((double)clamp_log_decay(g));
  }
  double total = 0.0;
  for (int hi = t_hi; hi > t_lo; hi -= DGT) {
    const int t = hi - 1 - tid;
    double x = 0.0;
    if (t >= t_lo) {  // one partial dot per 32 channels
      const int64_t at = ((int64_t)h * A.T_tot + bos + t) * 4;
      const f32x4 a = *reinterpret_cast<const f32x4*>(dotq + at);
      const f32x4 b = *reinterpret_cast<const f32x4*>(dotk + at);
      x = ((double)a[0] - (double)b[0]) + ((double)a[1] - (double)b[1]);
      if (dk > CT) x += ((double)a[2] - (double)b[2]) + ((double)a[3] - (double)b[3]);
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
    run += all_waves();
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
      const double s = all_waves();
      dg_part[2 * (slot * A.H + h)] = (float)s;
      dg_part[2 * (slot * A.H + h) + 1] = (float)(s - (double)(float)s);
    }
  }
}

// dg [H] from the slots' sums, in order.  One workgroup per head.
__global__ void __launch_bounds__(64) dg_heads_kernel(Args A, const float* part, int64_t slots,
                                                      float* dg) {
  const int h = blockIdx.x;
  double sum = 0.0;
  for (int64_t j = threadIdx.x; j < slots; j += 64) {
    const int64_t at = 2 * (j * A.H + h);
    sum += (double)part[at] + (double)part[at + 1];
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
  // rows of no sequence stay as they are
  int64_t t0 = 0, t1 = A.T_tot;
  if (A.cu) {
    const int b = A.cu[0], e = A.cu[A.N];
    t0 = b < 0 ? 0 : b;
    t1 = e < 0 ? 0 : (e > A.T_tot ? A.T_tot : e);
  }
  const int64_t t = i / per;
  if (t < t0 || t >= t1) return;
  const int rest = static_cast<int>(i - t * per);
  const int hk_i = rest / (d / 4), c = (rest % (d / 4)) * 4;
  const float* src = blockIdx.y ? hk : hq;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < group; ++j)
    s += *reinterpret_cast<const f32x4*>(src + (t * A.H + hk_i * group + j) * (int64_t)d + c);
  store4(blockIdx.y ? dk : dq, (t * Hk + hk_i) * (int64_t)d + c, s, bf16);
}

// Zeros from row *end on of up to four tensors of T rows.  blockIdx.y: the tensor.
struct Cleared {
  char* p[kMaxCleared];
  int64_t row_bytes[kMaxCleared];
};
__global__ void __launch_bounds__(NTHR) zero_rows_kernel(const int32_t* end, int T, Cleared t) {
  char* const p = t.p[blockIdx.y];
  const int64_t row = t.row_bytes[blockIdx.y];
  const int e = *end;
  const int64_t from = (e < 0 ? 0 : e > T ? T : e) * row, to = T * row;
  const int64_t at = (int64_t)blockIdx.x * NTHR + threadIdx.x, step = (int64_t)gridDim.x * NTHR;
  if (row % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    for (int64_t i = from + at * 16; i < to; i += step * 16)
      *reinterpret_cast<u32x4*>(p + i) = u32x4{0, 0, 0, 0};
  } else {
    for (int64_t i = from + at * 4; i < to; i += step * 4) *reinterpret_cast<uint32_t*>(p + i) = 0;
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// workgroups of a walk of contraction width kd (see walk)
int64_t walk_blocks(const Args& A, int kd) {
  const int hb = heads_per_xcd(A.H);
  return cdiv((int64_t)A.N * A.nseg * A.H, 8 * hb) * 8 * hb * (A.walk[0].s_elems / kd / CT);
}
// workgroups of scan_kernel and group_sum_kernel
int64_t scan_blocks(const Args& A, int kd) {
  return (int64_t)A.N * A.H * (A.walk[0].s_elems / kd / CT) * (kd / 16);
}
int64_t group_sum_blocks(const Problem& p) { return cdiv(p.T_tot * p.Hk * (p.dk / 4), NTHR); }

// A launch holds fewer than 2^32 work items an axis.
bool fits(int64_t blocks, int threads) { return blocks * threads < (int64_t(1) << 32); }

template <bool WIDE, int KD, bool FULL, bool DOTS, int PL>
hipError_t launch_walk_kd(const Args& A, int walks, hipStream_t s) {
  const int64_t blocks = walk_blocks(A, KD);
  walk_kernel<WIDE, KD, FULL, DOTS, PL><<<dim3((unsigned)blocks, walks),
                                          Waves<WIDE, FULL>::threads, 0, s>>>(A);
  return hipGetLastError();
}
// `walks` walks of one contraction width kd from A.first on.  S and P enter the products for out as
//   three values  with dots: dg is a small difference of their sums, and for one
//                 decay a head a sum of those; with two values it was up to 3e-5 off
//   two           out is fp32, or bf16 and the sequence has at most one chunk of tokens
//                 (kByLength), where the few roundings do not average out and the cost
//                 is small (H = 96: T = 64 7.6 against 7.5 us, 512 packed sequences of 64
//                 with states 3,010 against 2,850; T = 256 14.3 against 13.3, T = 4096
//                 146 against 124).  By the sequence, not by the call: a sequence gets
//                 the same digits whatever it is packed with
//   one           out is bf16: off by 2.3e-3 of its norm where bf16's own rounding is
//                 1.7e-3 off
template <bool DOTS>
hipError_t launch_walk(const Args& A, int walks, bool wide, int kd, bool full, bool out_bf16,
                       hipStream_t s) {
#define KDA_LW(KDV)                                                              \
  do {                                                                           \
    if (wide)                                                                    \
      return full ? launch_walk_kd<true, KDV, true, DOTS, 3>(A, walks, s)        \
                  : launch_walk_kd<true, KDV, false, false, 3>(A, walks, s);     \
    if (!full) return launch_walk_kd<false, KDV, false, false, 1>(A, walks, s);  \
    if constexpr (DOTS) return hipErrorInvalidValue; /* launch_gradients */      \
    else if (out_bf16) return launch_walk_kd<false, KDV, true, false, kByLength>(A, walks, s); \
    else return launch_walk_kd<false, KDV, true, false, 2>(A, walks, s);         \
  } while (0)
  if (kd == 128) KDA_LW(128);
  KDA_LW(64);
#undef KDA_LW
}

template <int DK, int DV>
hipError_t launch_gradients_kd(const Args& A, bool alike, bool out_bf16, hipStream_t s) {
  const int64_t qk = walk_blocks(A, DV), v = walk_blocks(A, DK), blocks = 2 * qk + v;
  // A workgroup of dq or dk takes about half as long again as one of dv.  Where a
  // third round of workgroups would leave more than half of the CUs idle and the
  // sequences are alike, two thirds of dv's go before dk's: the CUs then get two of the
  // long ones or three of the short ones each.  us in this order / in the order dq, dk,
  // dv, bf16, dk = dv = 128: T = 4096 x 96 heads 437 / 454, x 88 388 / 412, x 104 475 /
  // 471; two of 2,048 x 48 193 / 206, twelve of 1,000 x 8 104 / 110; dk = dv = 64, T =
  // 4096 x 192 325 / 345.  Sequences of different lengths start longest first, and
  // splitting dv's short ones off delays dk's long ones: 4,000 and 96 x 48 280 / 229;
  // 2,500, 1,200, 300 and 96 x 24 148 / 123; with more rounds, 8 sequences x 96, 3640 /
  // 3515.
  const bool mixed = alike && qk == v && blocks > 2 * kCus && blocks <= 5 * kCus / 2;
  const int v1 = mixed ? (int)(v / 12 * 8) : 0;
  const dim3 grid((unsigned)blocks), block(Waves<false, true>::threads);
  if (out_bf16) gradient_kernel<DK, DV, kByLength><<<grid, block, 0, s>>>(A, (int)qk, v1);
  else gradient_kernel<DK, DV, 2><<<grid, block, 0, s>>>(A, (int)qk, v1);
  return hipGetLastError();
}
// all walks of the backward, bf16 operands; alike: no sequence is much longer than another
hipError_t launch_gradients(const Args& A, int dk, int dv, bool alike, bool out_bf16,
                            hipStream_t s) {
  if (dk == 128)
    return dv == 128 ? launch_gradients_kd<128, 128>(A, alike, out_bf16, s)
                     : launch_gradients_kd<128, 64>(A, alike, out_bf16, s);
  return dv == 128 ? launch_gradients_kd<64, 128>(A, alike, out_bf16, s)
                   : launch_gradients_kd<64, 64>(A, alike, out_bf16, s);
}

hipError_t launch_scan(const Args& A, int walks, int kd, hipStream_t s) {
  const dim3 grid((unsigned)scan_blocks(A, kd), walks);
  if (kd == 128) scan_kernel<128><<<grid, NTHR, 0, s>>>(A);
  else scan_kernel<64><<<grid, NTHR, 0, s>>>(A);
  return hipGetLastError();
}

// Chunks a segment when sequences are cut, 0 when they are walked whole.  A CU
// holds one workgroup, so whole sequences take the time of the longest one or, if
// that is more, of an even share of all chunks (`walkers` workgroups each); cut
// they take the even share for out, nearly as much again for the segments' own
// states, and two more launches.  Whole against cut, us, one sequence, dk = dv =
// 128: H = 1, T = 4096 106 / 23; H = 16, T = 512 18 / 22, T = 1024 32 / 25, T =
// 131072 3290 / 785; H = 32, T = 8192 211 / 105; H = 48, T = 4096 110 / 98; H =
// 64, T = 16384 422 / 417; H = 80, T = 16384 429 / 530.
// rounds: segments a CU gets in all.  One forward (fewer states to hand on; 1
// against 2: H = 16, T = 4096 40 / 47, H = 1, T = 131072 84 / 113, H = 16, T =
// 131072 788 / 779); two backward, where workgroups of different length even out
// (H = 8, T = 32768 609 / 556).
int cut_chunks(int64_t T_tot, int64_t N, int64_t walkers, int64_t longest, int rounds) {
  const int64_t chunks = cdiv(T_tot, C), all = chunks * walkers, even = cdiv(all, kCus);
  // (the bounds on N keep the workspace small: a state per sequence and segment)
  if (chunks < N * 4 * kMinSegChunks || N * walkers >= 4 * kCus) return 0;
  if (4 * longest < 9 * even + 12 * kMinSegChunks) return 0;
  const int64_t sc = cdiv(all, rounds * kCus);
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
    dotq = c.take(T_tot * H * 4);
    dotk = c.take(T_tot * H * 4);
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

// chunks of the longest sequence: from the host copy, or the most it can be
int64_t longest_chunks(const Problem& p) {
  if (!p.cu) return cdiv(p.T_tot / p.N, C);
  if (!p.cu_host) return cdiv(p.T_tot, C);
  int64_t m = 0;
  for (int n = 0; n < p.N; ++n)
    m = p.cu_host[n + 1] - p.cu_host[n] > m ? p.cu_host[n + 1] - p.cu_host[n] : m;
  return cdiv(m, C);
}
// segments of seg chunks that a grid over the sequences has to cover
int segments(const Problem& p, int seg) {
  const int64_t n = cdiv(longest_chunks(p), seg);
  return n > 1 ? static_cast<int>(n) : 1;
}
// the longest to decide by: lengths that are not known are taken as equal
int64_t longest_guess(const Problem& p) {
  return p.cu && !p.cu_host ? cdiv(p.T_tot / p.N, C) : longest_chunks(p);
}

}  // namespace

size_t prefill_workspace_bytes(int64_t T_tot, int N, int H, int dk, int dv) {
  const int seg = cut_chunks(T_tot, N, (int64_t)H * (dv / CT), cdiv(T_tot, C), 1);
  return seg ? ForwardWs(nullptr, T_tot, N, H, dk, dv, seg).bytes : 0;
}

bool prefill_fits(const Problem& p, bool wide) {
  const int seg = cut_chunks(p.T_tot, p.N, (int64_t)p.H * (p.dv / CT), longest_guess(p), 1);
  Args A{};
  A.N = p.N;
  A.H = p.H;
  A.nseg = seg ? segments(p, seg) : 1;
  A.walk[0].s_elems = (int64_t)p.dk * p.dv;
  return fits(walk_blocks(A, p.dk), wide ? Waves<true, true>::threads : Waves<false, true>::threads) &&
         (A.nseg == 1 || fits(scan_blocks(A, p.dk), NTHR));
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
  const int seg = cut_chunks(p.T_tot, p.N, (int64_t)p.H * (p.dv / CT), longest_guess(p), 1);
  const ForwardWs f(ws, p.T_tot, p.N, p.H, p.dk, p.dv, seg);
  if (seg && ws && ws_bytes >= f.bytes) {
    A.seg_chunks = seg;
    A.nseg = segments(p, seg);
    W.seg_state = f.state;
    W.seg_decay = f.decay;
  }
  if (A.nseg > 1) {
    hipError_t e = launch_walk<false>(A, 1, wide, p.dk, false, o_bf16, s);
    if (e == hipSuccess) e = launch_scan(A, 1, p.dk, s);
    if (e != hipSuccess) return e;
  }
  return launch_walk<false>(A, 1, wide, p.dk, true, o_bf16, s);
}

namespace {
// chunks a segment of dg's sums, and whether the walks are cut there
int border_chunks(int64_t T_tot, int N, int H, int dk, int dv, int64_t longest, bool* cut) {
  const int seg = cut_chunks(T_tot, N, (int64_t)H * (2 * (dk / CT) + dv / CT), longest, 2);
  *cut = seg > 0;
  return seg ? seg : kBorderChunks;
}
}  // namespace

size_t backward_workspace_bytes(int64_t T_tot, int N, int H, int Hk, int dk, int dv) {
  // by the longest that a sequence can be; where they turn out even, they are walked whole
  bool cut;
  const int seg = border_chunks(T_tot, N, H, dk, dv, cdiv(T_tot, C), &cut);
  const size_t a = BackwardWs(nullptr, T_tot, N, H, Hk, dk, dv, seg, cut).bytes;
  const size_t b = BackwardWs(nullptr, T_tot, N, H, Hk, dk, dv, kBorderChunks, false).bytes;
  return a > b ? a : b;
}

bool backward_fits(const Problem& p, bool wide) {
  bool cut;
  const int seg = border_chunks(p.T_tot, p.N, p.H, p.dk, p.dv, longest_guess(p), &cut);
  Args A{};
  A.N = p.N;
  A.H = p.H;
  A.nseg = cut ? segments(p, seg) : 1;
  A.walk[0].s_elems = (int64_t)p.dk * p.dv;
  const int64_t qk = walk_blocks(A, p.dv), v = walk_blocks(A, p.dk);
  return (wide ? fits(qk > v ? qk : v, Waves<true, true>::threads)
               : fits(2 * qk + v, Waves<false, true>::threads)) &&
         (A.nseg == 1 || (fits(scan_blocks(A, p.dv), NTHR) && fits(scan_blocks(A, p.dk), NTHR))) &&
         fits(slots_of(p.T_tot, p.N, seg) * p.H, DGT) &&
         (p.Hk == p.H || fits(group_sum_blocks(p), NTHR));
}

hipError_t launch_backward(const Problem& p, const Operand& q, const Operand& k, const Operand& v,
                           const float* S0, const Operand& d_o, const float* dS, void* dq, void* dk,
                           void* dv, bool grad_bf16, float* dg, float* dS0, void* ws,
                           hipStream_t s) {
  const int DK = p.dk, DV = p.dv, group = p.H / p.Hk;
  bool cut;
  const int seg = border_chunks(p.T_tot, p.N, p.H, DK, DV, longest_guess(p), &cut);
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
  A.nseg = cut ? segments(p, seg) : 1;

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
  Args B = A;  // dv needs no dots (and for dk != dv contracts over another width)
  B.first = 2;
  // the longest is at most a quarter longer than the mean (the longest that it can be where
  // the lengths are not known); segments are alike
  const bool alike = A.nseg > 1 || 4 * longest_chunks(p) * p.N <= 5 * cdiv(p.T_tot, C);
  for (int phase = A.nseg > 1 ? 0 : 2; phase < 3; ++phase) {
    hipError_t e;
    if (phase == 1) {
      e = launch_scan(A, 2, DV, s);
      if (e == hipSuccess) e = launch_scan(B, 1, DK, s);
    } else if (phase == 2 && !wide) {
      e = launch_gradients(A, DK, DV, alike, grad_bf16, s);
    } else {
      const bool full = phase == 2;
      e = launch_walk<true>(A, 2, wide, DV, full, grad_bf16, s);
      if (e == hipSuccess) e = launch_walk<false>(B, 1, wide, DK, full, grad_bf16, s);
    }
    if (e != hipSuccess) return e;
  }
  const int64_t slots = slots_of(p.T_tot, p.N, seg);
  dg_kernel<<<dim3((unsigned)(slots * p.H)), DGT, 0, s>>>(A, b.dotq, b.dotk, b.ends_s, b.ends_d,
                                                          DK, DV, dS != nullptr, dg, b.dg_part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!A.g.per_token) {
    dg_heads_kernel<<<dim3(p.H), 64, 0, s>>>(A, b.dg_part, slots, dg);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (group > 1 && p.T_tot > 0) {
    group_sum_kernel<<<dim3((unsigned)group_sum_blocks(p), 2), NTHR, 0, s>>>(
        A, b.hq, b.hk, DK, group, dq, dk, grad_bf16);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_zero_rows_behind(const int32_t* end, int T_tot, void* const* p,
                                   const int64_t* row_bytes, int count, hipStream_t s) {
  Cleared t{};
  int64_t most = 0;
  for (int i = 0; i < count; ++i) {
    t.p[i] = static_cast<char*>(p[i]);
    t.row_bytes[i] = row_bytes[i];
    most = row_bytes[i] > most ? row_bytes[i] : most;
  }
  // usually there is little or nothing to clear: no more workgroups than two a CU
  const int64_t blocks = cdiv(T_tot * most, NTHR * 16);
  zero_rows_kernel<<<dim3((unsigned)(blocks < 2 * kCus ? blocks : 2 * kCus), count), NTHR, 0, s>>>(
      end, T_tot, t);
  return hipGetLastError();
}

}  // namespace linattn
}  // namespace kda
