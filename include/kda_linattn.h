/*
 * kda_linattn.h - linear attention with one decay per head, and layer norm,
 * beside the KDA core of kda.h (same library, conventions, statuses and
 * KDA_DEBUG mode).
 *
 * Linear attention with a decay for each head is the KDA recurrence without
 * its delta correction and with one decay a head in place of one a channel.
 * For one sequence and one head, with a d_k x d_v fp32 state S (element
 * S[c][j]) and, per token t, the log-decay g_t <= 0:
 *
 *     S_t = exp(g_t) S_{t-1} + k_t v_t^T          o_t = scale * S_t^T q_t
 *
 * It has KDA's two regimes: a chunked form for prompts and training and a
 * one-token step over a pool of states for serving, which a prefill and the
 * decode of kda.h's pools hand states to in the same way.  Layer norm is the
 * layer's epilogue (over each head's output channels, or over a whole row).
 *
 * Heads: v, o and the states have H heads; q and k have Hk heads, H a multiple
 * of Hk, and head h reads q/k head h / (H / Hk).  dk and dv are 64 or 128 each.
 *
 * Decay: g holds one log-decay per token and head ([T_tot, H], g_len ==
 * T_tot*H) or, given explicitly, one per head used for every token ([H],
 * g_len == H); other lengths are refused (KDA_ERR_SHAPE).  A g below -110 is
 * taken as -110: exp(-110) is 0 beside any fp32 value that is not tiny.
 *
 * q, k, v, d_o and the states must be finite: a NaN or an infinity of one token
 * may reach every token of its chunk of 64 of that sequence and head, those
 * before it too.  A NaN in g is carried on.  (Rows of q, k, v, g and d_o that belong
 * to no sequence, and those of sequences that the decode skips, may hold anything;
 * KDA_DEBUG does not look at them.)
 *
 * Sizes: T_tot < 2^31, H <= 16384, N*H <= 2^24; and the work items of a launch (fewer
 * than 2^32) have to hold the call, which ends at about 3 million (sequence, head) pairs
 * in the prefill, 1 million in its gradients (dk = dv = 128) and 8.3 million in the
 * decode.  Calls beyond that are refused (KDA_ERR_UNSUPPORTED).
 *
 * Strides: q, k and v give the distance between tokens (sequences, in the
 * decode) in elements: at least heads * dim, so that they may be slices of a
 * fused projection; heads and channels are dense.  Rows are 16-byte aligned.
 * Everything else is dense.
 */
#ifndef KDA_LINATTN_H_
#define KDA_LINATTN_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kda_linattn_chunk_prefill - the recurrence over a packed variable-length batch.
 *
 *   q, k  [T_tot, Hk, dk], v [T_tot, H, dv]   dtype qkv_dt, token strides
 *         q_stride, k_stride, v_stride (elements)
 *   g     fp32 [T_tot, H] or [H] (g_len says which)
 *   cu_seqlens [N+1] int32, device copy; sequence n owns tokens cu_seqlens[n]
 *         .. cu_seqlens[n+1]-1.  It must not decrease and begins at 0.  NULL: N
 *         sequences of T_tot / N tokens each (T_tot % N == 0).  cu_seqlens_host:
 *         as for kda_chunk_prefill (NULL allowed; the kernels clamp every range
 *         into [0, T_tot]).  Rows of o that belong to no sequence, behind the
 *         last one, are left as they were.
 *   initial_state, final_state: pools [num_slots, H, dk, dv] of state_dt, either
 *         NULL, possibly the same (an in-place update), addressed by
 *         state_indices or by sequence, with the rules of
 *         kda_chunk_prefill_gated: a slot outside the pool starts from zeros
 *         and is not written, two sequences must not share a written slot.
 *   o     [T_tot, H, dv] dtype o_dt
 *   workspace: kda_linattn_chunk_prefill_workspace_bytes, 256-byte aligned.  It
 *         is needed to cut long sequences into segments when there are few of
 *         them; a NULL or smaller workspace is allowed, the sequences are then
 *         walked whole (the same result to rounding, with fewer workgroups).
 * Accuracy: products run on bf16 MFMA with fp32 accumulation.  bf16 q, k and v
 * enter exactly and the values that make the state as sums of three bf16 values:
 * the state agrees with an fp64 recurrence to about 3e-7 of its norm.  The scores
 * and states that make o enter as one bf16 value where o is bf16 and the sequence
 * has more than 64 tokens (each off by at most 2^-8 of itself: o is 2.3e-3 of its
 * norm off, where bf16's own rounding makes 1.7e-3), else as two (o fp32: about
 * 3e-6).  What a sequence is packed with does not change the digits of its o, but
 * for the last ones of fp32 where a batch is cut into segments.
 * fp32 q, k and v enter as three bf16 values each, and so does everything that
 * they meet (about 3e-7).
 */
kda_status kda_linattn_chunk_prefill(const void* q, int64_t q_stride, const void* k,
                                     int64_t k_stride, const void* v, int64_t v_stride,
                                     kda_dtype qkv_dt, const float* g, int64_t g_len,
                                     const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                                     int32_t N, const void* initial_state, void* final_state,
                                     kda_dtype state_dt, int64_t num_slots,
                                     const int32_t* state_indices, void* o, kda_dtype o_dt,
                                     int64_t T_tot, int32_t H, int32_t Hk, int32_t dk, int32_t dv,
                                     float scale, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* Workspace bytes of kda_linattn_chunk_prefill (0: none is used, or the
 * arguments are unsupported). */
size_t kda_linattn_chunk_prefill_workspace_bytes(int64_t T_tot, int32_t N, int32_t H, int32_t dk,
                                                 int32_t dv);

/*
 * kda_linattn_chunk_prefill_backward - gradients of kda_linattn_chunk_prefill.
 *
 * For the loss sum(d_o * o) + sum(d_final_state * final_state) of the forward
 * with the same q, k, v, g, cu_seqlens, scale and fp32 initial_state
 * [N, H, dk, dv] (or NULL), writes
 *   dq, dk [T_tot, Hk, dk], dv [T_tot, H, dv]  dtype grad_dt (q and k shared by
 *         several heads get the sum of their gradients)
 *   dg    fp32, g's shape ([T_tot, H], or [H]: summed over every token)
 *   d_initial_state [N, H, dk, dv] fp32 (NULL: not wanted)
 * d_o [T_tot, H, dv] has dtype do_dt; d_o and d_final_state [N, H, dk, dv] fp32
 * may be NULL (zero).  Rows behind the last sequence are left as they were.
 * A g below -110 gets the gradient of the recurrence at -110.
 * The sums run in a fixed order: the same call gives the same bits.
 * Accuracy: dv as o above; dq, dk and d_initial_state 3e-7 of their norm plus
 * their rounding; dg is a small difference of sums of products, formed from
 * three-value factors and summed in 64 bits: 1e-6 to 5e-6 of its norm.
 * workspace: kda_linattn_chunk_prefill_backward_workspace_bytes, 256-byte
 * aligned, KDA_ERR_WORKSPACE below it.
 */
kda_status kda_linattn_chunk_prefill_backward(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, kda_dtype qkv_dt, const float* g, int64_t g_len, const int32_t* cu_seqlens,
    const int32_t* cu_seqlens_host, int32_t N, const float* initial_state, const void* d_o,
    kda_dtype do_dt, const float* d_final_state, void* dq, void* dk, void* dv, kda_dtype grad_dt,
    float* dg, float* d_initial_state, int64_t T_tot, int32_t H, int32_t Hk, int32_t dk_dim,
    int32_t dv_dim, float scale, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of kda_linattn_chunk_prefill_backward; 0 for unsupported arguments. */
size_t kda_linattn_chunk_prefill_backward_workspace_bytes(int64_t T_tot, int32_t N, int32_t H,
                                                          int32_t Hk, int32_t dk, int32_t dv);

/*
 * kda_zero_rows_behind - zeros the rows behind the last sequence.
 *
 * The calls above leave those rows of o and of the gradients as they were; where the
 * host does not know cu_seqlens[N], this clears them.  For each of `count` (0 to 4)
 * tensors of T_tot rows, row i has row_bytes[i] bytes (a multiple of 4, pointers 4-byte
 * aligned): bytes [cu_seqlens[N] * row_bytes[i], T_tot * row_bytes[i]) become 0
 * (cu_seqlens[N] clamped into [0, T_tot]).  `tensors` and `row_bytes` are host arrays.
 */
kda_status kda_zero_rows_behind(const int32_t* cu_seqlens, int32_t N, int64_t T_tot,
                                void* const* tensors, const int64_t* row_bytes, int32_t count,
                                void* stream);

/*
 * kda_linattn_recurrent_decode - one token per sequence over a pool of states.
 *
 *   q, k  [N, Hk, dk], v [N, H, dv] dtype qkv_dt, strides between sequences
 *   g     fp32 [N, H] or [H] (g_len)
 *   state [num_slots, H, dk, dv] dtype state_dt, read and overwritten in place;
 *         sequence n uses slot state_indices[n] (int32, device; NULL: slot n,
 *         then num_slots >= N).  A slot outside [0, num_slots) skips the
 *         sequence: its o is zeros and no state is touched.  Two sequences of
 *         one call must not share a slot (their updates would race).
 *   o     [N, H, dv] dtype o_dt
 * The arithmetic is fp32; a bf16 state is rounded to nearest even each step, and
 * o is read from the state before that rounding.
 */
kda_status kda_linattn_recurrent_decode(const void* q, int64_t q_stride, const void* k,
                                        int64_t k_stride, const void* v, int64_t v_stride,
                                        kda_dtype qkv_dt, const float* g, int64_t g_len,
                                        void* state, kda_dtype state_dt, int64_t num_slots,
                                        const int32_t* state_indices, void* o, kda_dtype o_dt,
                                        int32_t N, int32_t H, int32_t Hk, int32_t dk, int32_t dv,
                                        float scale, void* stream);

/*
 * kda_layernorm - layer norm of every row:
 *
 *   y = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * weight + bias
 *
 *   x, y    [rows, d] dtype x_dt, y_dt; y may be x (same dtype)
 *   weight, bias  fp32 [groups, d], either NULL (1 and 0); row r uses row
 *           r % groups: groups = 1 shares one weight, groups = H over an
 *           [T, H, d] tensor (rows = T*H) gives every head its own.
 * 1 <= d <= 16384, rows % groups == 0, groups <= 65535.  Pointers need only their
 * element's alignment.  The mean and the mean square of the differences are sums in
 * fp32 over values held in registers; the mean's own rounding error comes off both, so
 * a row whose spread is far below its mean keeps its digits.
 */
kda_status kda_layernorm(const void* x, kda_dtype x_dt, const float* weight, const float* bias,
                         int64_t groups, void* y, kda_dtype y_dt, int64_t rows, int32_t d,
                         float eps, void* stream);

/*
 * kda_layernorm_backward - gradients of kda_layernorm, from dy and x (the
 * statistics are formed again from x).  With xh the normalised row and t = dy * weight:
 *
 *   dx      = (t - mean(t) - xh mean(t xh)) / sqrt(var + eps)     dtype x_dt
 *   dweight = sum over the rows of a group of dy * xh             fp32 [groups, d]
 *   dbias   = sum over the rows of a group of dy                  fp32 [groups, d]
 *
 * dweight and dbias may be NULL; dx may be dy or x (same dtype).  workspace:
 * kda_layernorm_backward_workspace_bytes, 16-byte aligned (needed when dweight
 * or dbias is wanted, KDA_ERR_WORKSPACE below it).  The sums over the rows run
 * in a fixed order: the same call gives the same bits.
 */
kda_status kda_layernorm_backward(const void* dy, kda_dtype dy_dt, const void* x, kda_dtype x_dt,
                                  const float* weight, int64_t groups, void* dx, float* dweight,
                                  float* dbias, int64_t rows, int32_t d, float eps,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of kda_layernorm_backward; 0 for unsupported arguments. */
size_t kda_layernorm_backward_workspace_bytes(int64_t rows, int64_t groups, int32_t d);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LINATTN_H_ */
