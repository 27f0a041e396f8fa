/*
 * kda_gatedrec.h - gated linear recurrence and RMS norm, beside the KDA core of kda.h and
 * the linear attention of kda_linattn.h (same library, conventions, statuses and KDA_DEBUG
 * mode).
 *
 * The gated linear recurrence is the recurrence with a state of one value a channel.  For
 * one sequence and channel c, from the state h_0 (0, or an entry of a pool):
 *
 *     g_t = -exp(A_log[c]) * softplus(r[t,c] + dt_bias[c])     the gate of kda_gate
 *     m_t = sqrt(1 - exp(2 g_t))  if normalize, else 1
 *     h_t = exp(g_t) h_{t-1} + m_t * sigmoid(i[t,c]) * x[t,c]
 *
 * It has the regimes of the library's other recurrences: a scan for prompts and training,
 * its gradients, and a one-token step over a pool of states [num_slots, C] that scan and
 * step share.  RMS norm, with the residual's addition, stands before the layer.
 *
 * Inputs: x, r and i are [T_tot, C] of one dtype; each gives the distance between its tokens
 * in elements (at least C, at most 2^24), so that they may be columns of one fused
 * projection.  i may be NULL: no input gate (sigmoid(i) is 1).  A_log NULL: r holds the
 * log-decays themselves, at most 0 (dt_bias must be NULL).  The kernels take one above 0 for 0
 * (g = min(r, 0), without a gradient); KDA_DEBUG=1 refuses it, as it does in every recurrence of
 * the library.  dt_bias NULL: zeros.
 * Tensors need only their element's alignment; C is 1 to 2^20.  Everything but x, r and i is
 * dense.
 *
 * Values: x and the states have to be finite, exp(A_log) a normal fp32 number, logits must not
 * be NaN (infinite ones are the gates' limits).  What is not stays in its channel of its
 * sequence: what comes before it, other channels and the sequences around it do not see it.
 * Rows that belong to no sequence, and sequences that the step skips, may hold anything.
 *
 * Accuracy: sums and states are fp32.  h agrees with the 64-bit recurrence to about 1e-6 of
 * its norm plus its rounding, also for channels that decay by 1e-5 a token (decays near 1
 * are carried as 1 - exp(g)).
 *
 * Sizes: T_tot < 2^31, and the work items of a launch have to hold the call: about 2^30
 * (token, 64 channels) pairs in the scan, 2^28 in the gradients (KDA_ERR_UNSUPPORTED beyond).
 */
#ifndef KDA_GATEDREC_H_
#define KDA_GATEDREC_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kda_gatedrec_scan - the recurrence over a packed variable-length batch.
 *
 *   x, r, i [T_tot, C] dtype in_dt; A_log, dt_bias [C] fp32 (see above)
 *   cu_seqlens [N+1] int32, device copy; sequence n owns tokens cu_seqlens[n] ..
 *         cu_seqlens[n+1]-1.  It must not decrease and begins at 0.  NULL: N sequences of
 *         T_tot / N tokens each (T_tot % N == 0).  cu_seqlens_host: the same on the host or
 *         NULL; when given it is validated.  The kernels clamp every range into [0, T_tot].
 *         Rows of h behind the last sequence are left as they were.
 *   initial_state, final_state: pools [num_slots, C] of state_dt, either NULL, possibly the
 *         same (an in-place update), addressed by state_indices (int32 [N], device) or by
 *         sequence (NULL; then num_slots >= N).  A slot outside the pool starts from zeros
 *         and is not written; two sequences must not share a written slot.
 *   h     [T_tot, C] dtype h_dt
 *   starts: NULL, or fp32 [ceil(T_tot / 32), C] (kda_gatedrec_starts_bytes) that the call
 *         fills with states on its way, for kda_gatedrec_scan_backward of the same inputs.
 *         What lies behind the last sequence is left as it was.
 *   workspace: kda_gatedrec_scan_workspace_bytes (0 for up to 128 tokens), 16-byte aligned,
 *         KDA_ERR_WORKSPACE below it; what it holds does not matter.  It must not be used by
 *         anything else until the stream has finished this call.
 * The same call gives the same bits.
 */
kda_status kda_gatedrec_scan(const void* x, int64_t x_stride, const void* r, int64_t r_stride,
                             const void* i, int64_t i_stride, kda_dtype in_dt, const float* A_log,
                             const float* dt_bias, int32_t normalize, const int32_t* cu_seqlens,
                             const int32_t* cu_seqlens_host, int32_t N, const void* initial_state,
                             void* final_state, kda_dtype state_dt, int64_t num_slots,
                             const int32_t* state_indices, void* h, kda_dtype h_dt, float* starts,
                             int64_t T_tot, int32_t C, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Workspace bytes of kda_gatedrec_scan (0: none is needed, or the arguments are unsupported). */
size_t kda_gatedrec_scan_workspace_bytes(int64_t T_tot, int32_t C);

/* Bytes of `starts`; 0 for unsupported arguments. */
size_t kda_gatedrec_starts_bytes(int64_t T_tot, int32_t C);

/*
 * kda_gatedrec_scan_backward - gradients of kda_gatedrec_scan.
 *
 * For the loss sum(dh * h) + sum(d_final_state * final_state) of the scan of the same
 * inputs, parameters, cu_seqlens and fp32 initial_state [N, C] (or NULL), writes
 *   dx, dr, di [T_tot, C] dtype grad_dt (di NULL where i is; with A_log NULL dr is the
 *         gradient of the log-decays, 0 where r > 0)
 *   dA_log, ddt_bias [C] fp32 (either NULL: not wanted; both NULL without A_log)
 *   d_initial_state [N, C] fp32 (NULL: not wanted)
 * dh [T_tot, C] has dtype dh_dt; dh and d_final_state [N, C] fp32 may be NULL (zero).
 * starts: what the scan wrote, or NULL: the states are formed again first (a second walk).
 * The square root's slope has no bound where g is 0: its part of the gradient is taken as 0
 * where m is, and is sigmoid(i) x / m elsewhere, which has to be within fp32's range (such an m is
 * 1e-23 or more: for x up to 1e15 it is).  Rows behind the last sequence are left as they were.
 * The sums run in a fixed order: the same call gives the same bits.
 * workspace: kda_gatedrec_scan_backward_workspace_bytes, 16-byte aligned,
 * KDA_ERR_WORKSPACE below it.
 */
kda_status kda_gatedrec_scan_backward(
    const void* x, int64_t x_stride, const void* r, int64_t r_stride, const void* i,
    int64_t i_stride, kda_dtype in_dt, const float* A_log, const float* dt_bias, int32_t normalize,
    const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, int32_t N,
    const float* initial_state, const float* starts, const void* dh, kda_dtype dh_dt,
    const float* d_final_state, void* dx, void* dr, void* di, kda_dtype grad_dt, float* dA_log,
    float* ddt_bias, float* d_initial_state, int64_t T_tot, int32_t C, void* workspace,
    size_t workspace_bytes, void* stream);

/* Workspace bytes of kda_gatedrec_scan_backward, with `starts` or without (has_starts 0);
 * 0 for unsupported arguments. */
size_t kda_gatedrec_scan_backward_workspace_bytes(int64_t T_tot, int32_t C, int32_t has_starts);

/*
 * kda_gatedrec_decode - one token per sequence over a pool of states.
 *
 *   x, r, i [N, C] dtype in_dt, strides between sequences
 *   state [num_slots, C] dtype state_dt, read and overwritten in place; sequence n uses slot
 *         state_indices[n] (int32, device; NULL: slot n, then num_slots >= N).  A slot outside
 *         [0, num_slots) skips the sequence: its h is zeros and no state is touched.  Two
 *         sequences of one call must not share a slot (their updates would race).
 *   h     [N, C] dtype h_dt
 * The arithmetic is fp32; a bf16 state is rounded to nearest even each step, and h is the
 * state before that rounding.
 */
kda_status kda_gatedrec_decode(const void* x, int64_t x_stride, const void* r, int64_t r_stride,
                               const void* i, int64_t i_stride, kda_dtype in_dt,
                               const float* A_log, const float* dt_bias, int32_t normalize,
                               void* state, kda_dtype state_dt, int64_t num_slots,
                               const int32_t* state_indices, void* h, kda_dtype h_dt, int32_t N,
                               int32_t C, void* stream);

/*
 * kda_rmsnorm - RMS norm of every row, with the residual's addition:
 *
 *   s = x + residual                 (s = x where residual is NULL)
 *   y = s / sqrt(mean(s^2) + eps) * weight
 *
 *   x     [rows, d] dtype x_dt; rows come in tokens of `groups` rows, x_stride elements
 *         between tokens (at least groups*d), the rows of a token dense
 *   residual, s [rows, d] dtype res_dt (x_dt or KDA_F32), both or neither; s may be residual,
 *         or a dense x of the same dtype.  What is normalised is s as it is stored (rounded
 *         to res_dt), so that kda_rmsnorm_backward of s is the gradient of what was computed.
 *   weight fp32 [groups, d] or NULL (1); row r uses row r % groups: groups = 1 shares one
 *         weight, groups = H over an [T, H, d] tensor gives every head its own
 *   y     [rows, d] dtype y_dt; may be a dense x of the same dtype
 * 1 <= d <= 16384, rows % groups == 0, groups <= 65535.  Pointers need only their element's
 * alignment.  The mean square is a sum in fp32 over values held in registers.
 */
kda_status kda_rmsnorm(const void* x, kda_dtype x_dt, int64_t x_stride, const void* residual,
                       void* s, kda_dtype res_dt, const float* weight, int64_t groups, void* y,
                       kda_dtype y_dt, int64_t rows, int32_t d, float eps, void* stream);

/*
 * kda_rmsnorm_e4m3 - the same with y in 8 bits (OCP e4m3, one byte a value) and its scales:
 *
 *   scales [rows, ceil(d / 128)] fp32, one for each 128 columns (scale_group 128), or [rows, 1],
 *         one a row (scale_group 0):  scale = max(|y|) / 448 over the columns
 *   y     [rows, d]: the quotient y / scale in fp32, rounded to nearest even (a largest |y| below
 *         2^-85: of that or the fp32 number beside it), so that y8 * scale is about y
 * A largest |y| below 2^-100 counts as 2^-100.  A NaN makes its scale and values NaN.
 */
kda_status kda_rmsnorm_e4m3(const void* x, kda_dtype x_dt, int64_t x_stride, const void* residual,
                            void* s, kda_dtype res_dt, const float* weight, int64_t groups,
                            uint8_t* y, float* scales, int32_t scale_group, int64_t rows,
                            int32_t d, float eps, void* stream);

/*
 * kda_rmsnorm_backward - gradients of kda_rmsnorm (and, straight through the rounding, of
 * kda_rmsnorm_e4m3), from dy and s (x where there was no residual; the mean square is formed
 * again).  With xh = s / sqrt(mean(s^2) + eps) and t = dy * weight:
 *
 *   dx      = (t - xh mean(t xh)) / sqrt(mean(s^2) + eps) + d_residual     dtype s_dt
 *   dweight = sum over the rows of a group of dy * xh                      fp32 [groups, d]
 *
 *   s [rows, d] dtype s_dt, s_stride as x_stride above; dy [rows, d] dtype dy_dt; d_residual
 *   [rows, d] dtype s_dt or NULL: the gradient that reaches s by the residual stream.  dx is
 *   the gradient of x and of residual both; it may be dy, a dense s or d_residual (same
 *   dtype).  dweight may be NULL.  workspace: kda_rmsnorm_backward_workspace_bytes, 16-byte
 *   aligned (needed when dweight is wanted, KDA_ERR_WORKSPACE below it).  The sums over the
 *   rows run in a fixed order: the same call gives the same bits.
 */
kda_status kda_rmsnorm_backward(const void* dy, kda_dtype dy_dt, const void* s, kda_dtype s_dt,
                                int64_t s_stride, const float* weight, int64_t groups,
                                const void* d_residual, void* dx, float* dweight, int64_t rows,
                                int32_t d, float eps, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Workspace bytes of kda_rmsnorm_backward; 0 for unsupported arguments. */
size_t kda_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t groups, int32_t d);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GATEDREC_H_ */
