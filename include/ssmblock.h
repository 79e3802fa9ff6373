/*
 * ssmblock.h -- C ABI of libssmscan, second part: the operators that a block of
 * a recurrent language model needs around its scan (ssmscan.h holds the scans).
 *
 *   ssm_add_norm_*    residual add, residual scale and norm before a block
 *   ssm_gated_norm_*  the norm after a block, over groups of channels, with
 *                     the SiLU gate
 *   ssm_linattn_*     linear attention with a decay for each head
 *   ssm_q4_*          products of few rows with 4-bit weights
 *
 * Ownership, errors, asynchrony, graph capture and reproducibility are those
 * of ssmscan.h: every pointer is a device pointer owned by the caller, every
 * argument is checked on the host before anything is enqueued, a non-OK status
 * means that nothing was enqueued and ssm_last_error() says why, calls enqueue
 * only kernels on `stream` (and the stream-ordered workspace that a call's
 * comment names), and results are bitwise reproducible (no atomics).
 * These calls need no alignment beyond the element's unless their comment says
 * so.  Outputs must not overlap an input or each other except where stated.
 * A required pointer may be NULL only when its tensor has no elements.
 */
#ifndef SSMBLOCK_H
#define SSMBLOCK_H

#include "ssmscan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A call whose comment names a workspace takes it from the library's pool of the
 * device, which costs tens of microseconds of the host's time.  ssm_workspace
 * offers memory of the caller's for the calling thread's next such call, of at least
 * ssm_workspace_bytes() bytes, 16-byte aligned, that nothing but the call's stream uses
 * until the call's kernels have run; the call takes from the pool what does not
 * fit.  The offer ends with that call, also if it is refused; NULL withdraws it.
 * ssm_workspace_bytes: what the thread's last such call wanted (0: nothing, as where it
 * was refused); it depends on the call's sizes, types, flags, plan and absent tensors,
 * on whether a state is updated in place, and on the device's number of CUs, alone.  The
 * sizes in the calls' comments are for orientation (the parts of a workspace are each
 * rounded up to 16 bytes): this is the one to allocate by.
 */
ssm_status ssm_workspace(void* memory, int64_t bytes);
int64_t ssm_workspace_bytes(void);

/*
 * Bits of the norm calls' flags:
 *   SSM_NORM_CENTER     subtract the mean first (layer norm); without it the
 *                       rows are divided by their root mean square.
 *   SSM_NORM_GATE_LAST  gated norm only: norm first, then the gate.
 */
#define SSM_NORM_CENTER 1
#define SSM_NORM_GATE_LAST 2

/* Largest width that one norm runs over (width, or width / ngroups, of at most
 * 65535 groups and 2^24 channels in all). */
#define SSM_NORM_MAX_WIDTH 8192

/*
 * The norm before a block, with the residual add that precedes it:
 *
 *   r[i,d]   = alpha * residual[i,d] + scale[d] * x[i,d]
 *   out[i,d] = (r[i,d] - m_i) / sqrt(v_i + eps) * weight[d] + bias[d]
 *
 * with m_i the row's mean under SSM_NORM_CENTER and 0 without it, and v_i the
 * mean of (r[i,.] - m_i)^2.  Statistics and r are fp32; out is formed from the
 * fp32 r, not from the rounded residual_out.  A row's sum of squares has to stay within
 * fp32 (magnitudes below 2e17 always do): past it the row's statistics are infinite.
 *   x            : [rows, width] in x_dtype, rows x_stride elements apart
 *                  (x_stride >= width)
 *   residual     : [rows, width] in res_dtype, or NULL (r = scale x)
 *   weight, bias, scale: [width] fp32, or NULL (1, 0, 1)
 *   residual_out : [rows, width] in res_dtype, or NULL (r is not stored); may be
 *                  the same buffer as residual (in place)
 *   out          : [rows, width] in out_dtype
 */
ssm_status ssm_add_norm_fwd(const void* x, int64_t x_stride, const void* residual, const float* weight,
                            const float* bias, const float* scale, float alpha, float eps, int flags, void* out,
                            void* residual_out, int64_t rows, int64_t width, ssm_dtype x_dtype,
                            ssm_dtype res_dtype, ssm_dtype out_dtype, void* stream);

/*
 * Its gradients, from the stored r (= residual_out), dout = dL/dout and,
 * optionally, dresidual_out = dL/dresidual_out (what arrives at the residual
 * stream behind the block; NULL: nothing).  With n the normed rows before
 * weight and u = dout weight:
 *
 *   dr        = (u - [mean u] - n mean(u n)) / sqrt(v + eps) + dresidual_out
 *               ([mean u] under SSM_NORM_CENTER)
 *   dresidual = alpha dr;  dx = scale dr;  dweight[d] = sum_i dout n;
 *   dbias[d] = sum_i dout;  dscale[d] = sum_i x dr
 *
 *   dout in out_dtype; r, dresidual_out, dresidual in res_dtype; x, dx in
 *   x_dtype; dweight, dbias, dscale: [width] fp32.  Each output may be NULL (not
 *   computed); x is needed for dscale only.  dresidual may be the same buffer as
 *   dresidual_out.  The sums over rows run in a fixed order over a workspace
 *   of at most SSM_NORM_MAX_BLOCKS * 3 * width * 4 bytes, taken on `stream`
 *   where one of them is asked for.
 */
#define SSM_NORM_MAX_BLOCKS 1024
ssm_status ssm_add_norm_bwd(const void* dout, const void* r, const float* weight, const void* dresidual_out,
                            const void* x, int64_t x_stride, const float* scale, float alpha, float eps, int flags,
                            void* dx, void* dresidual, float* dweight, float* dbias, float* dscale, int64_t rows,
                            int64_t width, ssm_dtype x_dtype, ssm_dtype res_dtype, ssm_dtype out_dtype,
                            void* stream);

/*
 * The norm after a block's mixer, over ngroups contiguous groups of
 * width / ngroups channels, with the gate z (NULL: no gate):
 *
 *   without SSM_NORM_GATE_LAST:  out = norm(x * silu(z)) * weight + bias
 *   with it:                     out = (norm(x) * weight + bias) * silu(z)
 *
 *   x, z : [rows, width] in in_dtype, rows x_stride and z_stride elements apart
 *   weight, bias: [width] fp32, or NULL (1, 0);  out: [rows, width] in out_dtype
 */
ssm_status ssm_gated_norm_fwd(const void* x, int64_t x_stride, const void* z, int64_t z_stride, const float* weight,
                              const float* bias, float eps, int flags, void* out, int64_t rows, int64_t width,
                              int64_t ngroups, ssm_dtype in_dtype, ssm_dtype out_dtype, void* stream);

/*
 * Its gradients, from the forward's inputs and dout [rows, width] in out_dtype:
 * dx and dz (iff z is given) [rows, width] in in_dtype; dweight and dbias
 * [width] fp32, each NULL if not wanted (bias enters dz under
 * SSM_NORM_GATE_LAST).  Workspace as for ssm_add_norm_bwd.
 */
ssm_status ssm_gated_norm_bwd(const void* dout, const void* x, int64_t x_stride, const void* z, int64_t z_stride,
                              const float* weight, const float* bias, float eps, int flags, void* dx, void* dz,
                              float* dweight, float* dbias, int64_t rows, int64_t width, int64_t ngroups,
                              ssm_dtype in_dtype, ssm_dtype out_dtype, void* stream);

/*
 * Linear attention with a decay for each head:
 *
 *   S_t = exp(g[b,t,h]) S_{t-1} + v_t k_t^T          (S: [dv, dk] per head)
 *   out_t = scale * S_t q_t
 *
 * computed for prompts chunk by chunk with matrix products (as the Mamba-2 scan
 * of ssmscan.h, whose decay is tied to its input's coefficient, and which has no
 * gradient), and for single tokens by the recurrence.
 *   q, k      : [batch, seqlen, ngroups, dk] bf16: each of the ngroups serves
 *               nheads / ngroups consecutive heads
 *   v, out    : [batch, seqlen, nheads, dv]; v bf16, out in out_dtype
 *   log_decay : [batch, seqlen, nheads] fp32, or with SSM_LINATTN_FIXED_DECAY
 *               [nheads], the same for every step.  Decays are meant to be <= 0;
 *               minus infinity forgets everything before its step.
 *   initial_state, last_state: [batch, nheads, dv, dk] fp32, each NULL for zero or
 *               not stored; last_state may be initial_state (in place).
 * q, k and v may be slices of packed tensors: token (b, t)'s values start
 * (b * seqlen + t) * q_row (k_row, v_row) elements after the first token's.
 * dk and dv: multiples of 8 up to SSM_LINATTN_MAX_DIM; q, k, v 16-byte aligned,
 * rows multiples of 8 elements and at most 2^24; nheads a multiple of ngroups,
 * at most 65535, as batch, and batch * nheads below 2^23 (backward: 2.7 million);
 * states and out 16-byte aligned.  The state, the sums and the
 * decays are fp32; the products run on bf16 matrix cores with fp32 sums, computed
 * operands split into three bf16 terms (all 24 bits), so that fp32 outputs, gradients and
 * states are off by fp32 roundings alone.  A value of v that is
 * not finite makes its column not finite from its step on, one of q, k or the
 * decays every column; earlier steps are not touched.
 *
 * Plans: as for ssm_ssd_fwd.  A workgroup walks 64 columns of one (batch row,
 * head); where they are few, the sequence is cut into time chunks (chunk_len a
 * multiple of 32 where it cuts, at most 65535 of them), which costs one more pass
 * over k and v and a workspace of
 * batch * n_chunks * nheads * (dk * dv + 1) * 4 bytes on `stream` (plus a copy of
 * an in-place initial state).  plan may be NULL; its states_per_wave is ignored.
 */
#define SSM_LINATTN_FIXED_DECAY 1
#define SSM_LINATTN_MAX_DIM 128

ssm_status ssm_linattn_plan_query(int64_t batch, int64_t seqlen, int64_t nheads, int64_t dk, int64_t dv,
                                  ssm_plan* plan);

ssm_status ssm_linattn_fwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v, int64_t v_row,
                           const float* log_decay, int flags, float scale, const float* initial_state, void* out,
                           float* last_state, int64_t batch, int64_t seqlen, int64_t nheads, int64_t ngroups,
                           int64_t dk, int64_t dv, ssm_dtype in_dtype, ssm_dtype out_dtype, void* stream,
                           const ssm_plan* plan);

/*
 * Its gradients, from the forward's inputs, dout [batch, seqlen, nheads, dv] bf16
 * and, optionally, dlast_state = dL/dlast_state:
 *   dq, dk        : [batch, seqlen, ngroups, dk] in grad_dtype (summed over the
 *                   heads of a group in head order)
 *   dv            : [batch, seqlen, nheads, dv] in grad_dtype
 *   dlog_decay    : fp32, of log_decay's shape
 *   dinitial_state: [batch, nheads, dv, dk] fp32, or NULL (not computed)
 * The forward's outputs are not needed.  Values that are not finite reach what depends on
 * them; a decay also dk and dv of the steps behind it in its 32, and any value dlog_decay of
 * its head throughout the time chunk.  Sequences are cut into time chunks of at
 * most 2048 steps.  Workspace, on `stream`:
 * batch * seqlen * nheads * ceil(dk / 64) * 8 bytes, with more than one time chunk
 * 8 * batch * n_chunks * nheads * (dk * dv + 1), with dlast_state and
 * with initial_state batch * nheads * dk * dv * 4 each, with nheads > ngroups
 * batch * seqlen * nheads * dk * 8 more, with a fixed decay 8 for every time chunk and
 * 8 * dk * dv (each rounded up to 64 or 128) for every 128 steps in it but the last, of a
 * head.  Alignment and rows as above, gradients and dout 16-byte aligned.
 */
ssm_status ssm_linattn_bwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v, int64_t v_row,
                           const float* log_decay, int flags, float scale, const float* initial_state,
                           const void* dout, const float* dlast_state, void* dq, void* dk_, void* dv_,
                           float* dlog_decay, float* dinitial_state, int64_t batch, int64_t seqlen, int64_t nheads,
                           int64_t ngroups, int64_t dk, int64_t dv, ssm_dtype in_dtype, ssm_dtype grad_dtype,
                           void* stream);

/*
 * One token for every (b, h): state_out = exp(g) state + v k^T and
 * out = scale * state_out q.  state, state_out: [batch, nheads, dv, dk] fp32, which may
 * be one buffer (in place) or two (the state before the token is kept).
 * q, k: [batch, ngroups, dk]; v, out: [batch, nheads, dv]; log_decay: [batch, nheads],
 * or [nheads] with SSM_LINATTN_FIXED_DECAY.  in_dtype fp32 or bf16; dk a multiple of
 * 4 up to SSM_LINATTN_MAX_STEP_DK; dv from 1 to 2^24; nheads and batch at most 65535.  States
 * 16-byte aligned, q and k aligned to four elements.
 */
#define SSM_LINATTN_MAX_STEP_DK 256
ssm_status ssm_linattn_state_update(const float* state, float* state_out, const void* q, const void* k, const void* v,
                                    const float* log_decay, int flags, float scale, void* out, int64_t batch,
                                    int64_t nheads, int64_t ngroups, int64_t dk, int64_t dv, ssm_dtype in_dtype,
                                    ssm_dtype out_dtype, void* stream);

/*
 * Products of few rows with 4-bit weights and group scales, for the projections
 * of a decode step:
 *
 *   out[m,n] = sum_k x[m,k] * (code[n,k] - zero[n,g]) * scale[n,g] + bias[n],  g = k / group
 *
 *   x      : [m, k] in in_dtype, rows x_row elements apart, 16-byte aligned and
 *            rows multiples of 16 bytes
 *   codes  : [n, k / 2] bytes, two codes (0..15) per byte, the lower k in the low
 *            four bits; 16-byte aligned
 *   scales : [n, k / group] fp32 or bf16 (scale_dtype)
 *   zeros  : [n, k / group] bytes, or NULL: 8 for every group
 *   bias   : [n] fp32, or NULL;   out: [m, n] in out_dtype
 * group is 32, 64 or 128 and divides k; n < 2^28 - 1024, k < 2^31 - 1024,
 * m at most 327675.  The kernel is made for up to about 64 rows, past which the codes are read again for every 64 (fp32
 * x: 21).  Above 16 rows (5) x is laid out in a workspace of about 2 m k bytes (6) on
 * `stream`.  Sums are fp32; x enters the matrix cores exactly (fp32 as three bf16
 * terms, in magnitude up to 3.38e38, bf16's largest).  A value of x that is not finite makes its row's outputs NaN.  With
 * k = 0, out is the bias (or 0).
 */
ssm_status ssm_q4_matvec(const void* x, int64_t x_row, const uint8_t* codes, const void* scales, const uint8_t* zeros,
                         const float* bias, void* out, int64_t m, int64_t n, int64_t k, int64_t group,
                         ssm_dtype in_dtype, ssm_dtype scale_dtype, ssm_dtype out_dtype, void* stream);

/*
 * Quantises w [n, k] (w_dtype) into that form: per group,
 * scale = (max(w, 0) - min(w, 0)) / 15 rounded to scale_dtype, zero = the nearest
 * code to -min / scale, code = the nearest to w / scale + zero, within 0..15.
 * |w - (code - zero) scale| is at most scale (half a step, and the rounding of
 * the zero point) up to scale_dtype's rounding.  Finite weights only, whose largest less
 * smallest in a group is finite too.
 */
ssm_status ssm_q4_quantize(const void* w, uint8_t* codes, void* scales, uint8_t* zeros, int64_t n, int64_t k,
                           int64_t group, ssm_dtype w_dtype, ssm_dtype scale_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSMBLOCK_H */
