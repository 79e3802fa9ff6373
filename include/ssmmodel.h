/*
 * ssmmodel.h -- C ABI of libssmscan, third part: what training a language model of
 * recurrent layers needs besides its scans (ssmscan.h) and what stands around them
 * (ssmblock.h): a recurrence with one state for each channel, and the losses at its end.
 *
 *   ssm_gscan_*    gated linear recurrence for each channel
 *   ssm_xent_*     softmax cross entropy against a large vocabulary, from the
 *                  rows and the vocabulary's weights, without storing the logits
 *   ssm_distill_*  the same for a teacher's top logits
 *
 * Ownership, errors, asynchrony, graph capture and workspaces (ssm_workspace) are
 * those of ssmblock.h.  Results are bitwise reproducible: no sum depends on the
 * order in which workgroups run.
 */
#ifndef SSMMODEL_H
#define SSMMODEL_H

#include "ssmblock.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gated linear recurrence, for each channel d of each batch row:
 *
 *   a_t = exp(-rate[d] sigmoid(r_t))          or, with rate NULL, sigmoid(r_t)
 *   m_t = sqrt(1 - a_t^2)                     or, with SSM_GSCAN_LERP, 1 - a_t
 *   h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t  or, with i NULL, a_t h_{t-1} + m_t x_t
 *   out_t = h_t
 *
 *   x, r, i      : [batch, seqlen, width] in in_dtype; token (b, t)'s values start
 *                  (b * seqlen + t) * x_row (r_row, i_row) elements after the first
 *                  token's (slices of a packed projection; rows may not overlap, and are
 *                  at most 2^24 elements apart)
 *   rate         : [width] fp32 or NULL; meant to be >= 0 (below, a > 1, and without
 *                  SSM_GSCAN_LERP m is NaN; with it, where the product of the decays of up to
 *                  16 tiles leaves fp32's range, a state of 0 stays 0 and others are infinite)
 *   initial_state, last_state: [batch, width] fp32, each NULL for zero or not stored;
 *                  last_state may be initial_state (in place)
 *   out          : [batch, seqlen, width] in out_dtype
 *   states       : [batch, ceil(seqlen / SSM_GSCAN_SEGMENT), width] fp32 or NULL: the
 *                  state before step 0, SSM_GSCAN_SEGMENT, 2 SSM_GSCAN_SEGMENT, ..,
 *                  which the gradients need
 * States, gates and sums are fp32.  1 - a and 1 - a^2 are formed without cancellation.
 * A value that is not finite reaches its channel's later steps only.
 * Workspace, where a sequence is longer than one tile of SSM_GSCAN_TILE steps: about
 * 9 bytes for every tile and channel of a batch row, channels counted in 128s.  width at
 * most 2^24, batch * width at most 2^31 - 1024, and
 * batch * ceil(width / 64) * ceil(seqlen / 64) at most 2^23 - 2.
 */
#define SSM_GSCAN_LERP 1
#define SSM_GSCAN_SEGMENT 32
#define SSM_GSCAN_TILE 128

ssm_status ssm_gscan_fwd(const void* x, int64_t x_row, const void* r, int64_t r_row, const void* i, int64_t i_row,
                         const float* rate, int flags, const float* initial_state, void* out, float* last_state,
                         float* states, int64_t batch, int64_t seqlen, int64_t width, ssm_dtype in_dtype,
                         ssm_dtype out_dtype, void* stream);

/*
 * Its gradients, from the forward's inputs and states, dout [batch, seqlen, width] in
 * out_dtype and, optionally, dlast_state = dL/dlast_state [batch, width] fp32.  With
 * g_t = dout_t + a_{t+1} g_{t+1} (g = dlast_state behind the last step) and
 * e_t = g_t (a_t h_{t-1} + u_t dm_t/dlog a_t), u_t = sigmoid(i_t) x_t:
 *   dx = g m sigmoid(i);  di = g m x sigmoid(i) (1 - sigmoid(i));  dr = e dlog a/dr
 *   drate[d] = -sum e sigmoid(r) over batch and steps;  dinitial_state = a_0 g_0
 * dm/dlog a is -a, or -a^2 / m, taken as 0 where m is 0 (there m has no derivative).
 *   dx, dr, di : [batch, seqlen, width] in in_dtype, contiguous; di iff i is given
 *   drate      : [width] fp32, or NULL (not computed; iff rate is NULL it has to be)
 *   dinitial_state: [batch, width] fp32, or NULL
 * Workspace: as for the forward with tiles half as long, and 4 bytes for every such tile
 * and channel of a batch row (and for up to 64 tiles more) where drate is computed.
 */
ssm_status ssm_gscan_bwd(const void* x, int64_t x_row, const void* r, int64_t r_row, const void* i, int64_t i_row,
                         const float* rate, int flags, const float* states, const void* dout,
                         const float* dlast_state, void* dx, void* dr, void* di, float* drate, float* dinitial_state,
                         int64_t batch, int64_t seqlen, int64_t width, ssm_dtype in_dtype, ssm_dtype out_dtype,
                         void* stream);

/*
 * One token for every (b, d).  state, state_out: [batch, width] fp32, one buffer (in
 * place) or two; x, r, i, out: [batch, width], rows of x, r and i x_row, r_row and i_row
 * elements apart.  width at most 2^24, batch * width at most 2^31 - 1024.
 */
ssm_status ssm_gscan_update(const float* state, float* state_out, const void* x, int64_t x_row, const void* r,
                            int64_t r_row, const void* i, int64_t i_row, const float* rate, int flags, void* out,
                            int64_t batch, int64_t width, ssm_dtype in_dtype, ssm_dtype out_dtype, void* stream);

/*
 * Softmax cross entropy of rows against a vocabulary, z = scale x weight^T:
 *
 *   lse[t]  = log sum_v exp(z[t,v])
 *   loss[t] = lse[t] - z[t, target[t]] + z_loss lse[t]^2
 *
 * The logits are not stored: the forward keeps a maximum and a sum for every tile of
 * columns of a row, and the gradients compute the logits again, a piece of the
 * vocabulary at a time.
 *   x      : [rows, width] bf16, rows x_row elements apart
 *   weight : [vocab, width] bf16, rows w_row elements apart
 *   target : [rows] int64.  A negative target is none: its loss is 0, and its row
 *            takes no part in the gradients, whatever x holds there.  One of vocab
 *            or more makes the loss NaN and takes no part in the gradients.
 *   loss, lse: [rows] fp32 (lse of every row, with a target or without)
 * width a multiple of 8 up to SSM_VOCAB_MAX_WIDTH; x and weight 16-byte aligned, their rows a
 * multiple of 8 elements apart, at most 2^22; rows at most 2^22, vocab from 1 to 2^30, x and
 * weight of at most 2^37 elements, and at most 2^22 tiles of 256 rows by 256 columns.
 * Logits and sums are fp32.  Workspace: 8 bytes for every row and 256 columns, or 128
 * where tiles are few, and 4 for every row; up to 16 rows of at most 4096: 8 bytes for every
 * row and wavefront of the device.
 */
#define SSM_VOCAB_MAX_WIDTH 65536
ssm_status ssm_xent_fwd(const void* x, int64_t x_row, const void* weight, int64_t w_row, const int64_t* target,
                        float scale, float z_loss, float* loss, float* lse, int64_t rows, int64_t width,
                        int64_t vocab, ssm_dtype in_dtype, void* stream);

/*
 * Its gradients for dloss [rows] fp32 (what arrives at each loss) and the forward's lse:
 *   dz[t,v] = dloss[t] scale (softmax(z)[t,v] (1 + 2 z_loss lse[t]) - [v = target[t]])
 *   dx = dz weight [rows, width];  dweight = dz^T x [vocab, width]   (bf16, each NULL
 *   if not wanted, contiguous, 16-byte aligned)
 * dz is rounded to bf16 for its two products, whose sums are fp32: off by at most 2^-8 of
 * each of their terms, and 2^-8 of the result for the result's own rounding.
 * Workspace: dz of a piece of the vocabulary, 2 rows v bytes with v columns of it, where
 * v is chosen so that this is at most SSM_VOCAB_PIECE_BYTES or v at most 8192; 16 bytes a
 * row; where dweight is wanted a copy of x, 2 rows width; where dx is the sum of several
 * pieces its fp32 sums, 4 rows width; and where tiles are few such sums of up to 64 slices
 * of dx and 16 of dweight.
 */
#define SSM_VOCAB_PIECE_BYTES 268435456
ssm_status ssm_xent_bwd(const float* dloss, const void* x, int64_t x_row, const void* weight, int64_t w_row,
                        const int64_t* target, float scale, float z_loss, const float* lse, void* dx, void* dweight,
                        int64_t rows, int64_t width, int64_t vocab, ssm_dtype in_dtype, void* stream);

/*
 * Distillation from a teacher's top logits.  With q[t] the softmax of the row's top
 * teacher logits over the temperature and p[t] the softmax of z / temperature over the
 * whole vocabulary:
 *
 *   loss[t] = temperature^2 sum_k q[t,k] (log q[t,k] - log p[t, index[t,k]])
 *
 *   index  : [rows, top] int64, places in the vocabulary.  A negative one is none: its
 *            teacher logit does not count.  One of vocab or more makes the row's loss
 *            NaN, and the row takes no part in the gradients.  The same index twice
 *            counts twice, its q added.
 *   teacher: [rows, top] fp32 logits; minus infinity is q = 0, as none
 *   loss   : [rows];  lse: [rows], log sum exp of z / temperature;  logits: [rows, top],
 *            z / temperature at the indices (0 where there is none): the gradients need
 *            both.  All fp32.
 * A row without any index has loss 0 and no part in the gradients, whatever x
 * holds there.  top from 1 to SSM_DISTILL_MAX_TOP, temperature positive
 * with a normal square; the rest as for ssm_xent_fwd, and where rows,
 * tiles of columns and top are many 8 rows top bytes more of workspace, and 2 for every row and tile.
 */
#define SSM_DISTILL_MAX_TOP 1024
ssm_status ssm_distill_fwd(const void* x, int64_t x_row, const void* weight, int64_t w_row, const int64_t* index,
                           const float* teacher, float scale, float temperature, float* loss, float* lse,
                           float* logits, int64_t rows, int64_t width, int64_t vocab, int64_t top, ssm_dtype in_dtype,
                           void* stream);

/*
 * Its gradients with respect to x and weight (the teacher gets none):
 *   dz[t,v] = dloss[t] temperature scale (p[t,v] - sum_{k: index[t,k] = v} q[t,k])
 * The rest as for ssm_xent_bwd; workspace also 4 rows top bytes.
 */
ssm_status ssm_distill_bwd(const float* dloss, const void* x, int64_t x_row, const void* weight, int64_t w_row,
                           const int64_t* index, const float* teacher, float scale, float temperature,
                           const float* lse, const float* logits, void* dx, void* dweight, int64_t rows,
                           int64_t width, int64_t vocab, int64_t top, ssm_dtype in_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSMMODEL_H */
