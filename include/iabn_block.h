/*
 * iabn_block.h -- row operators of libiabn.so for transformer blocks: the
 * norms before and after a block fused with its gate and residual scale, the
 * gated activation inside it, and 8-bit checkpoints with the backward passes
 * that read them.
 *
 * iabn.h's layers take their statistics over the batch, one pair a channel;
 * here they are one token's own, over the columns of its row.  What a layer
 * keeps for its backward is, as there, either the storage-type tensors that
 * the program holds anyway (the "standard" form), or the normalised value
 * alone (the "checkpointing" form of [ABN] section 3, "Proposed
 * Checkpointing"), here in 8 bits.
 *
 * A tensor [rows, cols] holds one token a row.  Conventions of iabn.h hold:
 * device pointers, nothing allocated, work ordered on `stream`, arguments
 * checked on the host before anything is launched, gamma / beta / gate /
 * statistics / parameter gradients float32, arithmetic float32 with one
 * round-to-nearest-even for each element written.  They differ in this:
 *   - Tensors need only their element's alignment (IABN_ERR_MISALIGNED
 *     otherwise).  Widths that are multiples of 8 on 16-byte boundaries take
 *     the faster, vectorised path.
 *   - rows = 0 is valid: nothing is read, and gradients that sum over rows
 *     are written as zeros.
 *   - An output in the storage type may be the same tensor as an input in it
 *     (same start, same row stride), which it then overwrites; any other
 *     overlap of an output (codes, scales, statistics, parameter gradients and
 *     the workspace's needed bytes included) with an input or output is
 *     IABN_ERR_INVALID_ARG.  Tensors of different row strides count as
 *     overlapping where their ranges meet.
 *   - Calls keep no state: a workspace needs no clearing and may serve any
 *     calls that do not run at the same time.  All can be captured into a
 *     CUDA graph.
 *   - The same call gives the same bits every time.
 *   - A row's NaN or infinity stays in that row's outputs (and in the sums
 *     over rows).
 */
#ifndef IABN_BLOCK_H
#define IABN_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "iabn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * 8-bit checkpoints.  A [rows, cols] tensor is kept as one byte an element
 * and one float32 scale for every IABN_Q8_GROUP columns of a row (the last
 * group of a row may be shorter): codes [rows, cols], scales
 * [rows, ceil(cols / IABN_Q8_GROUP)], both contiguous.  With amax the group's
 * largest magnitude and Q the format's (448 or 127),
 *   scale = amax * (1 / Q),  code = round_to_nearest_even(x * (Q / amax)),
 *   value = code * scale,
 * 1 / Q, Q / amax and the three products each rounded to float32 (so scale may
 * be the float next to amax / Q).
 * A group whose amax is below 2^-110 is kept as zeros with scale 0.  A group
 * that holds a NaN or an infinity gets the scale NaN, so that all its values
 * read back as NaN.
 *   IABN_Q8_E4M3  4-bit exponent, 3-bit mantissa: a value's error is at most
 *                 2^-4 of itself (or scale * 2^-10 where that is more).
 *   IABN_Q8_INT8  a value's error is at most scale / 2: the finer one where a
 *                 group's values are of one size.
 * (Either error by itself; the five roundings to float32 add up to 2^-13 of it.)
 * ------------------------------------------------------------------------ */
typedef enum { IABN_Q8_E4M3 = 0, IABN_Q8_INT8 = 1 } iabn_q8;
#define IABN_Q8_GROUP 128

/* Keeps x [rows, cols] (storage type `dtype`, row stride ldx >= cols elements)
 * in 8 bits: q and scale are written.  cols >= 1. */
iabn_status iabn_checkpoint8_store(int64_t rows, int64_t cols, int64_t ldx, int32_t dtype,
                                   int32_t format, const void* x, void* q, float* scale,
                                   void* stream);

/* Reads it back: y = value, or gamma*value + beta by column, into y
 * [rows, cols] with row stride ldy >= cols.  gamma, beta [cols]: either may
 * be NULL (1 and 0).  With the codes of xhat this gives the input of the
 * block's first product again, as iabn_checkpoint_recompute does for z. */
iabn_status iabn_checkpoint8_load(int64_t rows, int64_t cols, int64_t ldy, int32_t dtype,
                                  int32_t format, const void* q, const float* scale,
                                  const float* gamma, const float* beta, void* y, void* stream);

/* ------------------------------------------------------------------------
 * The block norm: everything between one block's last product and the next
 * block's first one, in one pass.  u [rows, cols] is the block's output, h
 * the residual stream, D = cols:
 *   uhat = post(u),  p = gamma_post*uhat + beta_post,
 *   h'   = residual_scale*h + gate*p,
 *   xhat = pre(h'),  n = gamma_pre*xhat + beta_pre.
 * post and pre are
 *   IABN_NORM_NONE   the value itself (no gamma, no beta; pre: no n either),
 *   IABN_NORM_RMS    v*rstd,        rstd = 1/sqrt(sum v^2 / D + eps),
 *   IABN_NORM_LAYER  (v - mean)*rstd, rstd = 1/sqrt(sum (v - mean)^2 / D + eps).
 * gate is NULL (1), one row of D for all rows (rows_per_gate = 0), or one row
 * for every rows_per_gate rows: [ceil(rows / rows_per_gate), D], the row of a
 * token r being r / rows_per_gate (padded batches of equal length).
 * The pre-norm's statistics are those of h' before it is rounded.
 * ------------------------------------------------------------------------ */
typedef enum { IABN_NORM_NONE = 0, IABN_NORM_RMS = 1, IABN_NORM_LAYER = 2 } iabn_norm;

/* Largest cols of the block norm (IABN_ERR_UNSUPPORTED above). */
#define IABN_BLOCK_MAX_COLS 32768

typedef struct {
    int64_t rows, cols;
    int64_t rows_per_gate;   /* 0: one gate row for all rows */
    int32_t dtype;           /* iabn_dtype of u, h, n and their gradients */
    int32_t post, pre;       /* iabn_norm */
    int32_t format;          /* iabn_q8 of the checkpoints (the checkpoint8 calls) */
    float residual_scale;    /* finite */
    float eps_post, eps_pre; /* >= 0 */
} iabn_block_desc;

/* Forward.
 * u        [rows, cols], or NULL for the norm of h alone (then post = NONE,
 *          gate = NULL, residual_scale = 1 and h_out = NULL).
 * h        [rows, cols].
 * h_out    [rows, cols] h', or NULL.  n [rows, cols]: NULL iff pre = NONE.
 *          One of the two at least.
 * gamma_post, beta_post [cols]: NULL for 1 and 0, and where post = NONE.
 * gamma_pre, beta_pre   [cols]: NULL for 1 and 0, and where pre = NONE.
 * mean_post, rstd_post, mean_pre, rstd_pre [rows]: written where not NULL
 *          (mean with LAYER only); what the backward takes.  All NULL:
 *          inference, down to one token.
 * Kept for iabn_block_norm_backward: u and h_out. */
iabn_status iabn_block_norm_forward(const iabn_block_desc* d, const void* u, const void* h,
                                    void* h_out, void* n, const float* gamma_post,
                                    const float* beta_post, const float* gate,
                                    const float* gamma_pre, const float* beta_pre,
                                    float* mean_post, float* rstd_post, float* mean_pre,
                                    float* rstd_pre, void* stream);

/* The same, keeping uhat and xhat in 8 bits: q_post / scale_post and q_pre /
 * scale_pre, each pair NULL where it is not wanted (xhat's with pre = NONE
 * must be).  rstd_post, rstd_pre [rows]: written where not NULL. */
iabn_status iabn_block_norm_forward_checkpoint8(
    const iabn_block_desc* d, const void* u, const void* h, void* h_out, void* n,
    const float* gamma_post, const float* beta_post, const float* gate, const float* gamma_pre,
    const float* beta_pre, float* rstd_post, float* rstd_pre, void* q_post, float* scale_post,
    void* q_pre, float* scale_pre, void* stream);

/* Bytes of workspace of the two backward calls (a multiple of 256; depends on
 * rows, cols and rows_per_gate); 0 if they are invalid.  Host-only: the sums
 * over rows are laid out for the 148 SMs of a B200, whatever the device.
 * Every gate row keeps two rows of float32 sums there, 8 * cols bytes, so gates
 * are meant to cover many rows: 16384 x 4096 bf16 from codes takes 129 us with
 * one gate row, 370 us with one for every 64 rows and, with one a row, 11 ms and
 * 0.56 GB of workspace. */
size_t iabn_block_norm_workspace_size(const iabn_block_desc* d);

/* Backward, from the kept u and h_out and the forward's statistics.
 *   g = dn*gamma_pre,
 *   t = dh_out + rstd_pre*(g - [LAYER] mean(g) - xhat*mean(g*xhat)),
 *   dh = residual_scale*t,
 *   e = t*gate*gamma_post,
 *   du = rstd_post*(e - [LAYER] mean(e) - uhat*mean(e*uhat))   (post = NONE: e),
 *   dgamma_pre = sum dn*xhat,        dbeta_pre = sum dn,
 *   dgamma_post = sum t*gate*uhat,   dbeta_post = sum t*gate,
 *   dgate = sum over its rows of t*p,
 * means over a row, sums over rows.
 * u        needed where post != NONE or dgate is wanted, else NULL or unread.
 * h_out    needed where pre != NONE.
 * dh_out   dL/dh', or NULL (0).  dn: dL/dn, NULL iff pre = NONE.  One of the
 *          two at least.
 * dh, du   [rows, cols], written; du NULL: not wanted.
 * mean_*   with LAYER, rstd_* with RMS and LAYER: the forward's.
 * gate, gamma_post, beta_post, gamma_pre: the forward's (beta_post is read for
 *          dgate only).
 * dgamma_post, dbeta_post, dgamma_pre, dbeta_pre [cols], dgate (as gate):
 *          written, each NULL where it is not wanted; those of an absent norm
 *          or gate must be NULL.
 * workspace: iabn_block_norm_workspace_size(d) bytes on a 16-byte boundary. */
iabn_status iabn_block_norm_backward(
    const iabn_block_desc* d, const void* u, const void* h_out, const void* dh_out,
    const void* dn, void* dh, void* du, const float* gamma_post, const float* beta_post,
    const float* gate, const float* gamma_pre, const float* mean_post, const float* rstd_post,
    const float* mean_pre, const float* rstd_pre, float* dgamma_post, float* dbeta_post,
    float* dgate, float* dgamma_pre, float* dbeta_pre, void* workspace, size_t ws_bytes,
    void* stream);

/* The same, from the 8-bit checkpoints: uhat and xhat are the values that
 * q_post / scale_post and q_pre / scale_pre stand for. */
iabn_status iabn_block_norm_backward_checkpoint8(
    const iabn_block_desc* d, const void* q_post, const float* scale_post, const void* q_pre,
    const float* scale_pre, const void* dh_out, const void* dn, void* dh, void* du,
    const float* gamma_post, const float* beta_post, const float* gate, const float* gamma_pre,
    const float* rstd_post, const float* rstd_pre, float* dgamma_post, float* dbeta_post,
    float* dgate, float* dgamma_pre, float* dbeta_pre, void* workspace, size_t ws_bytes,
    void* stream);

/* ------------------------------------------------------------------------
 * The gated activation: z = phi(a)*b.
 *   IABN_GLU_SILU       phi(a) = a*s(a), s the logistic function
 *   IABN_GLU_GELU       phi(a) = a*(1 + erf(a/sqrt 2))/2
 *   IABN_GLU_GELU_TANH  phi(a) = a*(1 + tanh(sqrt(2/pi)*(a + 0.044715 a^3)))/2
 * a and b share a row stride (two halves of one [rows, 2*cols] product), so
 * do da and db; z and dz are contiguous.
 * ------------------------------------------------------------------------ */
typedef enum { IABN_GLU_SILU = 0, IABN_GLU_GELU = 1, IABN_GLU_GELU_TANH = 2 } iabn_glu;

typedef struct {
    int64_t rows, cols;
    int64_t ld;        /* row stride of a and b */
    int64_t ld_grad;   /* row stride of da and db */
    int32_t dtype;     /* iabn_dtype of a, b, z and their gradients */
    int32_t act;       /* iabn_glu */
    int32_t format;    /* iabn_q8 of the checkpoints (the checkpoint8 calls) */
} iabn_gated_desc;

/* z = phi(a)*b. */
iabn_status iabn_gated_forward(const iabn_gated_desc* d, const void* a, const void* b, void* z,
                               void* stream);

/* The same, keeping a and b in 8 bits. */
iabn_status iabn_gated_forward_checkpoint8(const iabn_gated_desc* d, const void* a,
                                           const void* b, void* z, void* qa, float* scale_a,
                                           void* qb, float* scale_b, void* stream);

/* da = dz*b*phi'(a), db = dz*phi(a); z again where z_out is not NULL (the
 * input of the block's last product, for its weights' gradient). */
iabn_status iabn_gated_backward(const iabn_gated_desc* d, const void* a, const void* b,
                                const void* dz, void* da, void* db, void* z_out, void* stream);

/* The same from the 8-bit checkpoints (d->ld is not read). */
iabn_status iabn_gated_backward_checkpoint8(const iabn_gated_desc* d, const void* qa,
                                            const float* scale_a, const void* qb,
                                            const float* scale_b, const void* dz, void* da,
                                            void* db, void* z_out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* IABN_BLOCK_H */
