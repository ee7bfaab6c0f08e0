/*
 * chunked_linear_scan — the gated delta rule and the norms around its block.
 * The third recurrence beside the SSD pass and the selective scan: its state
 * is corrected by what it answers wrongly for a key, not only added to.  For
 * prompts (forward, in chunks), for training (backward) and for single tokens
 * (step); and the two norms of a layer with any of the three recurrences: the
 * gated one behind it, and the one that joins the residual stream in front of
 * the next block.
 *
 * The rules of selective_scan.h hold here too: plain device pointers on the
 * current device, all work on `stream`, nothing synchronises or allocates,
 * arguments are checked on the host before anything is launched, workspaces
 * need no initial contents and keep nothing, pointers are aligned to their
 * element (states of the step, workspaces and checkpoints to 16 bytes), strides
 * are in elements and >= 0, no kernel uses atomics.
 */
#ifndef GATED_DELTA_H
#define GATED_DELTA_H

#include <stddef.h>
#include <stdint.h>

#include "chunked_linear_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gated delta rule, per sequence and head h, with the key head h / (heads / kheads):
 *     S_t = e^{g_t} S_{t-1} + beta_t (v_t - e^{g_t} S_{t-1} k_t) k_t^T
 *     y_t = scale S_t q_t
 * from S_{-1} = h0; S is [dv, dk] as the SSD pass has its state [headdim, dstate].
 *
 * Layouts:
 *   q, k      [batch, seqlen, kheads, dk]   dtype, strided (dk adjacent)
 *   v         [batch, seqlen, heads, dv]    dtype, strided (dv adjacent)
 *   g, beta   [batch, seqlen, heads]        fp32, strided (heads adjacent)
 *   h0        [batch, heads, dv, dk]        fp32, contiguous (NULL = zeros)
 *   seqlens   [batch]                       int32 (NULL = all of length seqlen)
 *   y         [batch, seqlen, heads, dv]    dtype, contiguous
 *   h_final   [batch, heads, dv, dk]        fp32 (NULL = not written)
 *   checkpoints: what gated_delta_bwd needs of the forward pass, of
 *             gated_delta_checkpoint_size bytes (NULL = not written)
 * g is a logarithm (usually <= 0; -infinity forgets the state at that token).
 * The rule is stable for |k| = 1 and beta in 0..2; other values are evaluated
 * as they are.  The tokens of sequence b at or past seqlens[b] (taken into
 * 0..seqlen) are padding, whatever they hold: their outputs and gradients are
 * zeros, and the final state is that before them.
 *
 * Tokens are taken gated_delta_chunk(dtype) at a time through matrix products.
 * States, their updates and all sums are fp32; with 16-bit elements a computed
 * operand of a product goes in as the sum of two numbers of that type (bf16: 16
 * bits in all).  With SSD_F16 such operands have that type's range.  States,
 * corrections of values and products of a chunk's keys and queries go in at their
 * own size: what they reach is not finite where they are past 65504, and they are
 * held to 2^-25 at best, so below 2^-3 they have fewer good bits than 22.
 * Gradients go in times a power of two, one for each sequence and head, that takes
 * the largest of |scale dy| and |dh_final| to 4..8: any size of those gives the
 * same bits behind the exponent, but a gradient of a state or of corrections that
 * grows to 8000 times the largest is not finite.
 * A value that is not finite reaches its head's outputs from the start of its
 * chunk on, one of dy its head's gradients up to the end of its chunk.
 *
 * heads is a multiple of kheads; dk is 1..256 and dv 1..65536
 * (SSD_ERR_UNSUPPORTED above).  SSD_ERR_SHAPE, too, for batch or heads above
 * 2^20, seqlen above 2^30, heads * dv (dv to whole vectors) or kheads * 256 above
 * 2^23, strides above 2^40, and where a launch would have 2^32 threads or more
 * (512 for each 32 of dv, head and sequence; 256 for each chunk, head and
 * sequence; with gradients and heads > kheads one for each element of q).
 */
typedef struct {
    int64_t batch, seqlen, kheads, heads, dk, dv;
    int32_t dtype; /* of q, k, v, y and their gradients */
    float scale;
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    const float* h0;
    const int32_t* seqlens;
    /* strides of one sequence, one token and one head */
    int64_t q_batch, q_token, q_head, k_batch, k_token, k_head, v_batch, v_token, v_head;
    int64_t g_batch, g_token, beta_batch, beta_token;
} gated_delta_inputs;

/* Tokens of a chunk: 64, with SSD_F32 32. */
int64_t gated_delta_chunk(int dtype);

/* Bytes of workspace for a forward or a backward call, and of the checkpoints
 * (0 for sizes that are refused).  They depend on the strides and pointers of q,
 * k and v, too: rows that are not whole 16-byte vectors, and tokens less than a
 * row or more than 2^23 elements apart, are copied into the workspace first. */
size_t gated_delta_workspace_size(const gated_delta_inputs* in);
size_t gated_delta_bwd_workspace_size(const gated_delta_inputs* in);
size_t gated_delta_checkpoint_size(const gated_delta_inputs* in);

int gated_delta_fwd(const gated_delta_inputs* in, void* y, float* h_final, void* checkpoints,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of gated_delta_fwd's y (and h_final) for the same inputs, with the
 * checkpoints that the forward pass wrote for them.
 *   dy        [batch, seqlen, heads, dv]   dtype, strided
 *   dh_final  [batch, heads, dv, dk]       fp32 (NULL = 0)
 * Written, contiguous: dq, dk (as q; summed over the heads of a key head), dv
 * in dtype; dg, dbeta [batch, seqlen, heads] fp32; dh0 as h0 (NULL = not written).
 * Where e^g is 0, dg is.
 */
typedef struct {
    const void* dy;
    int64_t dy_batch, dy_token, dy_head;
    const float* dh_final;
    const void* checkpoints;
    void* dq;
    void* dk;
    void* dv;
    float* dg;
    float* dbeta;
    float* dh0;
} gated_delta_grads;

int gated_delta_bwd(const gated_delta_inputs* in, const gated_delta_grads* g, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * One token for every sequence: the state h [batch, heads, dv, dk] (fp32,
 * contiguous, 16-byte aligned where dk is a multiple of 4) is updated in place.
 * `in` is read with seqlen 1: its token strides, h0 and seqlens are not used.
 * y [batch, heads, dv], contiguous.  All arithmetic is fp32.  Sizes are bounded
 * by this launch's threads alone: 256 for each 128, 64, 32 or 16 rows of a state
 * with dk up to 32, 64, 128 or 256.
 */
int gated_delta_step(const gated_delta_inputs* in, float* h, void* y, void* stream);

/*
 * Norm of each row by its root mean square, with a gate: for `rows` tokens of
 * `heads` rows of `dim` values,
 *     gate_first = 0:  y = (x rstd) weight silu(z),      rstd = 1 / sqrt(mean(x^2) + eps)
 *     gate_first = 1:  y = (u rstd) weight, u = x silu(z), rstd = 1 / sqrt(mean(u^2) + eps)
 * (without z: y = x rstd weight).
 *   x, z    [rows, heads, dim]  dtype, strided (dim adjacent; z may be NULL)
 *   weight  [dim]               fp32 (NULL = ones)
 *   y       [rows, heads, dim]  dtype, contiguous
 *   rstd    [rows, heads]       fp32: for the gradients (NULL = not written)
 * dim is 1..16384 (SSD_ERR_UNSUPPORTED above); SSD_ERR_SHAPE where rows * heads is above 2^31 - 1.
 */
typedef struct {
    int64_t rows, heads, dim;
    int32_t dtype;
    int32_t gate_first;
    float eps;
    const void* x;
    const void* z;
    const float* weight;
    int64_t x_row, x_head, z_row, z_head;
} gated_norm_inputs;

int gated_norm_fwd(const gated_norm_inputs* in, void* y, float* rstd, void* stream);

/* Its gradients from dy [rows, heads, dim] (strided) and the forward pass's
 * rstd: dx, dz (with z) in dtype, contiguous; dweight [dim] fp32 (NULL = not written). */
size_t gated_norm_bwd_workspace_size(int64_t rows, int64_t heads, int64_t dim);

int gated_norm_bwd(const gated_norm_inputs* in, const void* dy, int64_t dy_row, int64_t dy_head, const float* rstd,
                   void* dx, void* dz, float* dweight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The residual stream and the norm in front of the next block, of `rows` rows:
 *     r = residual + scale * x,   y = (r rstd) weight,   rstd = 1 / sqrt(mean(r^2) + eps)
 * where the norm sees r as it is kept, rounded to its type.
 *   x             [rows, dim]  dtype, strided (dim adjacent)
 *   residual      [rows, dim]  stream_dtype (SSD_F32 or dtype), strided (NULL = zeros)
 *   scale         [dim]        fp32 (NULL = ones)
 *   weight        [dim]        fp32 (NULL = ones)
 *   r             [rows, dim]  stream_dtype, contiguous
 *   y             [rows, dim]  dtype, contiguous
 *   rstd          [rows]       fp32 (NULL = not written)
 * dim is 1..16384 (SSD_ERR_UNSUPPORTED above); rows at most 2^31 - 1.
 */
typedef struct {
    int64_t rows, dim;
    int32_t dtype, stream_dtype;
    float eps;
    const void* x;
    const void* residual;
    const float* scale;
    const float* weight;
    int64_t x_row, residual_row;
} residual_norm_inputs;

int residual_norm_fwd(const residual_norm_inputs* in, void* y, void* r, float* rstd, void* stream);

/*
 * Its gradients from those of y and of r, with the forward pass's r and rstd
 * (`residual` and `eps` of `in` are not read; x only with dscale):
 *   dy  [rows, dim]  dtype, strided;  dr  [rows, dim]  stream_dtype, strided (NULL = zeros)
 *   r   [rows, dim]  stream_dtype, strided
 * Written, contiguous: dresidual (stream_dtype), dx (dtype), dweight [dim] and
 * dscale [dim] fp32 (each may be NULL but dresidual).
 */
typedef struct {
    const void* dy;
    const void* dr;
    const void* r;
    const float* rstd;
    int64_t dy_row, dr_row, r_row;
    void* dresidual;
    void* dx;
    float* dweight;
    float* dscale;
} residual_norm_grads;

size_t residual_norm_bwd_workspace_size(int64_t rows, int64_t dim);

int residual_norm_bwd(const residual_norm_inputs* in, const residual_norm_grads* g, void* workspace,
                      size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GATED_DELTA_H */
