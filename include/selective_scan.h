/*
 * chunked_linear_scan — the selective scan and what stands around it in a
 * layer: the short causal convolution in front of it, and an 8-bit cache for
 * the states that it and the SSD pass leave.  For prompts (forward), for
 * training (backward) and for single tokens (step).
 *
 * The rules of chunked_linear_scan.h hold here too: plain device pointers on
 * the current device, all work on `stream`, nothing synchronises or
 * allocates, arguments are checked on the host before anything is launched,
 * status codes SSD_OK / SSD_ERR_*.  Different from there:
 *   - workspaces need no initial contents and keep nothing from call to call;
 *     calls that may overlap need a workspace each;
 *   - activations may be slices of wider rows: each has a batch and a token
 *     stride (in elements, >= 0; the scan's token strides up to 2^26), its
 *     channels are adjacent;
 *   - pointers are aligned to their element (16-bit: 2 bytes, fp32: 4 bytes),
 *     not to 16 bytes; workspaces and checkpoints to 16 bytes.
 * No kernel uses atomics: results are the same from run to run.
 *
 * Element types (dtype): SSD_F32, SSD_BF16 or SSD_F16 for activations; A, D,
 * dt_bias, convolution weights and biases and all scan states are fp32.
 * Sums and states are held in fp32; an output is rounded to dtype once.
 *
 * seqlens (int32 [batch], device memory, or NULL = all of length seqlen):
 * the tokens of sequence b at or past seqlens[b] (taken into 0..seqlen) are
 * padding, whatever they hold: they take no step, their outputs and gradients
 * are written as zeros, and final states are those after the last token
 * before them.  A length of 0 leaves the state as it started.
 */
#ifndef SELECTIVE_SCAN_H
#define SELECTIVE_SCAN_H

#include <stddef.h>
#include <stdint.h>

#include "chunked_linear_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Selective scan: a decay for each channel and state.  With
 * dt' = softplus(dt + dt_bias) (or dt + dt_bias without softplus), per
 * sequence, channel d and state n, g = d / (channels / ngroups):
 *     h_t[d,n] = exp(dt'_t[d] A[d,n]) h_{t-1}[d,n] + dt'_t[d] B_t[g,n] u_t[d]
 *     y_t[d]   = (sum_n C_t[g,n] h_t[d,n] + D[d] u_t[d]) * silu(z_t[d])
 * from h_{-1} = h0; the factor silu(z) = z / (1 + exp(-z)) only with z.
 *
 * Layouts:
 *   u, dt, z   [batch, seqlen, channels]            dtype, strided (z may be NULL)
 *   B, C       [batch, seqlen, ngroups, dstate]     dtype, strided (states adjacent)
 *   A          [channels, dstate]                   fp32, contiguous
 *   D, dt_bias [channels]                           fp32 (each may be NULL = 0)
 *   h0         [batch, channels, dstate]            fp32, contiguous (NULL = zeros)
 *   y          [batch, seqlen, channels]            dtype, contiguous
 *   h_final    [batch, channels, dstate]            fp32 (NULL = not written)
 *   checkpoints: what selective_scan_bwd needs of the forward pass, of
 *              selective_scan_checkpoint_size bytes (NULL = not written): the
 *              state before every 8th token
 * dstate is 1..64 (SSD_ERR_UNSUPPORTED above), channels a multiple of
 * ngroups.  SSD_ERR_SHAPE, too, for batch or channels above 2^24, seqlen above
 * 2^30, batch * seqlen * channels above 2^40, channels * (dstate + 2) above
 * 2^30 - 2^22 - 64, and where the launch would pass 2^32 - 1 threads: one for
 * each four states, rounded up to a power of two, of each channel (a group's
 * rounded up to 64), sequence and, for long sequences that leave the device
 * nearly empty, segment.  Decays above 1 (A > 0) are evaluated as they are.  An input that is
 * not finite reaches its own channel's later outputs only (B and C: those of
 * their group), which it makes infinite or NaN.  Outputs must not alias inputs.
 */
typedef struct {
    int64_t batch, seqlen, channels, dstate, ngroups;
    int32_t dtype;    /* of u, dt, z, B, C, y and their gradients */
    int32_t softplus; /* 1: dt' = softplus(dt + dt_bias), 0: dt' = dt + dt_bias */
    const void* u;
    const void* dt;
    const void* z;
    const void* B;
    const void* C;
    const float* A;
    const float* D;
    const float* dt_bias;
    const float* h0;
    const int32_t* seqlens;
    /* strides in elements: of one sequence and of one token (B, C: and of one group) */
    int64_t u_batch, u_token, dt_batch, dt_token, z_batch, z_token;
    int64_t B_batch, B_token, B_group, C_batch, C_token, C_group;
} selective_scan_inputs;

/* Bytes of workspace for a forward or a backward call (0 where it needs none,
 * and for sizes that are refused). */
size_t selective_scan_workspace_size(int64_t batch, int64_t seqlen, int64_t channels,
                                     int64_t dstate, int64_t ngroups);
size_t selective_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t channels,
                                         int64_t dstate, int64_t ngroups);
size_t selective_scan_checkpoint_size(int64_t batch, int64_t seqlen, int64_t channels,
                                      int64_t dstate);

int selective_scan_fwd(const selective_scan_inputs* in, void* y, float* h_final,
                       void* checkpoints, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * Gradients of selective_scan_fwd's y (and h_final) for the same inputs, with
 * the checkpoints that the forward pass wrote for them.
 *   dy        [batch, seqlen, channels]  dtype, strided: the gradient of y
 *   dh_final  [batch, channels, dstate]  fp32: the gradient of h_final (NULL = 0)
 * Written (contiguous; each optional one may be NULL):
 *   du, ddt   [batch, seqlen, channels]         dtype
 *   dz        the same, where z is given (else ignored)
 *   dB, dC    [batch, seqlen, ngroups, dstate]  dtype: summed over the group's channels
 *   dA        [channels, dstate]  fp32, dD, ddt_bias [channels] fp32 (optional)
 *   dh0       [batch, channels, dstate] fp32 (optional)
 */
typedef struct {
    const void* dy;
    int64_t dy_batch, dy_token;
    const float* dh_final;
    const void* checkpoints;
    void* du;
    void* ddt;
    void* dz;
    void* dB;
    void* dC;
    float* dA;
    float* dD;
    float* ddt_bias;
    float* dh0;
} selective_scan_grads;

int selective_scan_bwd(const selective_scan_inputs* in, const selective_scan_grads* g,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token of the same recurrence for every sequence: the state h
 * [batch, channels, dstate] (fp32, contiguous, 16-byte aligned where dstate is a
 * multiple of 4) is updated in place.  `in` is read with seqlen 1: its token
 * strides, h0 and seqlens are not used.  y [batch, channels], contiguous.  Its
 * launch has a thread for each four states (rounded up to a power of two, four
 * sequences sharing one where there are many and dstate is above 8);
 * SSD_ERR_SHAPE where they would pass 2^32 - 1.
 */
int selective_scan_step(const selective_scan_inputs* in, float* h, void* y, void* stream);

/*
 * Short causal convolution of each channel over the tokens:
 *     p_t[d] = bias[d] + sum_{k=0..width-1} weight[d,k] x_{t-width+1+k}[d]
 *     y_t    = silu(p_t)  (silu = 1)   or  p_t  (silu = 0)
 * where the inputs before the first token are initial_state
 * [batch, width-1, channels] (oldest first; NULL = zeros).
 *   x            [batch, seqlen, channels]  dtype, strided
 *   weight       [channels, width]  fp32, width 2..4 (SSD_ERR_UNSUPPORTED else)
 *   bias         [channels]         fp32 (NULL = 0)
 *   y            as x, contiguous
 *   final_state  [batch, width-1, channels]  dtype: the last width-1 inputs
 *                (NULL = not written); it may not alias initial_state
 * SSD_ERR_SHAPE for batch or channels above 2^24, seqlen above 2^30, and where
 * batch * (ceil(seqlen / 4) + 1) is not below floor((2^32 - 256) / (channels + 64)).
 * Outputs must not alias inputs.
 */
typedef struct {
    int64_t batch, seqlen, channels, width;
    int32_t dtype;
    int32_t silu;
    const void* x;
    int64_t x_batch, x_token;
    const float* weight;
    const float* bias;
    const void* initial_state;
    const int32_t* seqlens;
} short_conv_inputs;

int short_conv_fwd(const short_conv_inputs* in, void* y, void* final_state, void* stream);

/*
 * Its gradients: dy [batch, seqlen, channels] (strided) of y, dfinal of
 * final_state (NULL = 0).  Written: dx (contiguous), dweight
 * [channels, width] and dbias [channels] (fp32, NULL = not written),
 * dinitial as initial_state (NULL = not written).  The workspace size is 0 for
 * sizes that are refused.
 */
size_t short_conv_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t channels, int64_t width);

int short_conv_bwd(const short_conv_inputs* in, const void* dy, int64_t dy_batch, int64_t dy_token,
                   const void* dfinal, void* dx, float* dweight, float* dbias, void* dinitial,
                   void* workspace, size_t workspace_bytes, void* stream);

/* One token for every sequence: state [batch, width-1, channels] (dtype,
 * contiguous) takes x in and drops its oldest row, in place.  `in` is read
 * with seqlen 1 (token stride, initial_state and seqlens not used); y
 * [batch, channels], contiguous. */
int short_conv_step(const short_conv_inputs* in, void* state, void* y, void* stream);

/*
 * A cache of fp32 states in 8 bits: snapshots of what ssd_fwd or
 * selective_scan_fwd ended with, to start from again later.  A state is
 * `rows` rows of `dstate` values; each row has one fp32 scale:
 *     m = max |h|,  scale = m / top,  q = round(h * (top / m)),  read: q * scale
 * with top 127 (SSD_I8: signed integers) or 448 (SSD_E4M3: 8-bit floats with
 * 4 exponent and 3 fraction bits, no infinities), ties to even, each step
 * rounded in fp32: the bytes are the same on every run and device.  Rows with
 * m < 2^-100 are held as zeros.  A row with an infinity or a NaN has a NaN
 * for its scale and is read back as NaN throughout.
 *   h       [batch, rows, dstate]   fp32, contiguous
 *   cache   [nslots, rows, dstate]  bytes, contiguous
 *   scales  [nslots, rows]          fp32, contiguous
 *   slots   [batch]                 int32, device memory: the slot of each state
 * dstate is 1..256 (SSD_ERR_UNSUPPORTED above); SSD_ERR_SHAPE from
 * batch * (rows + 256) = 2^26 or nslots = 2^31 on, and above
 * nslots * rows * dstate = 2^46.  Write: a state whose slot is outside 0..nslots-1 is not
 * written; where a slot is named more than once the last state that names it
 * is kept; all other slots stay as they are.  Read: a slot outside 0..nslots-1
 * gives a state of zeros, the start of a sequence without a snapshot.
 */
enum { SSD_I8 = 3, SSD_E4M3 = 4 };

int state_cache_write(const float* h, const int32_t* slots, int64_t batch, int64_t rows, int64_t dstate,
                      int64_t nslots, int format, void* cache, float* scales, void* stream);

int state_cache_read(const void* cache, const float* scales, const int32_t* slots, int64_t batch, int64_t rows,
                     int64_t dstate, int64_t nslots, int format, float* h, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SELECTIVE_SCAN_H */
