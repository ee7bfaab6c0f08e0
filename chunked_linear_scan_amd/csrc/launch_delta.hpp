// Launch interface between delta_api.cpp (checks, sizes) and the kernels of the
// gated delta rule and of the norms.  All arguments are validated.  Each
// returns 0, or -7 when a launch fails.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gated_delta.h"

namespace cls {
struct DeltaParams;
}

int cls_delta_pack_launch(const void* from, void* to, int64_t size, int64_t batch, int64_t L, int64_t heads, int64_t dim,
                          int64_t padded, int64_t sb, int64_t st, int64_t sh, hipStream_t stream);
int cls_delta_prep_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream);
int cls_delta_size_launch(const cls::DeltaParams& p, hipStream_t stream);
int cls_delta_fwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream);
int cls_delta_bwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream);
int cls_delta_grad_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream);
// Workgroups of 256 threads that a step of `heads` states (of all sequences) launches.
int64_t cls_delta_step_groups(int64_t heads, int64_t dk, int64_t dv);
int cls_delta_step_launch(const gated_delta_inputs& in, float* h, void* y, hipStream_t stream);

// The partial sums of parameters' gradients: rows of a norm's backward workspace.
int64_t cls_norm_parts(int64_t rows, int64_t dim);
// The forward pass without dy (y, and rstd where it is given, are written), the backward pass with it.
int cls_gated_norm_launch(const gated_norm_inputs& in, const void* dy, int64_t dy_row, int64_t dy_head, float* rstd,
                          void* y, void* dx, void* dz, float* dweight, float* parts, hipStream_t stream);
int cls_residual_norm_fwd_launch(const residual_norm_inputs& in, void* y, void* r, float* rstd, hipStream_t stream);
int cls_residual_norm_bwd_launch(const residual_norm_inputs& in, const residual_norm_grads& g, float* parts,
                                 hipStream_t stream);
