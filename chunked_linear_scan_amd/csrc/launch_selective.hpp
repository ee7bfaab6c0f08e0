// Launch interface between selective_api.cpp (checks, sizes) and the kernels
// of the selective scan, the short convolution and the state cache.  All
// arguments are validated.  Each returns 0, or -7 when a launch fails.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/selective_scan.h"

namespace cls {
struct ScanParams;
}

int cls_selective_scan_fwd_launch(const cls::ScanParams& p, int dtype, hipStream_t stream);
int cls_selective_scan_bwd_launch(const cls::ScanParams& p, int dtype, hipStream_t stream);
// The workgroups of 256 that the step's launch has.
int64_t cls_selective_scan_step_groups(const selective_scan_inputs& in);
int cls_selective_scan_step_launch(const selective_scan_inputs& in, float* h, void* y, hipStream_t stream);

// The most partial sums of weight gradients that short_conv_bwd adds up (rows of its workspace).
int64_t cls_short_conv_bwd_parts(int64_t batch, int64_t seqlen, int64_t channels);
int cls_short_conv_fwd_launch(const short_conv_inputs& in, void* y, void* final_state, hipStream_t stream);
int cls_short_conv_bwd_launch(const short_conv_inputs& in, const void* dy, int64_t dy_batch, int64_t dy_token,
                              const void* dfinal, void* dx, float* dweight, float* dbias, void* dinitial, float* parts,
                              hipStream_t stream);
int cls_short_conv_step_launch(const short_conv_inputs& in, void* state, void* y, hipStream_t stream);

int cls_state_cache_write_launch(const float* h, const int32_t* slots, int64_t batch, int64_t rows, int64_t S,
                                 int64_t nslots, int format, void* cache, float* scales, hipStream_t stream);
int cls_state_cache_read_launch(const void* cache, const float* scales, const int32_t* slots, int64_t batch,
                                int64_t rows, int64_t S, int64_t nslots, int format, float* h, hipStream_t stream);
