// Copies of activations whose rows the gated delta rule's kernels cannot read as
// they are (off 16-byte vectors, overlapping, or too far apart): contiguous, each
// row's end filled with zeros up to whole vectors.
#include <hip/hip_runtime.h>

#include "launch_delta.hpp"
#include "selective.hpp"

namespace cls {
namespace {

template <typename T>
__global__ __launch_bounds__(256) void delta_pack_kernel(const T* from, T* to, int64_t n, int64_t L, int heads, int dim,
                                                         int padded, int64_t batch, int64_t token, int64_t head) {
    for (int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x; at < n; at += int64_t(gridDim.x) * 256) {
        const int d = int(at % padded);
        const int64_t row = at / padded, h = row % heads, t = row / heads % L, b = row / heads / L;
        to[at] = d < dim ? from[b * batch + t * token + h * head + d] : T(0);
    }
}

}  // namespace
}  // namespace cls

int cls_delta_pack_launch(const void* from, void* to, int64_t size, int64_t batch, int64_t L, int64_t heads, int64_t dim,
                          int64_t padded, int64_t sb, int64_t st, int64_t sh, hipStream_t stream) {
    const int64_t n = batch * L * heads * padded, want = (n + 255) / 256;
    const unsigned wgs = unsigned(want < 65536 ? want : 65536);
    if (size == 4)
        cls::delta_pack_kernel<uint32_t><<<wgs, 256, 0, stream>>>(static_cast<const uint32_t*>(from), static_cast<uint32_t*>(to),
                                                                 n, L, int(heads), int(dim), int(padded), sb, st, sh);
    else
        cls::delta_pack_kernel<uint16_t><<<wgs, 256, 0, stream>>>(static_cast<const uint16_t*>(from), static_cast<uint16_t*>(to),
                                                                 n, L, int(heads), int(dim), int(padded), sb, st, sh);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}
