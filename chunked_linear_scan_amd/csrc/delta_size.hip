// Gated delta rule: how large a sequence's and head's gradients are, for the power
// of two that fp16 operands of the backward pass have (grad_power in delta.hpp).
// Each workgroup takes the largest finite |dY| and |dh_final| of a part of the
// tokens and of the state; the kernels that use it take the largest of the parts.
// One more read of dY and dh_final, bound by memory.
#include <hip/hip_runtime.h>

#include "delta.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

template <typename E>
__global__ __launch_bounds__(256) void delta_size_kernel(DeltaParams p) {
    typedef typename E::raw raw;
    constexpr int VE = 16 / int(sizeof(raw));
    __shared__ float scratch[2][4];
    const int part = blockIdx.x % p.nsize, tid = threadIdx.x;
    const int64_t of = blockIdx.x / p.nsize, b = of / p.H, h = of % p.H;
    const int end = seq_end(p.seqlens, b, p.L);
    // as few lanes to a token as have a vector each, so the others take the tokens behind it
    const int vectors = (p.dv + VE - 1) / VE;
    int lanes = 1;
    while (lanes < vectors && lanes < 256) lanes *= 2;
    const raw* Y = static_cast<const raw*>(p.dy) + b * p.sdy.batch + h * p.sdy.head;
    const int64_t last = int64_t(end) * (part + 1) / p.nsize;
    float y = 0.0f, m = 0.0f;
    for (int64_t t = int64_t(end) * part / p.nsize + tid / lanes; t < last; t += 256 / lanes)
        for (int c = tid % lanes; c < vectors; c += lanes) {
            const u32x4 v = ldg_b128(Y + t * p.sdy.token + c * VE);
#pragma unroll
            for (int e = 0; e < VE; ++e) y = larger(y, Mat<E>::at(v, e));
        }
    if (p.dh_last) {
        const int64_t size = int64_t(p.dv) * p.dk, to = size * (part + 1) / p.nsize;
        const float* D = p.dh_last + of * size;
        for (int64_t i = size * part / p.nsize + tid; i < to; i += 256) m = larger(m, D[i]);
    }
    y = wave_max(y);
    m = wave_max(m);
    if ((tid & 63) == 0) {
        scratch[0][tid >> 6] = y;
        scratch[1][tid >> 6] = m;
    }
    __syncthreads();
    if (tid < 2) {
        const float* s = scratch[tid];
        p.sizes[(of * 2 + tid) * kSizes + part] = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
    }
}

}  // namespace
}  // namespace cls

int cls_delta_size_launch(const cls::DeltaParams& p, hipStream_t stream) {
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * p.nsize);
    cls::delta_size_kernel<cls::ElemF16><<<wgs, 256, 0, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}
