// Selective scan, one token, on gfx950.
#include "selective.hpp"

#include "launch_selective.hpp"

namespace cls {
namespace {

struct StepArgs {
    selective_scan_inputs in;
    float* h;
    void* y;
};

// LS lanes hold a channel's states, four each.
template <typename E, int LS>
__global__ __launch_bounds__(256) void scan_step_kernel(StepArgs s) {
    typedef typename E::raw raw;
    const selective_scan_inputs& p = s.in;
    const int N = int(p.dstate), l = threadIdx.x % LS;
    const int64_t row = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LS;  // (b, ch)
    const bool on = row < p.batch * p.channels;
    const int64_t at = on ? row : p.batch * p.channels - 1;
    const int64_t b = at / p.channels;
    const int ch = int(at % p.channels);
    const int g = ch / int(p.channels / p.ngroups);
    const float u = E::get(static_cast<const raw*>(p.u)[b * p.u_batch + ch]);
    float d = E::get(static_cast<const raw*>(p.dt)[b * p.dt_batch + ch]) + (p.dt_bias ? p.dt_bias[ch] : 0.0f);
    if (p.softplus) d = softplus(d);
    const float du = d * u;
    const raw* B = static_cast<const raw*>(p.B) + b * p.B_batch + g * p.B_group;
    const raw* C = static_cast<const raw*>(p.C) + b * p.C_batch + g * p.C_group;
    float y = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = l * 4 + e;
        if (n >= N || !on) continue;
        const float a = fexp2(d * p.A[int64_t(ch) * N + n] * kLog2e);
        const float h = fmaf(a, s.h[at * N + n], du * E::get(B[n]));
        s.h[at * N + n] = h;
        y = fmaf(E::get(C[n]), h, y);
    }
#pragma unroll
    for (int o = LS / 2; o >= 1; o >>= 1) y += __shfl_xor(y, o, 64);
    if (l == 0 && on) {
        y = fmaf(p.D ? p.D[ch] : 0.0f, u, y);
        if (p.z) {
            const float z = E::get(static_cast<const raw*>(p.z)[b * p.z_batch + ch]);
            y *= z * sigmoid(z);
        }
        static_cast<raw*>(s.y)[at] = E::put(y);
    }
}

template <typename E>
int launch_type(const StepArgs& s, hipStream_t stream) {
    const int64_t lanes = (s.in.dstate + 3) / 4;
    const int64_t rows = s.in.batch * s.in.channels;
    const auto grid = [&](int64_t ls) { return dim3(uint32_t((rows * ls + 255) / 256)); };
    if (lanes <= 1) hipLaunchKernelGGL((scan_step_kernel<E, 1>), grid(1), dim3(256), 0, stream, s);
    else if (lanes <= 2) hipLaunchKernelGGL((scan_step_kernel<E, 2>), grid(2), dim3(256), 0, stream, s);
    else if (lanes <= 4) hipLaunchKernelGGL((scan_step_kernel<E, 4>), grid(4), dim3(256), 0, stream, s);
    else if (lanes <= 8) hipLaunchKernelGGL((scan_step_kernel<E, 8>), grid(8), dim3(256), 0, stream, s);
    else hipLaunchKernelGGL((scan_step_kernel<E, 16>), grid(16), dim3(256), 0, stream, s);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_selective_scan_step_launch(const selective_scan_inputs& in, float* h, void* y, hipStream_t stream) {
    const cls::StepArgs s{in, h, y};
    return in.dtype == 0 ? cls::launch_type<cls::ElemF32>(s, stream)
         : in.dtype == 1 ? cls::launch_type<cls::ElemBF16>(s, stream)
                         : cls::launch_type<cls::ElemF16>(s, stream);
}
