// Selective scan, one token, on gfx950.
//
// Reads and writes each sequence's state once (64 bytes per channel at 16
// states) and little else: bound by memory for a batch, by the launch for one
// sequence.  A float4 of states to a lane; the four sequences of a thread keep
// four such loads in flight and read A once.  256 sequences x 5120 channels x 16
// states, bf16: 31 us, 5.8 TB/s of its 179 MB (copy rate 5.2, part of the states
// stays in the last-level cache); one sequence to a thread with the states
// element by element took 75 us, B and C element by element 46.  One sequence
// of 1536 channels: 3.2 us.
#include <type_traits>

#include "selective.hpp"

#include "launch_selective.hpp"

namespace cls {
namespace {

struct StepArgs {
    selective_scan_inputs in;
    float* h;
    void* y;
    uint32_t blocks;  // workgroups side by side in the channels
};

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// The sum over LS adjacent lanes, in all of them: within four, then mirrored halves and rows.
template <int LS>
__device__ __forceinline__ float sum_lanes(float v) {
    if constexpr (LS > 1) v += dpp<0xb1>(v);
    if constexpr (LS > 2) v += dpp<0x4e>(v);
    if constexpr (LS > 4) v += dpp<0x141>(v);
    if constexpr (LS > 8) v += dpp<0x128>(v);
    return v;
}

// Lane R of the LS, to all of them.
template <int LS, int R>
__device__ __forceinline__ float from_lane(float v) {
    if constexpr (LS == 1) return v;
    else if constexpr (LS == 4) return dpp<R * 0x55>(v);
    else return __shfl(v, int(threadIdx.x & 63 & ~(LS - 1)) + R, 64);
}

// four values from n on; WIDE: an aligned vector, else element by element below N
template <bool WIDE>
__device__ __forceinline__ f32x4 load4(const float* p, int n, int N) {
    if constexpr (WIDE) {
        return n < N ? *reinterpret_cast<const f32x4*>(p + n) : f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = n + e < N ? p[n + e] : 0.0f;
        return v;
    }
}

template <typename E, bool WIDE>
__device__ __forceinline__ f32x4 load_row(const void* base, int64_t at, int n, int N) {
    typedef typename E::raw raw4 __attribute__((ext_vector_type(4)));
    const typename E::raw* p = static_cast<const typename E::raw*>(base) + at;
    f32x4 v;
    if constexpr (WIDE) {
        const raw4 q = *reinterpret_cast<const raw4*>(p + (n < N ? n : 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const typename E::raw x = q[e];
            v[e] = E::get(x);
        }
        return v;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = E::get(p[n + e < N ? n + e : 0]);
    return v;
}

// LS lanes hold a channel's states, four each; a thread has U sequences, whose
// loads are in flight together and which share A.  Sequence r's step and gate
// are computed by lane r of the LS alone and handed to the others.
template <typename E, int LS, int U, bool WIDE>
__global__ __launch_bounds__(256) void scan_step_kernel(StepArgs s) {
    typedef typename E::raw raw;
    static_assert(U == 1 || LS >= U, "a lane to each sequence");
    const selective_scan_inputs& p = s.in;
    const int N = int(p.dstate), l = threadIdx.x % LS;
    const int64_t b0 = int64_t(blockIdx.x / s.blocks) * U;
    const int c = int(blockIdx.x % s.blocks) * (256 / LS) + int(threadIdx.x) / LS;
    const bool on = c < p.channels;
    const int ch = on ? c : int(p.channels) - 1;
    const int g = ch / int(p.channels / p.ngroups);
    const int n = 4 * l;
    const int64_t mine = b0 + (U > 1 ? l & (U - 1) : 0);
    const int64_t bm = mine < p.batch ? mine : p.batch - 1;
    const float u = E::get(static_cast<const raw*>(p.u)[bm * p.u_batch + ch]);
    float d = E::get(static_cast<const raw*>(p.dt)[bm * p.dt_batch + ch]) + (p.dt_bias ? p.dt_bias[ch] : 0.0f);
    const float z = p.z ? E::get(static_cast<const raw*>(p.z)[bm * p.z_batch + ch]) : 0.0f;
    f32x4 h[U], B[U], C[U];
#pragma unroll
    for (int r = 0; r < U; ++r) {
        const int64_t b = b0 + r < p.batch ? b0 + r : p.batch - 1;
        const float* src = s.h + (b * p.channels + ch) * N;
        if constexpr (WIDE) {
            // each state is touched once a token: past the caches
            h[r] = n < N ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(src + n)) : f32x4{0.f, 0.f, 0.f, 0.f};
        } else {
            h[r] = load4<false>(src, n, N);
        }
        B[r] = load_row<E, WIDE>(p.B, b * p.B_batch + g * p.B_group, n, N);
        C[r] = load_row<E, WIDE>(p.C, b * p.C_batch + g * p.C_group, n, N);
    }
    f32x4 A2 = load4<WIDE>(p.A + int64_t(ch) * N, n, N);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = A2[e];
        A2[e] = a * kLog2e;
    }
    if (p.softplus) d = softplus(d);
    const float du = d * u;
    float y = 0.0f;
    const auto row = [&](auto R) {
        constexpr int r = decltype(R)::value;
        const float dr = from_lane<LS, r>(d), dur = from_lane<LS, r>(du);
        float part = 0.0f;
        f32x4 hn;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a2 = A2[e], ho = h[r][e], b = B[r][e], c4 = C[r][e];
            const float v = fmaf(fexp2(dr * a2), ho, dur * b);
            hn[e] = v;
            if (n + e < N) part = fmaf(c4, v, part);
        }
        part = sum_lanes<LS>(part);
        if (U == 1 || (l & (U - 1)) == r) y = part;
        if (on && b0 + r < p.batch) {
            float* dst = s.h + ((b0 + r) * p.channels + ch) * N + n;
            if constexpr (WIDE) {
                if (n < N) __builtin_nontemporal_store(hn, reinterpret_cast<f32x4*>(dst));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < N) dst[e] = hn[e];
            }
        }
    };
    row(std::integral_constant<int, 0>{});
    if constexpr (U > 1) {
        row(std::integral_constant<int, 1>{});
        row(std::integral_constant<int, 2>{});
        row(std::integral_constant<int, 3>{});
    }
    if (l < U && on && mine < p.batch) {
        y = fmaf(p.D ? p.D[ch] : 0.0f, u, y);
        if (p.z) y *= z * sigmoid(z);
        static_cast<raw*>(s.y)[mine * p.channels + ch] = E::put(y);
    }
}

// Lanes that hold a channel's states, four each, and the workgroups side by side in the channels.
inline int64_t step_lanes(int64_t N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
inline int64_t step_blocks(const selective_scan_inputs& in) { return (in.channels * step_lanes(in.dstate) + 255) / 256; }

// four sequences to a thread where that still leaves every CU a few workgroups
inline int64_t step_fours(const selective_scan_inputs& in) { return step_blocks(in) * ((in.batch + 3) / 4); }
inline bool step_in_fours(const selective_scan_inputs& in) { return step_lanes(in.dstate) >= 4 && step_fours(in) >= 1024; }

template <typename E, int LS>
int launch_lanes(StepArgs s, hipStream_t stream) {
    const selective_scan_inputs& in = s.in;
    s.blocks = uint32_t(step_blocks(in));
    // whole vectors of four states where every row of A, B and C starts on one
    const uint64_t at = reinterpret_cast<uintptr_t>(in.B) | reinterpret_cast<uintptr_t>(in.C) |
                        uint64_t(in.B_batch | in.B_group | in.C_batch | in.C_group) * sizeof(typename E::raw);
    const bool wide = in.dstate % 4 == 0 && reinterpret_cast<uintptr_t>(in.A) % 16 == 0 &&
                      at % (4 * sizeof(typename E::raw)) == 0;
    const dim3 grid(uint32_t(cls_selective_scan_step_groups(in)));
    if constexpr (LS >= 4) {
        if (step_in_fours(in)) {
            if (wide) hipLaunchKernelGGL((scan_step_kernel<E, LS, 4, true>), grid, dim3(256), 0, stream, s);
            else hipLaunchKernelGGL((scan_step_kernel<E, LS, 4, false>), grid, dim3(256), 0, stream, s);
            return hipGetLastError() == hipSuccess ? 0 : -7;
        }
    }
    if (wide) hipLaunchKernelGGL((scan_step_kernel<E, LS, 1, true>), grid, dim3(256), 0, stream, s);
    else hipLaunchKernelGGL((scan_step_kernel<E, LS, 1, false>), grid, dim3(256), 0, stream, s);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

template <typename E>
int launch_type(const StepArgs& s, hipStream_t stream) {
    switch (step_lanes(s.in.dstate)) {
        case 1: return launch_lanes<E, 1>(s, stream);
        case 2: return launch_lanes<E, 2>(s, stream);
        case 4: return launch_lanes<E, 4>(s, stream);
        case 8: return launch_lanes<E, 8>(s, stream);
        default: return launch_lanes<E, 16>(s, stream);
    }
}

}  // namespace
}  // namespace cls

int64_t cls_selective_scan_step_groups(const selective_scan_inputs& in) {
    return cls::step_in_fours(in) ? cls::step_fours(in) : cls::step_blocks(in) * in.batch;
}

int cls_selective_scan_step_launch(const selective_scan_inputs& in, float* h, void* y, hipStream_t stream) {
    const cls::StepArgs s{in, h, y, 0};
    return in.dtype == 0 ? cls::launch_type<cls::ElemF32>(s, stream)
         : in.dtype == 1 ? cls::launch_type<cls::ElemBF16>(s, stream)
                         : cls::launch_type<cls::ElemF16>(s, stream);
}
