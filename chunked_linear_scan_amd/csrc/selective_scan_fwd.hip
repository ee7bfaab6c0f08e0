// Selective scan, forward, on gfx950.
#include "selective_scan.hpp"

#include "launch_selective.hpp"

namespace cls {
namespace {

// AGG: a segment's own contribution only (state from zero, summed steps).
template <typename E, int NW, bool AGG>
__global__ __launch_bounds__(NW * 64) void scan_fwd_kernel(ScanParams p) {
    constexpr int K = kScanK, NP = NW * K;
    constexpr int TT = NW > 8 ? 8 : 16;
    constexpr int R = TT >= NW ? TT / NW : 1;  // token rows that a wave stages and finishes
    typedef typename E::raw raw;
    __shared__ float2 s_d[TT][kScanCh];        // dt', dt' u
    __shared__ float s_bc[2][TT][NP];
    __shared__ float s_y[AGG ? 1 : NW][AGG ? 1 : TT][kScanCh];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t wg = blockIdx.x;
    const int cb = int(wg % p.bpg); wg /= p.bpg;
    const int g = int(wg % p.G); wg /= p.G;
    const int64_t b = wg % p.batch;
    const int seg = int(wg / p.batch);
    const int c = cb * kScanCh + lane;
    const bool on = c < p.cpg;
    const int ch = g * p.cpg + (on ? c : p.cpg - 1);  // lanes past the group compute its last channel, unseen
    const int L_end = seq_end(p.seqlens, b, p.L);
    const int64_t first = int64_t(seg) * p.seg_len;
    const int64_t stop = first + p.seg_len < p.L ? first + p.seg_len : p.L;   // of the segment
    const int64_t last = stop < L_end ? stop : L_end;                         // of its tokens that count

    const raw* u = static_cast<const raw*>(p.u) + b * p.su.b + ch;
    const raw* dt = static_cast<const raw*>(p.dt) + b * p.sdt.b + ch;
    const raw* z = p.z ? static_cast<const raw*>(p.z) + b * p.sz.b + ch : nullptr;
    const raw* B = static_cast<const raw*>(p.B) + b * p.sB.b + g * p.sB.g;
    const raw* C = static_cast<const raw*>(p.C) + b * p.sC.b + g * p.sC.g;
    const float bias = p.dt_bias ? p.dt_bias[ch] : 0.0f;
    const float Dc = p.D ? p.D[ch] : 0.0f;

    const int n0 = wave * K;
    float A2[K], h[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int n = n0 + k;
        A2[k] = n < p.N ? p.A[int64_t(ch) * p.N + n] * kLog2e : 0.0f;
        h[k] = 0.0f;
    }
    if constexpr (!AGG) {
        if (p.h0) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (n0 + k < p.N) h[k] = p.h0[(b * p.ch + ch) * p.N + n0 + k];
        }
        for (int s = 0; s < seg; ++s) {  // what the earlier segments did to the state
            const int64_t sb = int64_t(s) * p.batch + b;
            const float sd = p.seg_dt[sb * p.ch + ch];
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (n0 + k < p.N) h[k] = fmaf(fexp2(A2[k] * sd), h[k], p.seg_h[(sb * p.N + n0 + k) * p.ch + ch]);
        }
    }
    float sum_dt = 0.0f;

    raw ru[R], rdt[R], rz[R];
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = wave + r * NW;
            const int64_t t = t0 + row;
            ru[r] = rdt[r] = rz[r] = 0;
            if (row < TT && t < last) {
                ru[r] = u[t * p.su.t];
                rdt[r] = dt[t * p.sdt.t];
                if (!AGG && z) rz[r] = z[t * p.sz.t];
            }
        }
    };
    load(first);
    for (int64_t t0 = first; t0 < last; t0 += TT) {
        float uc[R], zc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = wave + r * NW;
            uc[r] = E::get(ru[r]);
            zc[r] = E::get(rz[r]);
            float d = E::get(rdt[r]) + bias;
            if (p.softplus) d = softplus(d);
            if (t0 + row >= last) d = 0.0f;  // no step
            if (row < TT) s_d[row][lane] = make_float2(d, d * uc[r]);
        }
        for (int i = threadIdx.x; i < 2 * TT * NP; i += NW * 64) {
            const int n = i % NP, row = (i / NP) % TT, w = i / (NP * TT);
            float v = 0.0f;
            if (n < p.N && t0 + row < last && !(AGG && w))
                v = E::get(w ? C[(t0 + row) * p.sC.t + n] : B[(t0 + row) * p.sB.t + n]);
            s_bc[w][row][n] = v;
        }
        load(t0 + TT);
        __syncthreads();
        if constexpr (!AGG) {
            if (p.ckpt && on) {
                const int64_t tiles = (p.L + TT - 1) / TT;
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (n0 + k < p.N) p.ckpt[((b * tiles + t0 / TT) * p.N + n0 + k) * p.ch + ch] = h[k];
            }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float2 d = s_d[t][lane];
            const f32x4 bv = *reinterpret_cast<const f32x4*>(&s_bc[0][t][n0]);
            float yv = 0.0f;
            if constexpr (AGG) {
                sum_dt += d.x;
#pragma unroll
                for (int k = 0; k < K; ++k) h[k] = fmaf(fexp2(d.x * A2[k]), h[k], d.y * bv[k]);
            } else {
                const f32x4 cv = *reinterpret_cast<const f32x4*>(&s_bc[1][t][n0]);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    h[k] = fmaf(fexp2(d.x * A2[k]), h[k], d.y * bv[k]);
                    yv = fmaf(cv[k], h[k], yv);
                }
                s_y[wave][t][lane] = yv;
            }
        }
        __syncthreads();
        if constexpr (!AGG) {
            raw* y = static_cast<raw*>(p.y) + b * p.L * p.ch + ch;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = wave + r * NW;
                if (row >= TT || t0 + row >= last || !on) continue;
                float v = Dc * uc[r];
#pragma unroll
                for (int w = 0; w < NW; ++w) v += s_y[w][row][lane];
                if (z) v *= zc[r] * sigmoid(zc[r]);
                y[(t0 + row) * p.ch] = E::put(v);
            }
        }
    }
    if (!on) return;
    if constexpr (AGG) {
        const int64_t sb = int64_t(seg) * p.batch + b;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (n0 + k < p.N) p.seg_h[(sb * p.N + n0 + k) * p.ch + ch] = h[k];
        if (wave == 0) p.seg_dt[sb * p.ch + ch] = sum_dt;
    } else {
        raw* y = static_cast<raw*>(p.y) + b * p.L * p.ch + ch;
        for (int64_t t = (last > first ? last : first) + wave; t < stop; t += NW) y[t * p.ch] = E::put(0.0f);
        if (p.h_last && seg == p.nseg - 1) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (n0 + k < p.N) p.h_last[(b * p.ch + ch) * p.N + n0 + k] = h[k];
        }
    }
}

template <typename E, int NW>
int launch_fwd(const ScanParams& p, hipStream_t stream) {
    const uint32_t per_seg = uint32_t(p.bpg) * uint32_t(p.G) * uint32_t(p.batch);
    const dim3 block{NW * 64u, 1u, 1u};
    if (p.nseg > 1) {
        hipLaunchKernelGGL((scan_fwd_kernel<E, NW, true>), dim3(per_seg * uint32_t(p.nseg - 1)), block, 0, stream, p);
        if (hipGetLastError() != hipSuccess) return -7;
    }
    hipLaunchKernelGGL((scan_fwd_kernel<E, NW, false>), dim3(per_seg * uint32_t(p.nseg)), block, 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

template <typename E>
int launch_type(const ScanParams& p, hipStream_t stream) {
    switch (scan_waves(p.N)) {
        case 1: return launch_fwd<E, 1>(p, stream);
        case 2: return launch_fwd<E, 2>(p, stream);
        case 4: return launch_fwd<E, 4>(p, stream);
        case 8: return launch_fwd<E, 8>(p, stream);
        default: return launch_fwd<E, 16>(p, stream);
    }
}

}  // namespace
}  // namespace cls

int cls_selective_scan_fwd_launch(const cls::ScanParams& p, int dtype, hipStream_t stream) {
    return dtype == 0 ? cls::launch_type<cls::ElemF32>(p, stream)
         : dtype == 1 ? cls::launch_type<cls::ElemBF16>(p, stream)
                      : cls::launch_type<cls::ElemF16>(p, stream);
}
