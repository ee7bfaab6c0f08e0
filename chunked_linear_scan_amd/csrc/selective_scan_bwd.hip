// Selective scan, backward, on gfx950.
#include "selective_scan.hpp"

#include "launch_selective.hpp"

namespace cls {
namespace {

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Each halving step adds two lanes' values of two sums at once: a lane keeps
// the one that `bit` names and hands the other over.
__device__ __forceinline__ float swap_add32(float lo, float hi) {
    const auto r = __builtin_amdgcn_permlane32_swap(as_uint(lo), as_uint(hi), false, false);
    return as_float(r[0]) + as_float(r[1]);
}
__device__ __forceinline__ float swap_add16(float lo, float hi) {
    const auto r = __builtin_amdgcn_permlane16_swap(as_uint(lo), as_uint(hi), false, false);
    return as_float(r[0]) + as_float(r[1]);
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(bool bit, float lo, float hi) {
    return (bit ? hi : lo) + dpp<CTRL>(bit ? lo : hi);
}

template <typename E, int NW, bool AGG>
__global__ __launch_bounds__(NW * 64, NW > 8 ? 4 : 2) void scan_bwd_kernel(ScanParams p) {
    constexpr int K = kScanK, NP = NW * K;
    constexpr int TT = NW > 8 ? 8 : 16;
    constexpr int R = TT >= NW ? TT / NW : 1;
    typedef typename E::raw raw;
    __shared__ float2 s_d[TT][kScanCh];   // dt', dt' u
    __shared__ float s_dy[TT][kScanCh];   // the gradient of y before the gate
    __shared__ float s_bc[2][TT][NP];
    __shared__ float s_p[AGG ? 1 : NW][3][AGG ? 1 : TT][kScanCh];  // each wave's share of three sums over the states

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t wg = blockIdx.x;
    const int cb = int(wg % p.bpg); wg /= p.bpg;
    const int g = int(wg % p.G); wg /= p.G;
    const int64_t b = wg % p.batch;
    const int seg = int(wg / p.batch) + (AGG ? 1 : 0);
    const int c = cb * kScanCh + lane;
    const bool on = c < p.cpg;
    const int ch = g * p.cpg + (on ? c : p.cpg - 1);
    const int L_end = seq_end(p.seqlens, b, p.L);
    const int64_t first = int64_t(seg) * p.seg_len;
    const int64_t stop = first + p.seg_len < p.L ? first + p.seg_len : p.L;
    const int64_t last = stop < L_end ? stop : L_end;
    const int64_t tiles = (p.L + TT - 1) / TT;

    const raw* u = static_cast<const raw*>(p.u) + b * p.su.b + ch;
    const raw* dt = static_cast<const raw*>(p.dt) + b * p.sdt.b + ch;
    const raw* z = p.z ? static_cast<const raw*>(p.z) + b * p.sz.b + ch : nullptr;
    const raw* dy = static_cast<const raw*>(p.dy) + b * p.sdy.b + ch;
    const raw* B = static_cast<const raw*>(p.B) + b * p.sB.b + g * p.sB.g;
    const raw* C = static_cast<const raw*>(p.C) + b * p.sC.b + g * p.sC.g;
    const float bias = p.dt_bias ? p.dt_bias[ch] : 0.0f;
    const float Dc = p.D ? p.D[ch] : 0.0f;

    const int n0 = wave * K;
    float A2[K], carry[K], dA[K];  // carry: the gradient that reaches the state from later tokens
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int n = n0 + k;
        A2[k] = n < p.N ? p.A[int64_t(ch) * p.N + n] * kLog2e : 0.0f;
        carry[k] = dA[k] = 0.0f;
    }
    if constexpr (!AGG) {
        if (p.dh_last) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (n0 + k < p.N) carry[k] = p.dh_last[(b * p.ch + ch) * p.N + n0 + k];
        }
        for (int s = p.nseg - 1; s > seg; --s) {
            const int64_t sb = int64_t(s) * p.batch + b;
            const float sd = p.seg_dt[sb * p.ch + ch];
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (n0 + k < p.N)
                    carry[k] = fmaf(fexp2(A2[k] * sd), carry[k], p.seg_h[(sb * p.N + n0 + k) * p.ch + ch]);
        }
    }
    float sum_dt = 0.0f, dD = 0.0f, dbias = 0.0f;

    raw ru[R], rdt[R], rz[R], rdy[R];
    float hin[K];
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = wave + r * NW;
            const int64_t t = t0 + row;
            ru[r] = rdt[r] = rz[r] = rdy[r] = 0;
            if (row < TT && t >= first && t < last) {
                ru[r] = u[t * p.su.t];
                rdt[r] = dt[t * p.sdt.t];
                rdy[r] = dy[t * p.sdy.t];
                if (z) rz[r] = z[t * p.sz.t];
            }
        }
    };
    const int64_t top = last > first ? (last - 1) / TT * TT : first - TT;
    load(top);
    for (int64_t t0 = top; t0 >= first; t0 -= TT) {
        if constexpr (!AGG) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                hin[k] = n0 + k < p.N ? p.ckpt[((b * tiles + t0 / TT) * p.N + n0 + k) * p.ch + ch] : 0.0f;
        }
        float uc[R], zc[R], xc[R], dc[R], oc[R], gc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = wave + r * NW;
            uc[r] = E::get(ru[r]);
            zc[r] = E::get(rz[r]);
            oc[r] = E::get(rdy[r]);
            xc[r] = E::get(rdt[r]) + bias;
            dc[r] = p.softplus ? softplus(xc[r]) : xc[r];
            if (t0 + row >= last) dc[r] = 0.0f;
            gc[r] = z ? oc[r] * zc[r] * sigmoid(zc[r]) : oc[r];
            if (row < TT) {
                s_d[row][lane] = make_float2(dc[r], dc[r] * uc[r]);
                s_dy[row][lane] = gc[r];
            }
        }
        for (int i = threadIdx.x; i < 2 * TT * NP; i += NW * 64) {
            const int n = i % NP, row = (i / NP) % TT, w = i / (NP * TT);
            float v = 0.0f;
            if (n < p.N && t0 + row < last && !(AGG && !w))
                v = E::get(w ? C[(t0 + row) * p.sC.t + n] : B[(t0 + row) * p.sB.t + n]);
            s_bc[w][row][n] = v;
        }
        load(t0 - TT);
        __syncthreads();
        if constexpr (AGG) {
#pragma unroll
            for (int t = TT - 1; t >= 0; --t) {
                const float d = s_d[t][lane].x, gy = s_dy[t][lane];
                const f32x4 cv = *reinterpret_cast<const f32x4*>(&s_bc[1][t][n0]);
                sum_dt += d;
#pragma unroll
                for (int k = 0; k < K; ++k) carry[k] = fexp2(d * A2[k]) * fmaf(gy, cv[k], carry[k]);
            }
            __syncthreads();
        } else {
            float a[TT][K], hs[TT][K];
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const float2 d = s_d[t][lane];
                const f32x4 bv = *reinterpret_cast<const f32x4*>(&s_bc[0][t][n0]);
                float yv = 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    a[t][k] = fexp2(d.x * A2[k]);
                    hs[t][k] = fmaf(a[t][k], t ? hs[t - 1][k] : hin[k], d.y * bv[k]);
                }
                if (z) {
                    const f32x4 cv = *reinterpret_cast<const f32x4*>(&s_bc[1][t][n0]);
#pragma unroll
                    for (int k = 0; k < K; ++k) yv = fmaf(cv[k], hs[t][k], yv);
                    s_p[wave][2][t][lane] = yv;
                }
            }
            const bool bit3 = lane & 8, bit2 = lane & 4, bit1 = lane & 2, bit0 = lane & 1;
#pragma unroll
            for (int o = TT / 8 - 1; o >= 0; --o) {
                float r8[8];
#pragma unroll
                for (int i = 7; i >= 0; --i) {
                    const int t = o * 8 + i;
                    const float2 d = s_d[t][lane];
                    const float gy = s_dy[t][lane];
                    const f32x4 bv = *reinterpret_cast<const f32x4*>(&s_bc[0][t][n0]);
                    const f32x4 cv = *reinterpret_cast<const f32x4*>(&s_bc[1][t][n0]);
                    float vB[K], vC[K], to_sig = 0.0f, to_dt = 0.0f;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const float q = fmaf(gy, cv[k], carry[k]);
                        carry[k] = q * a[t][k];
                        const float qah = carry[k] * (t ? hs[t - 1][k] : hin[k]);
                        dA[k] = fmaf(qah, d.x, dA[k]);
                        to_dt = fmaf(qah, A2[k], to_dt);
                        to_sig = fmaf(q, bv[k], to_sig);
                        vB[k] = on ? q * d.y : 0.0f;
                        vC[k] = on ? gy * hs[t][k] : 0.0f;
                    }
                    s_p[wave][0][t][lane] = to_sig;
                    s_p[wave][1][t][lane] = to_dt;
                    const float w0 = swap_add32(vB[0], vC[0]), w1 = swap_add32(vB[1], vC[1]);
                    const float w2 = swap_add32(vB[2], vC[2]), w3 = swap_add32(vB[3], vC[3]);
                    r8[i] = dpp_add<0x128>(bit3, swap_add16(w0, w2), swap_add16(w1, w3));
                }
                // the eight tokens' sums over the last three lane bits: half-row mirror, then within four lanes
                const float x0 = dpp_add<0x141>(bit2, r8[0], r8[4]), x1 = dpp_add<0x141>(bit2, r8[1], r8[5]);
                const float x2 = dpp_add<0x141>(bit2, r8[2], r8[6]), x3 = dpp_add<0x141>(bit2, r8[3], r8[7]);
                const float y0 = dpp_add<0x4e>(bit1, x0, x2), y1 = dpp_add<0x4e>(bit1, x1, x3);
                const float sum = dpp_add<0xb1>(bit0, y0, y1);
                const int64_t t = t0 + o * 8 + (lane & 7);
                const int n = n0 + ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1);
                if (t < last && n < p.N)
                    p.part_bc[((((int64_t(cb) * p.batch + b) * p.L + t) * p.G + g) * 2 + (lane >> 5)) * p.N + n] = sum;
            }
            __syncthreads();
            raw* du = static_cast<raw*>(p.du) + b * p.L * p.ch + ch;
            raw* ddt = static_cast<raw*>(p.ddt) + b * p.L * p.ch + ch;
            raw* dz = static_cast<raw*>(p.dz) + b * p.L * p.ch + ch;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = wave + r * NW;
                if (row >= TT || t0 + row >= last || !on) continue;
                float to_sig = 0.0f, to_dt = 0.0f;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    to_sig += s_p[w][0][row][lane];
                    to_dt += s_p[w][1][row][lane];
                }
                const int64_t at = (t0 + row) * p.ch;
                du[at] = E::put(fmaf(Dc, gc[r], dc[r] * to_sig));
                float d = fmaf(uc[r], to_sig, to_dt * kLn2);  // A2 is A log2(e)
                if (p.softplus) d *= sigmoid(xc[r]);
                ddt[at] = E::put(d);
                dbias += d;
                dD = fmaf(gc[r], uc[r], dD);
                if (z) {
                    float y = Dc * uc[r];
#pragma unroll
                    for (int w = 0; w < NW; ++w) y += s_p[w][2][row][lane];
                    dz[at] = E::put(oc[r] * y * dsilu(zc[r], sigmoid(zc[r])));
                }
            }
        }
    }
    if constexpr (AGG) {
        if (!on) return;
        const int64_t sb = int64_t(seg) * p.batch + b;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (n0 + k < p.N) p.seg_h[(sb * p.N + n0 + k) * p.ch + ch] = carry[k];
        if (wave == 0) p.seg_dt[sb * p.ch + ch] = sum_dt;
    } else {
        __syncthreads();
        s_p[wave][0][0][lane] = dD;
        s_p[wave][1][0][lane] = dbias;
        __syncthreads();
        if (!on) return;
        float* pa = p.part_a + (b * p.nseg + seg) * int64_t(p.N + 2) * p.ch + ch;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (n0 + k < p.N) pa[int64_t(n0 + k) * p.ch] = dA[k];
        if (wave == 0) {
            float sD = 0.0f, sb = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                sD += s_p[w][0][0][lane];
                sb += s_p[w][1][0][lane];
            }
            pa[int64_t(p.N) * p.ch] = sD;
            pa[int64_t(p.N + 1) * p.ch] = sb;
        }
        if (p.dh0 && seg == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (n0 + k < p.N) p.dh0[(b * p.ch + ch) * p.N + n0 + k] = carry[k];
        }
        raw* du = static_cast<raw*>(p.du) + b * p.L * p.ch + ch;
        raw* ddt = static_cast<raw*>(p.ddt) + b * p.L * p.ch + ch;
        raw* dz = static_cast<raw*>(p.dz) + b * p.L * p.ch + ch;
        for (int64_t t = (last > first ? last : first) + wave; t < stop; t += NW) {
            du[t * p.ch] = ddt[t * p.ch] = E::put(0.0f);
            if (z) dz[t * p.ch] = E::put(0.0f);
        }
    }
}

// dB and dC: the sums of the group's channel blocks, one thread per value.
template <typename E>
__global__ __launch_bounds__(256) void scan_bwd_bc_kernel(ScanParams p) {
    typedef typename E::raw raw;
    const int64_t per = int64_t(p.batch) * p.L * p.G * 2 * p.N;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < per; i += int64_t(gridDim.x) * 256) {
        const int n = int(i % p.N);
        const int64_t j = i / p.N, row = j >> 1;  // row: (b, t, g)
        const int64_t bt = row / p.G;
        float s = 0.0f;
        if (bt % p.L < seq_end(p.seqlens, bt / p.L, p.L))
            for (int c = 0; c < p.bpg; ++c) s += p.part_bc[int64_t(c) * per + i];
        static_cast<raw*>(j & 1 ? p.dC : p.dB)[row * p.N + n] = E::put(s);
    }
}

// dA, dD, ddt_bias: the sums over sequences and segments, one thread per value.
__global__ __launch_bounds__(256) void scan_bwd_a_kernel(ScanParams p) {
    const int64_t per = int64_t(p.N + 2) * p.ch;
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= per) return;
    const int ch = int(i % p.ch), r = int(i / p.ch);
    float s = 0.0f;
    for (int64_t q = 0; q < int64_t(p.batch) * p.nseg; ++q) s += p.part_a[q * per + i];
    if (r < p.N) p.dA[int64_t(ch) * p.N + r] = s;
    else if (r == p.N) { if (p.dD) p.dD[ch] = s; }
    else if (p.dbias) p.dbias[ch] = s;
}

template <typename E, int NW>
int launch_bwd(const ScanParams& p, hipStream_t stream) {
    const uint32_t per_seg = uint32_t(p.bpg) * uint32_t(p.G) * uint32_t(p.batch);
    const dim3 block{NW * 64u, 1u, 1u};
    if (p.nseg > 1) {
        hipLaunchKernelGGL((scan_bwd_kernel<E, NW, true>), dim3(per_seg * uint32_t(p.nseg - 1)), block, 0, stream, p);
        if (hipGetLastError() != hipSuccess) return -7;
    }
    hipLaunchKernelGGL((scan_bwd_kernel<E, NW, false>), dim3(per_seg * uint32_t(p.nseg)), block, 0, stream, p);
    if (hipGetLastError() != hipSuccess) return -7;
    const int64_t values = int64_t(p.batch) * p.L * p.G * 2 * p.N;
    const int64_t blocks = (values + 255) / 256;
    hipLaunchKernelGGL((scan_bwd_bc_kernel<E>), dim3(uint32_t(blocks < 65536 ? blocks : 65536)), dim3(256), 0, stream, p);
    if (hipGetLastError() != hipSuccess) return -7;
    const int64_t per = int64_t(p.N + 2) * p.ch;
    hipLaunchKernelGGL(scan_bwd_a_kernel, dim3(uint32_t((per + 255) / 256)), dim3(256), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

template <typename E>
int launch_type(const ScanParams& p, hipStream_t stream) {
    switch (scan_waves(p.N)) {
        case 1: return launch_bwd<E, 1>(p, stream);
        case 2: return launch_bwd<E, 2>(p, stream);
        case 4: return launch_bwd<E, 4>(p, stream);
        case 8: return launch_bwd<E, 8>(p, stream);
        default: return launch_bwd<E, 16>(p, stream);
    }
}

}  // namespace
}  // namespace cls

int cls_selective_scan_bwd_launch(const cls::ScanParams& p, int dtype, hipStream_t stream) {
    return dtype == 0 ? cls::launch_type<cls::ElemF32>(p, stream)
         : dtype == 1 ? cls::launch_type<cls::ElemBF16>(p, stream)
                      : cls::launch_type<cls::ElemF16>(p, stream);
}
