// Selective scan, forward, on gfx950.
//
// Per token, channel and state: h = exp2(dt' A log2 e) h + (dt' u) B, and the
// output's share C h.  That is one exp2 (8 cycles of a SIMD for 64 lanes,
// measured; an ordinary instruction 4), the product in its exponent, one
// multiply-add for h and one for y: 20 cycles, the bound of this kernel, since
// each (token, channel) brings 8 bytes for 16 states' 320 cycles.  The product
// (dt' u) B is rank 1 over (state, channel), so a 4x4x1 matrix instruction
// gives it for four states beside the vector pipe, its block broadcast picking
// the token's four values of B out of one register that holds the tile; taking
// the four products of y through it, too, measured slower (705 us where DPP
// operands take 596).  B and C as scalar loads (wave-uniform, no registers)
// measured 3800 us: their latency is not hidden.
//
// Work that does not depend on the state (softplus, the gate, loads, stores)
// is done once per (token, channel): each wave stages a share of the tile's
// rows into LDS and finishes the same share from the waves' partial sums.
//
// Where channels and sequences give too few waves, a first launch takes every
// segment but the last from a zero state (16 cycles per value: no y); the
// second folds what came before its segment, exp2(A sum dt') h + own, and runs
// the outputs.  1 x 32768 x 4096 channels x 16 states, bf16: 916 us a call, in
// kernels of 379 and 548 us at their fastest (medians of a profiled run 412 and
// 602, at a lower clock; VALU busy 89-91 % of the time); one pass over its 1.1 GB
// at copy rate would be 209 us, its bare recurrence 562 us in both passes.
#include "selective_scan.hpp"

#include "launch_selective.hpp"

namespace cls {
namespace {

// AGG: a segment's own contribution only (state from zero, summed steps).
template <typename E, int NW, bool AGG>
__global__ __launch_bounds__(NW * 64, 4) void scan_fwd_kernel(ScanParams p) {
    constexpr int K = kScanK;
    constexpr int TT = kScanTile;
    constexpr int R = TT >= NW ? TT / NW : 1;  // token rows that a wave stages and finishes
    typedef typename E::raw raw;
    __shared__ float2 s_d[TT][kScanCh];        // dt', dt' u
    __shared__ float s_y[NW][AGG ? 1 : TT][kScanCh];  // each wave's share of the sum over the states

    const ScanPlace at = scan_place(p);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t b = at.b;
    const bool on = at.on;
    const uint32_t ch = uint32_t(at.ch);
    const int seg = at.seg;
    const int64_t first = at.first, last = at.last;
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
        scan_fold(p, 0, 1, seg, b, at.ch, n0, A2, h);  // what the earlier segments did to the state
    }
    float sum_dt = 0.0f;

    // rows of the tile to come, from wave-uniform pointers that step from tile to tile
    const raw* u = static_cast<const raw*>(p.u) + b * p.su.b + first * p.su.t;
    const raw* dt = static_cast<const raw*>(p.dt) + b * p.sdt.b + first * p.sdt.t;
    const raw* z = p.z ? static_cast<const raw*>(p.z) + b * p.sz.b + first * p.sz.t : nullptr;
    ScanRows<E> B(p.B, p.sB, b, at.g, first, n0, p.N, lane), C(p.C, p.sC, b, at.g, first, n0, p.N, lane);
    const uint32_t lane_off = ch * uint32_t(sizeof(raw));
    const int u_t = int(p.su.t), dt_t = int(p.sdt.t), z_t = int(p.sz.t);
    raw ru[R], rdt[R], rz[R];
    auto load = [&](int64_t t0) {
        // past the end: the last token that counts, whose values are read and not used
        const int rem = int(last - 1 - t0 < TT ? last - 1 - t0 : TT);
        B.load(rem);
        if (!AGG) C.load(rem);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = wave + r * NW < rem ? wave + r * NW : rem;
            ru[r] = at_bytes(u + row * u_t, lane_off);
            rdt[r] = at_bytes(dt + row * dt_t, lane_off);
            rz[r] = 0;
            if (!AGG && z) rz[r] = at_bytes(z + row * z_t, lane_off);
        }
        u += TT * int64_t(u_t);
        dt += TT * int64_t(dt_t);
        if (!AGG && z) z += TT * int64_t(z_t);
        B.step(1);
        if (!AGG) C.step(1);
    };
    raw* y = AGG ? nullptr : static_cast<raw*>(p.y) + (b * p.L + first) * p.ch;
    float* ckpt = AGG || !p.ckpt ? nullptr : p.ckpt + ((b * ((p.L + TT - 1) / TT) + first / TT) * p.N + n0) * p.ch;
    if (last > first) load(first);
    for (int64_t t0 = first; t0 < last; t0 += TT) {
        const int nt = int(last - t0 < TT ? last - t0 : TT);
        float uc[R], zc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = wave + r * NW;
            uc[r] = E::get(ru[r]);
            zc[r] = E::get(rz[r]);
            float d = E::get(rdt[r]) + bias;
            if (p.softplus) d = softplus(d);
            float du = d * uc[r];
            if (row >= nt) d = du = 0.0f;  // no step
            if (AGG && row < TT) sum_dt += d;
            if (row < TT) s_d[row][lane] = make_float2(d, du);
        }
        const float fB = B.get();
        float fC[2];
        if (!AGG) row_quads(C.get(), fC);
        load(t0 + TT);
        __syncthreads();
        if (!AGG && ckpt) {
            if (on) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (n0 + k < p.N) at_bytes(ckpt + k * p.ch, ch * 4) = h[k];
            }
            ckpt += int64_t(p.N) * p.ch;
        }
        [&]<int... T>(std::integer_sequence<int, T...>) {
            (
                [&] {
                    const float2 d = s_d[T][lane];
                    const f32x4 b4 = outer<T>(fB, d.y);
#pragma unroll
                    for (int k = 0; k < K; ++k) h[k] = fmaf(fexp2(d.x * A2[k]), h[k], b4[k]);
                    if constexpr (!AGG) s_y[wave][T][lane] = dot<T>(fC, h);
                }(),
                ...);
        }(std::make_integer_sequence<int, TT>{});
        __syncthreads();
        if constexpr (!AGG) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = wave + r * NW;
                if (row >= nt) continue;
                float v = Dc * uc[r];
#pragma unroll
                for (int w = 0; w < NW; ++w) v += s_y[w][row][lane];
                if (p.z) v *= zc[r] * sigmoid(zc[r]);
                if (on) at_bytes(y + int64_t(row) * p.ch, lane_off) = E::put(v);
            }
            y += int64_t(TT) * p.ch;
        }
    }
    if constexpr (AGG) {
        s_y[wave][0][lane] = sum_dt;
        __syncthreads();
        if (!on) return;
        const int64_t sb = int64_t(seg) * p.batch + b;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (n0 + k < p.N) p.seg_h[(sb * p.N + n0 + k) * p.ch + ch] = h[k];
        if (wave == 0) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += s_y[w][0][lane];
            p.seg_dt[sb * p.ch + ch] = s;
        }
    } else {
        if (!on) return;
        y = static_cast<raw*>(p.y) + b * p.L * p.ch;
        for (int64_t t = (last > first ? last : first) + wave; t < at.stop; t += NW) (y + t * p.ch)[ch] = E::put(0.0f);
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
