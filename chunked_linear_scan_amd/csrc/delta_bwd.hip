// Gradients of the gated delta rule, the part that walks the chunks: from the
// last to the first, a wave with 16 columns of dS, the gradient of the state, as
// the forward walk has them of S.  Per chunk, dS being that of the state behind it,
//     dN = e^(gamma_C - gamma) K dS + scale P^T dY,  Z = T^T dN,  dV = dR = beta Z,
//     dS' = e^gamma_C dS + scale Q^T e^gamma dY - K^T e^gamma dR.
// dS of every chunk and Z go to memory for the kernel that takes the chunks'
// other gradients all at once (delta_grad.hip).
#include <hip/hip_runtime.h>

#include "delta.hpp"
#include "device_once.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;  // of dv to a workgroup

template <typename E, int DK>
__global__ __launch_bounds__(kThreads) void delta_bwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef ChunkMats<E> CM;
    constexpr int C = M::kChunk, NT = C / 16, KT = DK / 16;
    constexpr int KP = DK + M::kPad, MP = CM::kPitch, NM = CM::kAll;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    raw* sK = reinterpret_cast<raw*>(lds);
    raw* sQ = sK + C * KP;
    raw* sT = sQ + C * KP;  // T, P (their parts)
    raw* sP = sT + CM::kParts * C * MP;
    float* sV = reinterpret_cast<float*>(sT + NM * C * MP);

    const int nblk = (p.dv + kCols - 1) / kCols;
    const int blk = blockIdx.x % nblk, h = blockIdx.x / nblk % p.H, b = blockIdx.x / nblk / p.H;
    const int end = seq_end(p.seqlens, b, p.L), kh = h / (p.H / p.Hk);
    const int tid = threadIdx.x, l16 = lane16(), g4 = group4();
    const int n = blk * kCols + (tid >> 6) * 16 + l16;
    const bool on = n < p.dv, wave_on = blk * kCols + (tid >> 6) * 16 < p.dv;

    const raw* K = static_cast<const raw*>(p.k) + b * p.sk.batch + kh * p.sk.head;
    const raw* Q = static_cast<const raw*>(p.q) + b * p.sq.batch + kh * p.sq.head;
    const raw* dY = static_cast<const raw*>(p.dy) + b * p.sdy.batch + h * p.sdy.head + n;
    const int64_t row = int64_t(p.H) * p.dv;  // of a token
    const int64_t out = (int64_t(b) * p.L * p.H + h) * p.dv + n;
    raw* dV = static_cast<raw*>(p.dv_) + out;

    f32x4 S[KT];
    const int64_t hat = ((int64_t(b) * p.H + h) * p.dv + n) * p.dk;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = 16 * t + 4 * g4 + r;
            S[t][r] = p.dh_last && on && d < p.dk ? p.dh_last[hat + d] : 0.0f;
        }

    TileRegs<E, C, DK, kThreads> rk, rq;
    TileRegs<E, C, C, kThreads> rm[NM];
    float rv = 0.0f;
    raw v[NT][4];
    const int chunks = (end + C - 1) / C;
    const auto fetch = [&](int c) {
        const int t0 = c * C;
        rk.load(K, p.sk.token, t0, end, p.dk, p.vec_k);
        rq.load(Q, p.sq.token, t0, end, p.dk, p.vec_q);
        const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
        const raw* mats = static_cast<const raw*>(p.mats) + chunk * CM::kAll * CM::kSize;
#pragma unroll
        for (int m = 0; m < NM; ++m) rm[m].load(mats + m * CM::kSize, C, 0, C, C, true);
        if (tid < 3 * C) rv = p.vecs[chunk * 3 * C + tid];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tok = t0 + 16 * t + 4 * g4 + r;
                v[t][r] = on && tok < end ? dY[tok * p.sdy.token] : raw(0);
            }
    };
    if (chunks > 0) fetch(chunks - 1);
    for (int c = chunks - 1; c >= 0; --c) {
        const int t0 = c * C;
        __syncthreads();  // the chunk before is read
        rk.store(sK, KP);
        rq.store(sQ, KP);
#pragma unroll
        for (int m = 0; m < NM; ++m) rm[m].store(sT + m * C * MP, MP);
        if (tid < 3 * C) sV[tid] = rv;
        f32x4 dy[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) dy[t][r] = E::get(v[t][r]);
        __syncthreads();
        if (c > 0) fetch(c - 1);
        if (!wave_on) continue;

        if (on) {
            float* to = p.dstates + (((int64_t(b) * p.nchunk + c) * p.H + h) * p.dk) * p.dv + n;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int d = 16 * t + 4 * g4 + r;
                    if (d < p.dk) to[int64_t(d) * p.dv] = S[t][r];
                }
        }
        f32x4 dN[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) dN[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) {
            const Two<E> st = two<E>(S[2 * s], S[2 * s + 1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) dN[t] = mma2<E>(M::rows(sK + (16 * t + l16) * KP + 32 * s), st, dN[t]);
        }
        typename M::frag df[NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) df[s] = M::cvt(dy[2 * s], dy[2 * s + 1]);  // exact
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4 later{0, 0, 0, 0};
#pragma unroll
            for (int s = t / 2; s < NT / 2; ++s) {  // later tokens' outputs
                Two<E> P;
                P.hi = M::cols(sP + 32 * s * MP + 16 * t, MP);
                if constexpr (M::kSplit) P.lo = M::cols(sP + C * MP + 32 * s * MP + 16 * t, MP);
                later = mma2<E>(P, df[s], later);
            }
            const f32x4 e = *reinterpret_cast<const f32x4*>(sV + C + 16 * t + 4 * g4);
#pragma unroll
            for (int r = 0; r < 4; ++r) dN[t][r] = fmaf(dN[t][r], e[r], p.scale * later[r]);
        }
        Two<E> dn[NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) dn[s] = two<E>(dN[2 * s], dN[2 * s + 1]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4 Z = dN[t];
#pragma unroll
            for (int s = t / 2; s < NT / 2; ++s) {
                Two<E> T;
                T.hi = M::cols(sT + 32 * s * MP + 16 * t, MP);
                if constexpr (M::kSplit) T.lo = M::cols(sT + C * MP + 32 * s * MP + 16 * t, MP);
                Z = mma3<E>(T, dn[s], Z);
            }
            const f32x4 e = *reinterpret_cast<const f32x4*>(sV + 16 * t + 4 * g4);
            const f32x4 be = *reinterpret_cast<const f32x4*>(sV + 2 * C + 16 * t + 4 * g4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tok = t0 + 16 * t + 4 * g4 + r;
                const float dr = be[r] * Z[r];
                dN[t][r] = -e[r] * dr;
                dy[t][r] *= p.scale * e[r];
                if (!on || tok >= p.L) continue;
                dV[tok * row] = tok < end ? E::put(dr) : raw(0);
                if (tok < end) p.z[out + tok * row] = Z[r];
            }
        }
        const float fade = sV[C - 1];
        Two<E> a[NT / 2], q[NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) {
            a[s] = two<E>(dN[2 * s], dN[2 * s + 1]);
            q[s] = two<E>(dy[2 * s], dy[2 * s + 1]);
        }
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            S[t] *= fade;
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) {
                S[t] = mma2<E>(M::cols(sQ + 32 * s * KP + 16 * t, KP), q[s], S[t]);
                S[t] = mma2<E>(M::cols(sK + 32 * s * KP + 16 * t, KP), a[s], S[t]);
            }
        }
    }
    if (!on) return;
    for (int tok = chunks * C + g4; tok < p.L; tok += 4) dV[tok * row] = raw(0);
    if (!p.dh0) return;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = 16 * t + 4 * g4 + r;
            if (d < p.dk) p.dh0[hat + d] = S[t][r];
        }
}

template <typename E, int DK>
int launch(const DeltaParams& p, hipStream_t stream) {
    typedef Mat<E> M;
    typedef ChunkMats<E> CM;
    constexpr size_t bytes = (2 * M::kChunk * (DK + M::kPad) + CM::kAll * M::kChunk * CM::kPitch) * sizeof(typename M::raw) +
                             3 * M::kChunk * sizeof(float);
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_bwd_kernel<E, DK>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + kCols - 1) / kCols));
    delta_bwd_kernel<E, DK><<<wgs, kThreads, bytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_bwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        return cls::launch<decltype(e), decltype(dk)::value>(p, stream);
    });
}
