// Gated delta rule over whole sequences: the walk over the chunks.  A wave has 16
// columns of the state S [dk, dv] in its registers and takes them through all
// chunks of a sequence; columns do not meet, so waves only share what the
// workgroup stages in LDS for them: the chunk's K, Q, T, P and factors.  Per chunk
//     R = beta (V - e^gamma K S),  N = T R,  Y = scale (e^gamma Q S + P N),
//     S' = e^gamma_C S + K^T (e^(gamma_C - gamma) N)
// where K S, T R and K^T N reach the state and take computed operands in two
// parts, and Q S and P N only reach y and take them in one.
#include <hip/hip_runtime.h>

#include "delta.hpp"
#include "device_once.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;  // of dv to a workgroup

template <typename E, int DK>
__global__ __launch_bounds__(kThreads) void delta_fwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef ChunkMats<E> CM;
    constexpr int C = M::kChunk, NT = C / 16, KT = DK / 16;
    constexpr int KP = DK + M::kPad, MP = CM::kPitch, NM = CM::kParts + 1;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    raw* sK = reinterpret_cast<raw*>(lds);
    raw* sQ = sK + C * KP;
    raw* sM = sQ + C * KP;  // T (its parts), P
    float* sV = reinterpret_cast<float*>(sM + NM * C * MP);

    const int nblk = (p.dv + kCols - 1) / kCols;
    const int blk = blockIdx.x % nblk, h = blockIdx.x / nblk % p.H, b = blockIdx.x / nblk / p.H;
    const int end = seq_end(p.seqlens, b, p.L), kh = h / (p.H / p.Hk);
    const int tid = threadIdx.x, l16 = lane16(), g4 = group4();
    const int n = blk * kCols + (tid >> 6) * 16 + l16;
    const bool on = n < p.dv, wave_on = blk * kCols + (tid >> 6) * 16 < p.dv;

    const raw* K = static_cast<const raw*>(p.k) + b * p.sk.batch + kh * p.sk.head;
    const raw* Q = static_cast<const raw*>(p.q) + b * p.sq.batch + kh * p.sq.head;
    const raw* V = static_cast<const raw*>(p.v) + b * p.sv.batch + h * p.sv.head + n;
    raw* Y = static_cast<raw*>(p.y) + (int64_t(b) * p.L * p.H + h) * p.dv + n;
    const int64_t row = int64_t(p.H) * p.dv;  // of a token

    f32x4 S[KT];
    const int64_t hat = ((int64_t(b) * p.H + h) * p.dv + n) * p.dk;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = 16 * t + 4 * g4 + r;
            S[t][r] = p.h0 && on && d < p.dk ? p.h0[hat + d] : 0.0f;
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
                v[t][r] = on && tok < end ? V[tok * p.sv.token] : raw(0);
            }
    };
    if (chunks > 0) fetch(0);
    for (int c = 0; c < chunks; ++c) {
        const int t0 = c * C;
        __syncthreads();  // the chunk before is read
        rk.store(sK, KP);
        rq.store(sQ, KP);
#pragma unroll
        for (int m = 0; m < NM; ++m) rm[m].store(sM + m * C * MP, MP);
        if (tid < 3 * C) sV[tid] = rv;
        f32x4 R[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) R[t][r] = E::get(v[t][r]);
        __syncthreads();
        if (c + 1 < chunks) fetch(c + 1);
        if (!wave_on) continue;

        if (p.states && on) {
            float* to = p.states + (((int64_t(b) * p.nchunk + c) * p.H + h) * p.dk) * p.dv + n;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int d = 16 * t + 4 * g4 + r;
                    if (d < p.dk) to[int64_t(d) * p.dv] = S[t][r];
                }
        }
        f32x4 ks[NT], O[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) ks[t] = O[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) {
            const Two<E> st = two<E>(S[2 * s], S[2 * s + 1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                ks[t] = mma2<E>(M::rows(sK + (16 * t + l16) * KP + 32 * s), st, ks[t]);
                O[t] = M::mma(M::rows(sQ + (16 * t + l16) * KP + 32 * s), st.hi, O[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 e = *reinterpret_cast<const f32x4*>(sV + 16 * t + 4 * g4);
            const f32x4 be = *reinterpret_cast<const f32x4*>(sV + 2 * C + 16 * t + 4 * g4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                R[t][r] = be[r] * fmaf(-e[r], ks[t][r], R[t][r]);
                O[t][r] *= e[r];
            }
        }
        // N = R + (T - I) R: tokens up to 32 (t / 2 + 1) reach tile t
        f32x4 N[NT];
        Two<E> rr[NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) rr[s] = two<E>(R[2 * s], R[2 * s + 1]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            N[t] = R[t];
#pragma unroll
            for (int s = 0; s <= t / 2; ++s) {
                Two<E> T;
                T.hi = M::rows(sM + (16 * t + l16) * MP + 32 * s);
                if constexpr (M::kSplit) T.lo = M::rows(sM + C * MP + (16 * t + l16) * MP + 32 * s);
                N[t] = mma3<E>(T, rr[s], N[t]);
            }
        }
        typename M::frag nf[NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) nf[s] = M::cvt(N[2 * s], N[2 * s + 1]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int s = 0; s <= t / 2; ++s)
                O[t] = M::mma(M::rows(sM + CM::kParts * C * MP + (16 * t + l16) * MP + 32 * s), nf[s], O[t]);
            if (on)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = t0 + 16 * t + 4 * g4 + r;
                    if (tok >= p.L) continue;
                    Y[tok * row] = tok < end ? E::put(p.scale * O[t][r]) : raw(0);
                    if (p.fixes && tok < end) p.fixes[(int64_t(b) * p.L + tok) * row + int64_t(h) * p.dv + n] = N[t][r];
                }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 e = *reinterpret_cast<const f32x4*>(sV + C + 16 * t + 4 * g4);
#pragma unroll
            for (int r = 0; r < 4; ++r) N[t][r] *= e[r];
        }
        const float fade = sV[C - 1];
        Two<E> nn[NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) nn[s] = two<E>(N[2 * s], N[2 * s + 1]);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            S[t] *= fade;
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) S[t] = mma2<E>(M::cols(sK + 32 * s * KP + 16 * t, KP), nn[s], S[t]);
        }
    }
    if (!on) return;
    for (int tok = chunks * C + g4; tok < p.L; tok += 4) Y[tok * row] = raw(0);
    if (!p.h_last) return;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = 16 * t + 4 * g4 + r;
            if (d < p.dk) p.h_last[hat + d] = S[t][r];
        }
}

template <typename E, int DK>
int launch(const DeltaParams& p, hipStream_t stream) {
    typedef Mat<E> M;
    typedef ChunkMats<E> CM;
    constexpr size_t bytes = (2 * M::kChunk * (DK + M::kPad) + (CM::kParts + 1) * M::kChunk * CM::kPitch) * sizeof(typename M::raw) +
                             3 * M::kChunk * sizeof(float);
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_fwd_kernel<E, DK>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + kCols - 1) / kCols));
    delta_fwd_kernel<E, DK><<<wgs, kThreads, bytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_fwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        return cls::launch<decltype(e), decltype(dk)::value>(p, stream);
    });
}
