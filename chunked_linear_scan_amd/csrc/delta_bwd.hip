// Gradients of the gated delta rule, the part that walks the chunks: from the
// last to the first, a wave with 16 columns of dS, the gradient of the state, as
// the forward walk has them of S.  Per chunk, dS being that of the state behind it,
//     dN = e^(gamma_C - gamma) K dS + scale P^T dY,  Z = T^T dN,  dV = dR = beta Z,
//     dS' = e^gamma_C dS + scale Q^T e^gamma dY - K^T e^gamma dR.
// dS of every chunk and Z go to memory for the kernel that takes the chunks'
// other gradients all at once (delta_grad.hip).
#include <hip/hip_runtime.h>

#include "delta_walk.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

template <typename E, int DK>
__global__ __launch_bounds__(kWalkThreads) void delta_bwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::frag frag;
    constexpr int kParts = ChunkMats<E>::kParts, NM = ChunkMats<E>::kAll;  // T - I, P, in their parts
    typedef WalkLds<E, DK, NM> Lds;
    constexpr int C = M::kChunk, NT = C / 16, KT = DK / 16, KS = DK / 32;
    extern __shared__ __attribute__((aligned(16))) char lds[];

    const int nblk = (p.dv + kWalkCols - 1) / kWalkCols;
    const int blk = blockIdx.x % nblk, h = blockIdx.x / nblk % p.H, b = blockIdx.x / nblk / p.H;
    const int end = seq_end(p.seqlens, b, p.L), chunks = (end + C - 1) / C;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= 4) {
        const WalkColumns w{p.dy, p.sdy, p.dv_, bool(p.vec_dy), bool(p.vec_out)};
        walk_load<E, DK, NM>(p, w, lds, b, h, blk * kWalkCols, end, chunks - 1, -1, chunks);
        return;
    }
    const int l16 = lane16(), g4 = group4();
    const int n = blk * kWalkCols + wave * 16 + l16;  // the lane's column
    const bool wave_on = blk * kWalkCols + wave * 16 < p.dv;

    f32x4 S[KT];
    load_state<KT>(S, p.dh_last, int64_t(b) * p.H + h, n, p);
    const typename Lds::KTile kt;
    const typename Lds::MTile mt;
    const typename Lds::XTile xt;
    const int oy = 4 * g4 * Lds::YP + wave * 16 + l16;

    walk<Lds>(lds, chunks, [&](int i, const Lds& m) {
        if (!wave_on) return;
        const int64_t chunk = (int64_t(b) * p.nchunk + chunks - 1 - i) * p.H + h;
        const auto factors = [&](int which, int t) { return *reinterpret_cast<const f32x4*>(m.v + which * C + 16 * t + 4 * g4); };
        store_state<KT>(S, p.dstates, chunk, n, p);

        // K dS, and beside it P^T dY
        f32x4 dN[NT], later[NT], e[NT];
        frag k[2][NT], y[NT / 2];
        Two<E> st[2], P[NT][NT / 2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dN[t] = later[t] = f32x4{0, 0, 0, 0};
            k[0][t] = kt.rows(m.k, t, 0);
        }
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) y[s] = xt.cols(m.x, s, wave);
        st[0] = two<E>(S[0], S[1]);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int at = s & 1;
            if (s + 1 < KS) {
#pragma unroll
                for (int t = 0; t < NT; ++t) k[at ^ 1][t] = kt.rows(m.k, t, s + 1);
            }
            if (s < NT / 2) {  // P of outputs 32 s.., which reach the tiles up to theirs
#pragma unroll
                for (int t = 0; t <= 2 * s + 1; ++t) {
                    P[t][s].hi = mt.cols(m.m + kParts * Lds::MS, s, t);
                    if constexpr (M::kSplit) P[t][s].lo = mt.cols(m.m + (kParts + 1) * Lds::MS, s, t);
                }
            }
            fence();
            if (s + 1 < KS) st[at ^ 1] = two<E>(S[2 * s + 2], S[2 * s + 3]);
#pragma unroll
            for (int t = 0; t < NT; ++t) dN[t] = mma2<E>(k[at][t], st[at], dN[t]);
            if (s > 0 && s <= NT / 2) {
#pragma unroll
                for (int t = 0; t <= 2 * s - 1; ++t) later[t] = mma2<E>(P[t][s - 1], y[s - 1], later[t]);
            }
            interleave<2 * NT, 4>();
            fence();
        }
        // the operands of the rest
        Two<E> T[NT][NT / 2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            e[t] = factors(kWrite, t);
#pragma unroll
            for (int s = t / 2; s < NT / 2; ++s) {
                T[t][s].hi = mt.cols(m.m, s, t);
                if constexpr (M::kSplit) T[t][s].lo = mt.cols(m.m + Lds::MS, s, t);
            }
        }
        fence();
        if constexpr (KS <= NT / 2) {
#pragma unroll
            for (int t = 0; t < NT; ++t) later[t] = mma2<E>(P[t][NT / 2 - 1], y[NT / 2 - 1], later[t]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) dN[t][r] = fmaf(dN[t][r], e[t][r], p.scale * later[t][r]);
        // Z = dN + (T - I)^T dN, from the last tokens: 32 s.. reach the tiles up to theirs
        f32x4 Z[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) Z[t] = dN[t];
        Two<E> dn = two<E>(dN[NT - 2], dN[NT - 1]);
        // beside it what dY adds to dS
        Two<E> q[NT / 2], a[NT / 2];
        f32x4 be[NT], bs[NT];
#pragma unroll
        for (int s = NT / 2 - 1; s >= 0; --s) {
            be[2 * s] = factors(kBeta, 2 * s);
            be[2 * s + 1] = factors(kBeta, 2 * s + 1);
            bs[2 * s] = factors(kBetaStart, 2 * s);
            bs[2 * s + 1] = factors(kBetaStart, 2 * s + 1);
            f32x4 r0 = factors(kRead, 2 * s), r1 = factors(kRead, 2 * s + 1);
            fence();
            Two<E> next;
            if (s > 0) next = two<E>(dN[2 * s - 2], dN[2 * s - 1]);
            if constexpr (M::kSplit) {
#pragma unroll
                for (int t = 0; t <= 2 * s + 1; ++t) Z[t] = M::mma(T[t][s].lo, dn.hi, Z[t]);
#pragma unroll
                for (int t = 0; t <= 2 * s + 1; ++t) Z[t] = M::mma(T[t][s].hi, dn.lo, Z[t]);
            }
#pragma unroll
            for (int t = 0; t <= 2 * s + 1; ++t) Z[t] = M::mma(T[t][s].hi, dn.hi, Z[t]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                r0[r] *= M::at(y[s], r);
                r1[r] *= M::at(y[s], 4 + r);
            }
            q[s] = two<E>(r0, r1);
            dn = next;
            interleave<3 * (NT - 2), 6>();
            fence();
        }
        const float fade = m.v[kStart * C + C - 1];
        frag kc[2][NT / 2], qc[2][NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) {
            qc[0][s] = kt.cols(m.q, s, 0);
            kc[0][s] = kt.cols(m.k, s, 0);
        }
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) a[s] = two<E>(-(bs[2 * s] * Z[2 * s]), -(bs[2 * s + 1] * Z[2 * s + 1]));
        store_tokens<C>(Z, p.z, chunk, n, p);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            if (t + 1 < KT) {
#pragma unroll
                for (int s = 0; s < NT / 2; ++s) {
                    qc[(t + 1) & 1][s] = kt.cols(m.q, s, t + 1);
                    kc[(t + 1) & 1][s] = kt.cols(m.k, s, t + 1);
                }
            }
            fence();
            S[t] *= fade;
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) {
                S[t] = mma2<E>(qc[t & 1][s], q[s], S[t]);
                S[t] = mma2<E>(kc[t & 1][s], a[s], S[t]);
            }
            if (t < NT) put_column<E, Lds::YP>(m.y + oy, t, be[t] * Z[t]);
        }
        settle(S[KT - 1]);
    });
    if (p.dh0) store_state<KT>(S, p.dh0, int64_t(b) * p.H + h, n, p);
}

template <typename E, int DK>
int launch(const DeltaParams& p, hipStream_t stream) {
    constexpr int bytes = WalkLds<E, DK, ChunkMats<E>::kAll>::kBytes;
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_bwd_kernel<E, DK>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + kWalkCols - 1) / kWalkCols));
    delta_bwd_kernel<E, DK><<<wgs, kWalkThreads, bytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_bwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        return cls::launch<decltype(e), decltype(dk)::value>(p, stream);
    });
}
