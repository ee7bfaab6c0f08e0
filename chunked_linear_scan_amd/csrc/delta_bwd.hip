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

template <typename E, int DK, int WAVES>
__global__ __launch_bounds__(64 * (WAVES + 4), 2) void delta_bwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::frag frag;
    constexpr int kParts = ChunkMats<E>::kParts, NM = ChunkMats<E>::kAll;  // T - I, P, in their parts
    typedef WalkLds<E, DK, NM, WAVES> Lds;
    constexpr int C = M::kChunk, NT = C / 16, KT = DK / 16, KS = DK / 32;
    constexpr bool AHEAD = DK <= 128;  // operands are read a step before their products: registers for it
    extern __shared__ __attribute__((aligned(16))) char lds[];

    const int nblk = (p.dv + Lds::kCols - 1) / Lds::kCols;
    const int rep = p.H / p.Hk;
    const UnitPart u = unit_part(p.batch * p.Hk, rep * nblk);
    const int blk = u.part % nblk, h = u.unit % p.Hk * rep + u.part / nblk, b = u.unit / p.Hk;
    const int end = seq_end(p.seqlens, b, p.L), chunks = (end + C - 1) / C;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= WAVES) {
        const WalkColumns w{p.dy, p.sdy, p.dv_, bool(p.vec_dy), bool(p.vec_out)};
        walk_load<E, DK, NM, WAVES>(p, w, lds, b, h, blk * Lds::kCols, end, chunks - 1, -1, chunks);
        return;
    }
    const int l16 = lane16(), g4 = group4();
    const int n = blk * Lds::kCols + wave * 16 + l16;  // the lane's column
    const bool wave_on = blk * Lds::kCols + wave * 16 < p.dv;

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
            if (AHEAD) k[0][t] = kt.rows(m.k, t, 0);
        }
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) y[s] = xt.cols(m.x, s, wave);
        st[0] = two<E>(S[0], S[1]);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int at = AHEAD ? s & 1 : 0, at1 = AHEAD ? at ^ 1 : 0;
            if (!AHEAD || s + 1 < KS) {
#pragma unroll
                for (int t = 0; t < NT; ++t) k[at1][t] = kt.rows(m.k, t, AHEAD ? s + 1 : s);
            }
            if (s < NT / 2) {  // P of outputs 32 s.., which reach the tiles up to theirs
#pragma unroll
                for (int t = 0; t <= 2 * s + 1; ++t) {
                    P[t][s].hi = mt.cols(m.m + kParts * Lds::MS, s, t);
                    if constexpr (M::kSplit) P[t][s].lo = mt.cols(m.m + (kParts + 1) * Lds::MS, s, t);
                }
            }
            fence();
            if (s + 1 < KS) st[(s + 1) & 1] = two<E>(S[2 * s + 2], S[2 * s + 3]);
            if constexpr (M::kSplit) {
#pragma unroll
                for (int t = 0; t < NT; ++t) dN[t] = M::mma(k[at][t], st[s & 1].lo, dN[t]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) dN[t] = M::mma(k[at][t], st[s & 1].hi, dN[t]);
            if (s > 0 && s <= NT / 2) {
#pragma unroll
                for (int t = 0; t <= 2 * s - 1; ++t) later[t] = M::mma(P[t][s - 1].hi, y[s - 1], later[t]);
                if constexpr (M::kSplit) {
#pragma unroll
                    for (int t = 0; t <= 2 * s - 1; ++t) later[t] = M::mma(P[t][s - 1].lo, y[s - 1], later[t]);
                }
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
        frag kc[2][2][NT / 2], qc[2][2][NT / 2];
        const auto next = [&](int at, int t) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int s = 0; s < NT / 2; ++s) {
                    qc[at][u][s] = kt.cols(m.q, s, t + u);
                    kc[at][u][s] = kt.cols(m.k, s, t + u);
                }
        };
        if (AHEAD) next(0, 0);
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) a[s] = two<E>(-(bs[2 * s] * Z[2 * s]), -(bs[2 * s + 1] * Z[2 * s + 1]));
        store_tokens<C>(Z, p.z, chunk, n, p);
        // two tiles in turn: a product waits for the one before it on its tile
#pragma unroll
        for (int t = 0; t < KT; t += 2) {
            const int at = AHEAD ? t / 2 & 1 : 0;
            if (!AHEAD) next(0, t);
            else if (t + 2 < KT) next(at ^ 1, t + 2);
            fence();
#pragma unroll
            for (int u = 0; u < 2; ++u) S[t + u] *= fade;
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) {
                if constexpr (M::kSplit) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) S[t + u] = M::mma(qc[at][u][s], q[s].lo, S[t + u]);
#pragma unroll
                    for (int u = 0; u < 2; ++u) S[t + u] = M::mma(kc[at][u][s], a[s].lo, S[t + u]);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) S[t + u] = M::mma(qc[at][u][s], q[s].hi, S[t + u]);
#pragma unroll
                for (int u = 0; u < 2; ++u) S[t + u] = M::mma(kc[at][u][s], a[s].hi, S[t + u]);
            }
            if (t < NT) {
#pragma unroll
                for (int u = 0; u < 2; ++u) put_column<E, Lds::YP>(m.y + oy, t + u, be[t + u] * Z[t + u]);
            }
        }
        settle(S[KT - 1]);
    });
    if (p.dh0) store_state<KT>(S, p.dh0, int64_t(b) * p.H + h, n, p);
}

template <typename E, int DK, int WAVES>
int launch(const DeltaParams& p, hipStream_t stream) {
    typedef WalkLds<E, DK, ChunkMats<E>::kAll, WAVES> Lds;
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_bwd_kernel<E, DK, WAVES>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, Lds::kBytes) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + Lds::kCols - 1) / Lds::kCols));
    delta_bwd_kernel<E, DK, WAVES><<<wgs, Lds::kThreads, Lds::kBytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_bwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        typedef decltype(e) E;
        constexpr int DK = decltype(dk)::value;
        return cls::walk_waves(p) == 2 ? cls::launch<E, DK, 2>(p, stream) : cls::launch<E, DK, 4>(p, stream);
    });
}
