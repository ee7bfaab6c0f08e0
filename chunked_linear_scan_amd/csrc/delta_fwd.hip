// Gated delta rule over whole sequences: the walk over the chunks.  A wave has 16
// columns of the state S [dk, dv] in its registers and takes them through all
// chunks of a sequence; columns do not meet, so waves only share what is
// staged in LDS for them: the chunk's K, Q, T - I, P and factors.  Per chunk
//     R = beta (V - e^gamma K S),  N = R + (T - I) R,  Y = scale (e^gamma Q S + P N),
//     S' = e^gamma_C S + K^T (e^(gamma_C - gamma) N)
// where K S, T R and K^T N reach the state and take computed operands in two
// parts, and Q S and P N only reach y and take them in one.
#include <hip/hip_runtime.h>

#include "delta_walk.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

// KEEP: with the states and corrections that the gradients need.
template <typename E, int DK, int WAVES, bool KEEP>
__global__ __launch_bounds__(64 * (WAVES + 4), 2) void delta_fwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::frag frag;
    constexpr int kParts = ChunkMats<E>::kParts, NM = kParts + 1;  // T - I in its parts, P
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
        const WalkColumns w{p.v, p.sv, p.y, bool(p.vec_v), bool(p.vec_out)};
        walk_load<E, DK, NM, WAVES>(p, w, lds, b, h, blk * Lds::kCols, end, 0, 1, chunks);
        return;
    }
    const int l16 = lane16(), g4 = group4();
    const int n = blk * Lds::kCols + wave * 16 + l16;  // the lane's column
    const bool wave_on = blk * Lds::kCols + wave * 16 < p.dv;

    f32x4 S[KT];
    load_state<KT>(S, p.h0, int64_t(b) * p.H + h, n, p);
    const typename Lds::KTile kt;
    const typename Lds::MTile mt;
    const typename Lds::XTile xt;
    const int oy = 4 * g4 * Lds::YP + wave * 16 + l16;

    walk<Lds>(lds, chunks, [&](int c, const Lds& m) {
        if (!wave_on) return;
        const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
        const auto factors = [&](int which, int t) { return *reinterpret_cast<const f32x4*>(m.v + which * C + 16 * t + 4 * g4); };
        if constexpr (KEEP) store_state<KT>(S, p.states, chunk, n, p);

        // K S and Q S; the operands of a step are read, and S is taken apart, while the one before is multiplied
        f32x4 ks[NT], O[NT], R[NT], a[NT], e[NT];
        frag k[2][NT], q[2][NT], v[NT / 2];
        Two<E> T[NT][NT / 2], st[2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            ks[t] = O[t] = f32x4{0, 0, 0, 0};
            if (!AHEAD) continue;
            k[0][t] = kt.rows(m.k, t, 0);
            q[0][t] = kt.rows(m.q, t, 0);
        }
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) v[s] = xt.cols(m.x, s, wave);
#pragma unroll
        for (int t = 0; t < NT; ++t) a[t] = factors(kBeta, t);
        st[0] = two<E>(S[0], S[1]);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int at = AHEAD ? s & 1 : 0, at1 = AHEAD ? at ^ 1 : 0;
            if (!AHEAD || s + 1 < KS) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    k[at1][t] = kt.rows(m.k, t, AHEAD ? s + 1 : s);
                    q[at1][t] = kt.rows(m.q, t, AHEAD ? s + 1 : s);
                }
            }
            if (s + 1 == KS) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    a[t] = factors(kBetaStart, t);
                    e[t] = factors(kRead, t);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u <= t / 2; ++u) {
                        T[t][u].hi = mt.rows(m.m, t, u);
                        if constexpr (M::kSplit) T[t][u].lo = mt.rows(m.m + Lds::MS, t, u);
                    }
            }
            fence();
            if (s + 1 < KS) st[(s + 1) & 1] = two<E>(S[2 * s + 2], S[2 * s + 3]);
            if (s == 0) {  // beta V
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) R[t][r] = a[t][r] * M::at(v[t / 2], 4 * (t & 1) + r);
            }
            if constexpr (M::kSplit) {
#pragma unroll
                for (int t = 0; t < NT; ++t) ks[t] = M::mma(k[at][t], st[s & 1].lo, ks[t]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) ks[t] = M::mma(k[at][t], st[s & 1].hi, ks[t]);
            if (s + 1 == KS) fence();
#pragma unroll
            for (int t = 0; t < NT; ++t) O[t] = M::mma(q[at][t], st[s & 1].hi, O[t]);
            if (s + 1 < KS) {
                interleave<3 * NT, 4>();
                fence();
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) R[t][r] = fmaf(-a[t][r], ks[t][r], R[t][r]);
        // N = R + (T - I) R: tokens up to 32 (t / 2 + 1) reach tile t
        frag P[NT][NT / 2];
        f32x4 N[NT];
        Two<E> rr = two<E>(R[0], R[1]);
        interleave<NT, 10>();
        fence();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int s = 0; s <= t / 2; ++s) P[t][s] = mt.rows(m.m + kParts * Lds::MS, t, s);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            N[t] = R[t];
            O[t] *= e[t];
            e[t] = factors(kWrite, t);
        }
        const float fade = m.v[kStart * C + C - 1];
        frag kc[2][2][NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) {
            if (!AHEAD) continue;
            kc[0][0][s] = kt.cols(m.k, s, 0);
            kc[0][1][s] = kt.cols(m.k, s, 1);
        }
        Two<E> nn[NT / 2];
        frag nf[NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) {
            Two<E> next;
            if (s + 1 < NT / 2) next = two<E>(R[2 * s + 2], R[2 * s + 3]);
            if constexpr (M::kSplit) {
#pragma unroll
                for (int t = 2 * s; t < NT; ++t) N[t] = M::mma(T[t][s].lo, rr.hi, N[t]);
#pragma unroll
                for (int t = 2 * s; t < NT; ++t) N[t] = M::mma(T[t][s].hi, rr.lo, N[t]);
            }
#pragma unroll
            for (int t = 2 * s; t < NT; ++t) N[t] = M::mma(T[t][s].hi, rr.hi, N[t]);
            if (s > 0) {  // tiles 2 s - 2 and 2 s - 1 are done
                nn[s - 1] = two<E>(N[2 * s - 2] * e[2 * s - 2], N[2 * s - 1] * e[2 * s - 1]);
                nf[s - 1] = M::cvt(N[2 * s - 2], N[2 * s - 1]);
            }
            rr = next;
            interleave<3 * (NT - 2), 4>();
            fence();
        }
        nn[NT / 2 - 1] = two<E>(N[NT - 2] * e[NT - 2], N[NT - 1] * e[NT - 1]);
        nf[NT / 2 - 1] = M::cvt(N[NT - 2], N[NT - 1]);
        // the state, two tiles in turn (a product waits for the one before it on its tile), and beside it y
#pragma unroll
        for (int t = 0; t < KT; t += 2) {
            const int at = AHEAD ? t / 2 & 1 : 0, at1 = AHEAD ? at ^ 1 : 0;
            if (!AHEAD || t + 2 < KT) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int s = 0; s < NT / 2; ++s) kc[at1][u][s] = kt.cols(m.k, s, t + (AHEAD ? 2 : 0) + u);
            }
            fence();
#pragma unroll
            for (int u = 0; u < 2; ++u) S[t + u] *= fade;
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) {
                if constexpr (M::kSplit) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) S[t + u] = M::mma(kc[at][u][s], nn[s].lo, S[t + u]);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) S[t + u] = M::mma(kc[at][u][s], nn[s].hi, S[t + u]);
                if (t < NT) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (s <= (t + u) / 2) O[t + u] = M::mma(P[t + u][s], nf[s], O[t + u]);
                }
            }
            if (t >= NT && t < 2 * NT) {
#pragma unroll
                for (int u = 0; u < 2; ++u) put_column<E, Lds::YP>(m.y + oy, t + u - NT, O[t + u - NT]);
            }
        }
#pragma unroll
        for (int t = KT >= 2 * NT ? NT : 0; t < NT; ++t) put_column<E, Lds::YP>(m.y + oy, t, O[t]);
        if constexpr (KEEP) store_tokens<C>(N, p.fixes, chunk, n, p);
        settle(S[KT - 1]);
    });
    if (p.h_last) store_state<KT>(S, p.h_last, int64_t(b) * p.H + h, n, p);
}

template <typename E, int DK, int WAVES, bool KEEP>
int launch(const DeltaParams& p, hipStream_t stream) {
    typedef WalkLds<E, DK, ChunkMats<E>::kParts + 1, WAVES> Lds;
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_fwd_kernel<E, DK, WAVES, KEEP>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, Lds::kBytes) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + Lds::kCols - 1) / Lds::kCols));
    delta_fwd_kernel<E, DK, WAVES, KEEP><<<wgs, Lds::kThreads, Lds::kBytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_fwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        typedef decltype(e) E;
        constexpr int DK = decltype(dk)::value;
        if (cls::walk_waves(p) == 2)
            return p.states ? cls::launch<E, DK, 2, true>(p, stream) : cls::launch<E, DK, 2, false>(p, stream);
        return p.states ? cls::launch<E, DK, 4, true>(p, stream) : cls::launch<E, DK, 4, false>(p, stream);
    });
}
