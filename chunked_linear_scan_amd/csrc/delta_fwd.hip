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
template <typename E, int DK, bool KEEP>
__global__ __launch_bounds__(kWalkThreads) void delta_fwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef typename M::frag frag;
    constexpr int kParts = ChunkMats<E>::kParts, NM = kParts + 1;  // T - I in its parts, P
    typedef WalkLds<E, DK, NM> Lds;
    constexpr int C = M::kChunk, NT = C / 16, KT = DK / 16, KS = DK / 32;
    constexpr uint32_t SZ = sizeof(raw);
    extern __shared__ __attribute__((aligned(16))) char lds[];

    const int nblk = (p.dv + kWalkCols - 1) / kWalkCols;
    const int blk = blockIdx.x % nblk, h = blockIdx.x / nblk % p.H, b = blockIdx.x / nblk / p.H;
    const int end = seq_end(p.seqlens, b, p.L), chunks = (end + C - 1) / C;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= 4) {
        walk_load<E, DK, NM>(p, lds, b, h, end, 0, 1, chunks);
        return;
    }
    const int l16 = lane16(), g4 = group4();
    const int n = blk * kWalkCols + wave * 16 + l16;  // the lane's column
    const bool on = n < p.dv, wave_on = blk * kWalkCols + wave * 16 < p.dv;
    const raw* V = static_cast<const raw*>(p.v) + b * p.sv.batch + h * p.sv.head;
    const int64_t row = int64_t(p.H) * p.dv;  // of a token of y
    const int64_t out = int64_t(b) * p.L * row + int64_t(h) * p.dv;
    raw* Y = static_cast<raw*>(p.y) + out;

    f32x4 S[KT];
    load_state<KT>(S, p.h0, int64_t(b) * p.H + h, n, p);
    const LdsTile<E, DK> kt;
    const LdsTile<E, C> mt;
    const uint32_t vrow = uint32_t(p.sv.token) * SZ, yrow = uint32_t(row) * SZ;
    const uint32_t ov = on ? 4 * g4 * vrow + n * SZ : kOutside, oy = on ? 4 * g4 * yrow + n * SZ : kOutside;
    raw v[NT][4];
    f32x4 R[NT];  // V of the chunk to come
    const auto fetch = [&](int c) {
        const Buffer bv = buffer(V + c * C * p.sv.token, (end - c * C) * p.sv.token * SZ);
        const uint32_t at = here(ov);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[t][r] = load_one<E>(bv, at + (16 * t + r) * vrow);
    };
    // Loads are waited for where nothing was stored after them: the counter that a wave waits on counts both in turn.
    const auto arrived = [&] {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) R[t][r] = E::get(v[t][r]);
    };
    if (chunks > 0) {
        fetch(0);
        arrived();
    }

    walk<Lds>(lds, chunks, [&](int c, const Lds& m) {
        if (!wave_on) return;
        const int t0 = c * C;
        if constexpr (KEEP)
            keep_state<KT>(S, p.states, (int64_t(b) * p.nchunk + c) * p.H + h, on ? (4 * g4 * p.dv + n) * 4 : kOutside, p);
        fetch(c + 1 < chunks ? c + 1 : c);

        // K S and Q S; the operands of a step are read, and S is taken apart, while the one before is multiplied
        f32x4 ks[NT], O[NT], e[NT], be[NT];
        frag k[2][NT], q[2][NT];
        Two<E> T[NT][NT / 2], st[2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            ks[t] = O[t] = f32x4{0, 0, 0, 0};
            k[0][t] = kt.rows(m.k, t, 0);
            q[0][t] = kt.rows(m.q, t, 0);
        }
        st[0] = two<E>(S[0], S[1]);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int at = s & 1;
            if (s + 1 < KS) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    k[at ^ 1][t] = kt.rows(m.k, t, s + 1);
                    q[at ^ 1][t] = kt.rows(m.q, t, s + 1);
                }
            } else {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    e[t] = *reinterpret_cast<const f32x4*>(m.v + 16 * t + 4 * g4);
                    be[t] = *reinterpret_cast<const f32x4*>(m.v + 2 * C + 16 * t + 4 * g4);
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
            if (s + 1 < KS) st[at ^ 1] = two<E>(S[2 * s + 2], S[2 * s + 3]);
            if constexpr (M::kSplit) {
#pragma unroll
                for (int t = 0; t < NT; ++t) ks[t] = M::mma(k[at][t], st[at].lo, ks[t]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) ks[t] = M::mma(k[at][t], st[at].hi, ks[t]);
            if (s + 1 == KS) fence();
#pragma unroll
            for (int t = 0; t < NT; ++t) O[t] = M::mma(q[at][t], st[at].hi, O[t]);
            if (s + 1 < KS) {
                interleave<3 * NT, 3>();
                fence();
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) R[t][r] = be[t][r] * fmaf(-e[t][r], ks[t][r], R[t][r]);
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
            e[t] = *reinterpret_cast<const f32x4*>(m.v + C + 16 * t + 4 * g4);  // of the writes, from here on
        }
        const float fade = m.v[C - 1];
        frag kc[2][NT / 2];
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) kc[0][s] = kt.cols(m.k, s, 0);
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
        arrived();
        // the state, and beside it y
        const Buffer by = buffer(Y + t0 * row, int64_t(p.L - t0) * row * SZ);
        const uint32_t to = here(oy);
        const auto put = [&](int t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float y = t0 + C > end && t0 + 16 * t + 4 * g4 + r >= end ? 0.0f : p.scale * O[t][r];  // padding
                store_one<E>(by, to + (16 * t + r) * yrow, y);
            }
        };
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            if (t + 1 < KT) {
#pragma unroll
                for (int s = 0; s < NT / 2; ++s) kc[(t + 1) & 1][s] = kt.cols(m.k, s, t + 1);
            }
            fence();
            S[t] *= fade;
            if (t < NT) {
#pragma unroll
                for (int s = 0; s <= t / 2; ++s) O[t] = M::mma(P[t][s], nf[s], O[t]);
            }
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) S[t] = mma2<E>(kc[t & 1][s], nn[s], S[t]);
            if (t >= NT && t < 2 * NT) put(t - NT);
        }
#pragma unroll
        for (int t = KT >= 2 * NT ? NT : 0; t < NT; ++t) put(t);
        if constexpr (KEEP) {
            const Buffer bf = buffer(p.fixes + out + t0 * row, int64_t(p.L - t0) * row * 4);
            const uint32_t of = here(on ? (4 * g4 * uint32_t(row) + n) * 4 : kOutside);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) store_one<ElemF32>(bf, of + (16 * t + r) * uint32_t(row) * 4, N[t][r]);
        }
    });
    if (p.h_last) store_state<KT>(S, p.h_last, int64_t(b) * p.H + h, n, p);
    if (on)
        for (int tok = chunks * C + g4; tok < p.L; tok += 4) Y[tok * row + n] = raw(0);
}

template <typename E, int DK, bool KEEP>
int launch(const DeltaParams& p, hipStream_t stream) {
    constexpr int bytes = WalkLds<E, DK, ChunkMats<E>::kParts + 1>::kBytes;
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_fwd_kernel<E, DK, KEEP>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + kWalkCols - 1) / kWalkCols));
    delta_fwd_kernel<E, DK, KEEP><<<wgs, kWalkThreads, bytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_fwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        typedef decltype(e) E;
        constexpr int DK = decltype(dk)::value;
        return p.states ? cls::launch<E, DK, true>(p, stream) : cls::launch<E, DK, false>(p, stream);
    });
}
