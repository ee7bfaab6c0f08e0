// Gated delta rule over whole sequences: the walk over the chunks.  Columns of the
// state S [dk, dv] stay in registers, 16 of them in two waves, and go through all
// chunks of a sequence.  Columns do not meet: a workgroup's waves share the chunk's
// K, Q, T - I, P and factors in LDS, and the two waves of the same columns exchange
// their halves of K S and Q S, R, and N.  Per chunk
//     R = beta (V - e^gamma K S),  N = R + (T - I) R,  Y = scale (e^gamma Q S + P N),
//     S' = e^gamma_C S + K^T (e^(gamma_C - gamma) N)
// with all computed operands in two parts: y, too, is off by its own rounding and little else (with one part of
// S, P and N where only y reads them its 2-norm error was 2.8e-3 in bf16, of which 1.7e-3 are its rounding).
#include <hip/hip_runtime.h>

#include "delta_walk.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

// KEEP: with the states and corrections that the gradients need.
template <typename E, int DK, bool KEEP, int TILES>
__global__ __launch_bounds__(walk_threads(TILES)) void delta_fwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef HalfOps<E> Op;
    typedef typename M::frag frag;
    typedef typename Op::op op;
    constexpr bool kSplit = M::kSplit;
    constexpr int kParts = ChunkMats<E>::kParts, NM = ChunkMats<E>::kAll;  // T - I, P, in their parts
    typedef WalkLds<E, DK, NM> Lds;
    constexpr int C = M::kChunk, NT = C / 16, OT = Op::OT;      // tiles of a chunk's tokens, of a half's
    constexpr int KT = DK / 32, KS = DK / 64;                   // of a wave's half of the keys' elements: tiles, steps
    extern __shared__ __attribute__((aligned(16))) char lds[];

    const int nblk = (p.dv + walk_cols(TILES) - 1) / walk_cols(TILES);
    const int rep = p.H / p.Hk;
    const UnitPart u = unit_part(p.batch * p.Hk, rep * nblk);
    const int blk = u.part % nblk, h = u.unit % p.Hk * rep + u.part / nblk, b = u.unit / p.Hk;
    const int end = seq_end(p.seqlens, b, p.L), chunks = (end + C - 1) / C;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= 2 * TILES) {
        const WalkColumns w{p.v, p.sv, p.y, bool(p.vec_out), 1.0f};
        walk_load<E, DK, NM, TILES, false>(p, w, lds, b, h, blk * walk_cols(TILES), end, 0, 1, chunks);
        return;
    }
    const int a = wave & 1, tile = wave >> 1;  // the wave's half, its tile of the columns
    const int l16 = lane16(), g4 = group4();
    const int n = blk * walk_cols(TILES) + tile * 16 + l16;  // the lane's column

    f32x4 S[KT];
    load_state<KT>(S, p.h0, int64_t(b) * p.H + h, n, a * (DK / 2), p);
    const typename Lds::KTile kt(a * (DK / 2));
    const typename Lds::MTile mt, xt(16 * tile);
    const Exchange ex(lds, wave, Lds::kSlots);
    const int oy = (C / 2 * a + 4 * g4) * Lds::YP + tile * 16 + l16;
    constexpr int HALF = C / 2 * Lds::KTile::kPitch;  // of K or Q

    walk<Lds>(lds, chunks, [&](int c, const Lds& m) {
        const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
        const auto factors = [&](int which, int j) {
            return *reinterpret_cast<const f32x4*>(m.v + which * C + C / 2 * a + 16 * j + 4 * g4);
        };
        // operands of tiles j < OT of the wave's own tokens, then of the other half's
        const auto* ko = m.k + a * HALF;
        const auto* kx = m.k + (1 - a) * HALF;
        const auto* qo = m.q + a * HALF;
        const auto* qx = m.q + (1 - a) * HALF;
        const auto read = [&](frag (&k)[NT], frag (&q)[NT], int s) {
#pragma unroll
            for (int j = 0; j < OT; ++j) {
                k[OT + j] = kt.rows(kx, j, s);
                k[j] = kt.rows(ko, j, s);
                q[OT + j] = kt.rows(qx, j, s);
                q[j] = kt.rows(qo, j, s);
            }
        };

        // the wave's share of K S and Q S: the other half's first, so that they leave early
        f32x4 ks[NT], O[NT], R[OT], be[OT], bs[OT], e[OT];
        frag k[2][NT], q[2][NT];
        Two<E> st[2];
        read(k[0], q[0], 0);
        const op v = Op::tokens(xt, m.x, a, 0);
        op Th[OT], Tl[OT], Ph[OT], Pl[OT], Xh[OT], Xl[OT], Yh[OT], Yl[OT];
#pragma unroll
        for (int j = 0; j < OT; ++j) be[j] = factors(kBeta, j);
#pragma unroll
        for (int t = 0; t < NT; ++t) ks[t] = O[t] = f32x4{0, 0, 0, 0};
        st[0] = two<E>(S[0], S[1]);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (s + 1 < KS) {
                read(k[(s + 1) & 1], q[(s + 1) & 1], s + 1);
            } else {
#pragma unroll
                for (int j = 0; j < OT; ++j) {
                    bs[j] = factors(kBetaStart, j);
                    e[j] = factors(kStart, j);
                    Th[j] = Op::rows(mt, m.m, Lds::M1, a, a, j);
                    if constexpr (kSplit) Tl[j] = Op::rows(mt, m.m + Lds::MS, Lds::M1, a, a, j);
                }
            }
            fence();
            if (s + 1 < KS) st[(s + 1) & 1] = two<E>(S[2 * s + 2], S[2 * s + 3]);
            if (s == 0) {  // beta V
#pragma unroll
                for (int j = 0; j < OT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) R[j][r] = be[j][r] * Op::at(v, j, r);
            }
            if constexpr (kSplit) {
#pragma unroll
                for (int t = NT - 1; t >= 0; --t) ks[t] = M::mma(k[s & 1][t], st[s & 1].lo, ks[t]);
#pragma unroll
                for (int t = NT - 1; t >= 0; --t) O[t] = M::mma(q[s & 1][t], st[s & 1].lo, O[t]);
            }
#pragma unroll
            for (int t = NT - 1; t >= 0; --t) ks[t] = M::mma(k[s & 1][t], st[s & 1].hi, ks[t]);
#pragma unroll
            for (int t = NT - 1; t >= 0; --t) O[t] = M::mma(q[s & 1][t], st[s & 1].hi, O[t]);
            interleave<4 * NT, 3>();
            fence();
        }
#pragma unroll
        for (int j = 0; j < OT; ++j) ex.put(j, ks[OT + j]);
#pragma unroll
        for (int j = 0; j < OT; ++j) ex.put(OT + j, O[OT + j]);
        lds_meet();  // 1: both halves' shares
        f32x4 x[2 * OT];
#pragma unroll
        for (int j = 0; j < 2 * OT; ++j) ex.get(j, x[j]);
#pragma unroll
        for (int j = 0; j < OT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) R[j][r] = fmaf(-bs[j][r], ks[j][r] + x[j][r], R[j][r]);
        // N = R + (T - I) R: the first half's tokens reach the second's
        const auto rr = Op::two(R);
        if (a == 0) {
            ex.put(4, rr.hi);
            if constexpr (kSplit) ex.put(5, rr.lo);
        }
        f32x4 N[OT];
#pragma unroll
        for (int j = 0; j < OT; ++j) N[j] = R[j];
        if constexpr (kSplit) {
#pragma unroll
            for (int j = 0; j < OT; ++j) {
                if (small_parts(DK)) N[j] = Op::mma(Tl[j], rr.lo, N[j]);
                N[j] = Op::mma(Tl[j], rr.hi, N[j]);
            }
#pragma unroll
            for (int j = 0; j < OT; ++j) N[j] = Op::mma(Th[j], rr.lo, N[j]);
        }
#pragma unroll
        for (int j = 0; j < OT; ++j) N[j] = Op::mma(Th[j], rr.hi, N[j]);
#pragma unroll
        for (int j = 0; j < OT; ++j) {
            O[j] = (O[j] + x[OT + j]) * e[j];
            e[j] = factors(kWrite, j);
            Ph[j] = Op::rows(mt, m.m + kParts * Lds::MS, Lds::M1, a, a, j);
            if constexpr (kSplit) Pl[j] = Op::rows(mt, m.m + (kParts + 1) * Lds::MS, Lds::M1, a, a, j);
            if (a == 0) continue;
            Xh[j] = Op::rows(mt, m.m, Lds::M1, 1, 0, j);
            if constexpr (kSplit) Xl[j] = Op::rows(mt, m.m + Lds::MS, Lds::M1, 1, 0, j);
            Yh[j] = Op::rows(mt, m.m + kParts * Lds::MS, Lds::M1, 1, 0, j);
            if constexpr (kSplit) Yl[j] = Op::rows(mt, m.m + (kParts + 1) * Lds::MS, Lds::M1, 1, 0, j);
        }
        op kc[2][2];
        kc[0][0] = Op::tokens(kt, m.k, a, 0);
        kc[0][1] = Op::tokens(kt, m.k, a, 1);
        const float fade = m.v[kStart * C + C - 1];
        lds_meet();  // 2: the first half's R
        if (a) {
            auto xx = rr;
            ex.get(4, xx.hi);
            if constexpr (kSplit) {
                ex.get(5, xx.lo);
#pragma unroll
                for (int j = 0; j < OT; ++j) {
                    if (small_parts(DK)) N[j] = Op::mma(Xl[j], xx.lo, N[j]);
                    N[j] = Op::mma(Xl[j], xx.hi, N[j]);
                }
#pragma unroll
                for (int j = 0; j < OT; ++j) N[j] = Op::mma(Xh[j], xx.lo, N[j]);
            }
#pragma unroll
            for (int j = 0; j < OT; ++j) N[j] = Op::mma(Xh[j], xx.hi, N[j]);
        }
        f32x4 w[OT];
#pragma unroll
        for (int j = 0; j < OT; ++j) w[j] = N[j] * e[j];
        const auto nn = Op::two(w);
        const auto nf = Op::two(N);
        ex.put(0, nn.hi);
        if constexpr (kSplit) ex.put(1, nn.lo);
        if (a == 0) {
            ex.put(2, nf.hi);
            if constexpr (kSplit) ex.put(3, nf.lo);
        }
        fence();
        // the state, by the half's own tokens, then by the others; two tiles in turn, as a product waits for the one
        // before it on its tile
        const auto add = [&](int half, const auto& by, bool next) {
#pragma unroll
            for (int t = 0; t < KT; t += 2) {
                const int at = t / 2 & 1;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (t + 2 < KT) kc[at ^ 1][i] = Op::tokens(kt, m.k, half, t + 2 + i);
                    else if (next) kc[at ^ 1][i] = Op::tokens(kt, m.k, 1 - half, i);
                }
                fence();
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (next) S[t + i] *= fade;
                if constexpr (kSplit) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) S[t + i] = Op::mma(kc[at][i], by.lo, S[t + i]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) S[t + i] = Op::mma(kc[at][i], by.hi, S[t + i]);
            }
        };
        if constexpr (KEEP) {
            keep_state<KT>(S, p.states, chunk, n, a * (DK / 2), p);
            store_tokens<C>(N, p.fixes, chunk, n, a, p);
        }
        add(a, nn, true);
        if constexpr (KT / 2 % 2 == 1) {  // the other half's first tiles are where the last ones were not
            kc[0][0] = kc[1][0];
            kc[0][1] = kc[1][1];
        }
        const auto read_out = [&](const op (&h)[OT], const op (&l)[OT], const auto& by) {
            if constexpr (kSplit) {
#pragma unroll
                for (int j = 0; j < OT; ++j) O[j] = Op::mma(l[j], by.hi, O[j]);
#pragma unroll
                for (int j = 0; j < OT; ++j) O[j] = Op::mma(h[j], by.lo, O[j]);
            }
#pragma unroll
            for (int j = 0; j < OT; ++j) O[j] = Op::mma(h[j], by.hi, O[j]);
        };
        read_out(Ph, Pl, nf);
        lds_meet();  // 3: the other half's corrections
        auto xx = nn;
        ex.get(0, xx.hi);
        if constexpr (kSplit) ex.get(1, xx.lo);
        if (a) {
            auto xf = nf;
            ex.get(2, xf.hi);
            if constexpr (kSplit) ex.get(3, xf.lo);
            read_out(Yh, Yl, xf);
        }
        add(1 - a, xx, false);
#pragma unroll
        for (int j = 0; j < OT; ++j) put_column<E, Lds::YP>(m.y + oy, j, p.scale * O[j]);
    });
    if (p.h_last) store_state<KT>(S, p.h_last, int64_t(b) * p.H + h, n, a * (DK / 2), p);
}

template <typename E, int DK, bool KEEP, int TILES>
int launch(const DeltaParams& p, hipStream_t stream) {
    typedef WalkLds<E, DK, ChunkMats<E>::kAll> Lds;
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_fwd_kernel<E, DK, KEEP, TILES>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, Lds::kBytes) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + walk_cols(TILES) - 1) / walk_cols(TILES)));
    delta_fwd_kernel<E, DK, KEEP, TILES><<<wgs, walk_threads(TILES), Lds::kBytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_fwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        typedef decltype(e) E;
        constexpr int DK = decltype(dk)::value;
        return cls::by_tiles(p, [&](auto tiles) {
            constexpr int TILES = decltype(tiles)::value;
            return p.states ? cls::launch<E, DK, true, TILES>(p, stream) : cls::launch<E, DK, false, TILES>(p, stream);
        });
    });
}
