// Gradients of the gated delta rule, the part that walks the chunks: from the
// last to the first, two waves with 16 columns of dS, the gradient of the state, as
// the forward walk has them of S.  They exchange their halves of K dS, dN, and what
// their tokens add to dS.  Per chunk, dS being that of the state behind it,
//     dN = e^(gamma_C - gamma) K dS + scale P^T dY,  Z = T^T dN,  dV = dR = beta Z,
//     dS' = e^gamma_C dS + scale Q^T e^gamma dY - K^T e^gamma dR.
// dS of every chunk and Z go to memory for the kernel that takes the chunks'
// other gradients all at once (delta_grad.hip).  All of it is times a power of two
// in fp16 (grad_power), which what leaves is divided by.
#include <hip/hip_runtime.h>

#include "delta_walk.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

template <typename E, int DK, int TILES>
__global__ __launch_bounds__(walk_threads(TILES)) void delta_bwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef HalfOps<E> Op;
    typedef typename M::frag frag;
    typedef typename Op::op op;
    constexpr bool kSplit = M::kSplit;
    constexpr int kParts = ChunkMats<E>::kParts, NM = ChunkMats<E>::kAll;  // T - I, P, in their parts
    typedef WalkLds<E, DK, NM> Lds;
    constexpr int C = M::kChunk, NT = C / 16, OT = Op::OT;  // tiles of a chunk's tokens, of a half's
    constexpr int KT = DK / 32, KS = DK / 64;               // of a wave's half of the keys' elements: tiles, steps
    extern __shared__ __attribute__((aligned(16))) char lds[];

    const int nblk = (p.dv + walk_cols(TILES) - 1) / walk_cols(TILES);
    const int rep = p.H / p.Hk;
    const UnitPart u = unit_part(p.batch * p.Hk, rep * nblk);
    const int blk = u.part % nblk, h = u.unit % p.Hk * rep + u.part / nblk, b = u.unit / p.Hk;
    const int end = seq_end(p.seqlens, b, p.L), chunks = (end + C - 1) / C;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= 2 * TILES) {
        const WalkColumns w{p.dy, p.sdy, p.dv_, bool(p.vec_out), grad_power<E>(p, int64_t(b) * p.H + h).dy};
        walk_load<E, DK, NM, TILES, true>(p, w, lds, b, h, blk * walk_cols(TILES), end, chunks - 1, -1, chunks);
        return;
    }
    const int a = wave & 1, tile = wave >> 1;  // the wave's half, its tile of the columns
    const int l16 = lane16(), g4 = group4();
    const int n = blk * walk_cols(TILES) + tile * 16 + l16;  // the lane's column

    const GradPower size = grad_power<E>(p, int64_t(b) * p.H + h);
    const float scale = p.scale * size.ratio;
    f32x4 S[KT];
    load_state<KT>(S, p.dh_last, int64_t(b) * p.H + h, n, a * (DK / 2), p);
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] *= size.up;
    const typename Lds::KTile kt(a * (DK / 2));
    const typename Lds::MTile mt, xt(16 * tile);
    const Exchange ex(lds, wave, Lds::kSlots);
    const int oy = (C / 2 * a + 4 * g4) * Lds::YP + tile * 16 + l16;
    constexpr int HALF = C / 2 * Lds::KTile::kPitch;  // of K

    walk<Lds>(lds, chunks, [&](int i, const Lds& m) {
        const int64_t chunk = (int64_t(b) * p.nchunk + chunks - 1 - i) * p.H + h;
        const auto factors = [&](int which, int j) {
            return *reinterpret_cast<const f32x4*>(m.v + which * C + C / 2 * a + 16 * j + 4 * g4);
        };
        const auto* ko = m.k + a * HALF;
        const auto* kx = m.k + (1 - a) * HALF;
        const auto read = [&](frag (&k)[NT], int s) {
#pragma unroll
            for (int j = 0; j < OT; ++j) {
                k[OT + j] = kt.rows(kx, j, s);
                k[j] = kt.rows(ko, j, s);
            }
        };

        // the wave's share of K dS, tiles of its own tokens and of the other half's, and beside it P^T dY of its own
        f32x4 kd[NT], later[OT], e[OT], rd[OT], be[OT], bs[OT];
        frag k[2][NT];
        Two<E> st[2];
        read(k[0], 0);
        const op yo = Op::tokens(xt, m.x, a, 0), yx = Op::tokens(xt, m.x, 1, 0);  // of dY: own tokens, the second half's
        op Ph[OT], Pl[OT], Th[OT], Tl[OT], Xh[OT], Xl[OT];
#pragma unroll
        for (int j = 0; j < OT; ++j) {
            Ph[j] = Op::cols(mt, m.m + kParts * Lds::MS, Lds::M1, a, a, j);
            if constexpr (kSplit) Pl[j] = Op::cols(mt, m.m + (kParts + 1) * Lds::MS, Lds::M1, a, a, j);
            later[j] = f32x4{0, 0, 0, 0};
            rd[j] = factors(kRead, j) * size.ratio;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) kd[t] = f32x4{0, 0, 0, 0};
        st[0] = two<E>(S[0], S[1]);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (s + 1 < KS) {
                read(k[(s + 1) & 1], s + 1);
            } else {
#pragma unroll
                for (int j = 0; j < OT; ++j) {
                    e[j] = factors(kWrite, j);
                    Th[j] = Op::cols(mt, m.m, Lds::M1, a, a, j);
                    if constexpr (kSplit) Tl[j] = Op::cols(mt, m.m + Lds::MS, Lds::M1, a, a, j);
                }
            }
            fence();
            if (s + 1 < KS) st[(s + 1) & 1] = two<E>(S[2 * s + 2], S[2 * s + 3]);
            if constexpr (kSplit) {
#pragma unroll
                for (int t = NT - 1; t >= 0; --t) kd[t] = M::mma(k[s & 1][t], st[s & 1].lo, kd[t]);
            }
#pragma unroll
            for (int t = NT - 1; t >= 0; --t) kd[t] = M::mma(k[s & 1][t], st[s & 1].hi, kd[t]);
            if (s == 0) {
                if constexpr (kSplit) {
#pragma unroll
                    for (int j = 0; j < OT; ++j) later[j] = Op::mma(Pl[j], yo, later[j]);
                }
#pragma unroll
                for (int j = 0; j < OT; ++j) later[j] = Op::mma(Ph[j], yo, later[j]);
                // what dY adds to dS: e^gamma dY of its own tokens
#pragma unroll
                for (int j = 0; j < OT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) rd[j][r] *= Op::at(yo, j, r);
            }
            interleave<2 * NT, 5>();
            fence();
        }
#pragma unroll
        for (int j = 0; j < OT; ++j) ex.put(j, kd[OT + j]);
        if (a == 0) {  // outputs of the second half
#pragma unroll
            for (int j = 0; j < OT; ++j) {
                Ph[j] = Op::cols(mt, m.m + kParts * Lds::MS, Lds::M1, 0, 1, j);
                later[j] = Op::mma(Ph[j], yx, later[j]);
                if constexpr (kSplit) {
                    Pl[j] = Op::cols(mt, m.m + (kParts + 1) * Lds::MS, Lds::M1, 0, 1, j);
                    later[j] = Op::mma(Pl[j], yx, later[j]);
                }
            }
        }
        const auto qq = Op::two(rd);
        lds_meet();  // 1: both halves' shares
        f32x4 x[OT], dN[OT], Z[OT];
#pragma unroll
        for (int j = 0; j < OT; ++j) ex.get(j, x[j]);
#pragma unroll
        for (int j = 0; j < OT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) dN[j][r] = fmaf(kd[j][r] + x[j][r], e[j][r], scale * later[j][r]);
        // Z = dN + (T - I)^T dN: the second half's tokens reach the first's
        const auto dn = Op::two(dN);
        if (a) {
            ex.put(4, dn.hi);
            if constexpr (kSplit) ex.put(5, dn.lo);
        }
#pragma unroll
        for (int j = 0; j < OT; ++j) Z[j] = dN[j];
        if constexpr (kSplit) {
#pragma unroll
            for (int j = 0; j < OT; ++j) {
                if (small_parts(DK)) Z[j] = Op::mma(Tl[j], dn.lo, Z[j]);
                Z[j] = Op::mma(Tl[j], dn.hi, Z[j]);
            }
#pragma unroll
            for (int j = 0; j < OT; ++j) Z[j] = Op::mma(Th[j], dn.lo, Z[j]);
        }
#pragma unroll
        for (int j = 0; j < OT; ++j) Z[j] = Op::mma(Th[j], dn.hi, Z[j]);
#pragma unroll
        for (int j = 0; j < OT; ++j) {
            be[j] = factors(kBeta, j);
            bs[j] = factors(kBetaStart, j);
            if (a) continue;
            Xh[j] = Op::cols(mt, m.m, Lds::M1, 0, 1, j);
            if constexpr (kSplit) Xl[j] = Op::cols(mt, m.m + Lds::MS, Lds::M1, 0, 1, j);
        }
        op kc[2][2], qc[2][2];
        const auto next = [&](int at, int half, int t) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                qc[at][y] = Op::tokens(kt, m.q, half, t + y);
                kc[at][y] = Op::tokens(kt, m.k, half, t + y);
            }
        };
        next(0, a, 0);
        const float fade = m.v[kStart * C + C - 1];
        lds_meet();  // 2: the second half's dN
        if (a == 0) {
            auto xx = dn;
            ex.get(4, xx.hi);
            if constexpr (kSplit) {
                ex.get(5, xx.lo);
#pragma unroll
                for (int j = 0; j < OT; ++j) {
                    if (small_parts(DK)) Z[j] = Op::mma(Xl[j], xx.lo, Z[j]);
                    Z[j] = Op::mma(Xl[j], xx.hi, Z[j]);
                }
#pragma unroll
                for (int j = 0; j < OT; ++j) Z[j] = Op::mma(Xh[j], xx.lo, Z[j]);
            }
#pragma unroll
            for (int j = 0; j < OT; ++j) Z[j] = Op::mma(Xh[j], xx.hi, Z[j]);
        }
        f32x4 w[OT];
#pragma unroll
        for (int j = 0; j < OT; ++j) w[j] = -(bs[j] * Z[j]);
        const auto aa = Op::two(w);
        ex.put(0, aa.hi);
        ex.put(1, qq.hi);
        if constexpr (kSplit) {
            ex.put(2, aa.lo);
            ex.put(3, qq.lo);
        }
        fence();
        keep_state<KT>(S, p.dstates, chunk, n, a * (DK / 2), p);
        store_tokens<C>(Z, p.z, chunk, n, a, p);
        // the state's gradient, by the half's own tokens, then by the others; two tiles in turn, as a product waits for
        // the one before it on its tile
        const auto add = [&](int half, const auto& ka, const auto& qy, bool more) {
#pragma unroll
            for (int t = 0; t < KT; t += 2) {
                const int at = t / 2 & 1;
                if (t + 2 < KT) next(at ^ 1, half, t + 2);
                else if (more) next(at ^ 1, 1 - half, 0);
                fence();
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    if (more) S[t + y] *= fade;
                if constexpr (kSplit) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) S[t + y] = Op::mma(qc[at][y], qy.lo, S[t + y]);
#pragma unroll
                    for (int y = 0; y < 2; ++y) S[t + y] = Op::mma(kc[at][y], ka.lo, S[t + y]);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) S[t + y] = Op::mma(qc[at][y], qy.hi, S[t + y]);
#pragma unroll
                for (int y = 0; y < 2; ++y) S[t + y] = Op::mma(kc[at][y], ka.hi, S[t + y]);
            }
        };
        add(a, aa, qq, true);
        if constexpr (KT / 2 % 2 == 1) {  // the other half's first tiles are where the last ones were not
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                kc[0][y] = kc[1][y];
                qc[0][y] = qc[1][y];
            }
        }
        lds_meet();  // 3: what the other half's tokens add
        auto xa = aa, xq = qq;
        ex.get(0, xa.hi);
        ex.get(1, xq.hi);
        if constexpr (kSplit) {
            ex.get(2, xa.lo);
            ex.get(3, xq.lo);
        }
        add(1 - a, xa, xq, false);
#pragma unroll
        for (int j = 0; j < OT; ++j) put_column<E, Lds::YP>(m.y + oy, j, size.down * (be[j] * Z[j]));
    });
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] *= size.down;
    if (p.dh0) store_state<KT>(S, p.dh0, int64_t(b) * p.H + h, n, a * (DK / 2), p);
}

template <typename E, int DK, int TILES>
int launch(const DeltaParams& p, hipStream_t stream) {
    typedef WalkLds<E, DK, ChunkMats<E>::kAll> Lds;
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_bwd_kernel<E, DK, TILES>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, Lds::kBytes) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + walk_cols(TILES) - 1) / walk_cols(TILES)));
    delta_bwd_kernel<E, DK, TILES><<<wgs, walk_threads(TILES), Lds::kBytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_bwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        return cls::by_tiles(p, [&](auto tiles) {
            return cls::launch<decltype(e), decltype(dk)::value, decltype(tiles)::value>(p, stream);
        });
    });
}
