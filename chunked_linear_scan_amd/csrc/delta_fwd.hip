// Gated delta rule over whole sequences: the walk over the chunks.  A wave has 16
// (or 32) columns of the state S [dk, dv] in its registers and takes them through all
// chunks of a sequence; columns do not meet, so waves only share what the
// workgroup stages in LDS for them: the chunk's K, Q, T - I, P and factors.  Per chunk
//     R = beta (V - e^gamma K S),  N = R + (T - I) R,  Y = scale (e^gamma Q S + P N),
//     S' = e^gamma_C S + K^T (e^(gamma_C - gamma) N)
// where K S, T R and K^T N reach the state and take computed operands in two
// parts, and Q S and P N only reach y and take them in one.
#include <hip/hip_runtime.h>

#include "delta.hpp"
#include "device_once.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

// COLS tiles of 16 columns to a wave, WAVES waves to a workgroup.
template <typename E, int DK, int COLS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, DK == 256 ? 1 : 2) void delta_fwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef ChunkMats<E> CM;
    typedef LdsTile<E, DK> KTile;
    typedef LdsTile<E, M::kChunk> MTile;
    typedef typename M::frag frag;
    constexpr int C = M::kChunk, NT = C / 16, KT = DK / 16, THREADS = 64 * WAVES, WG = 16 * COLS * WAVES;
    constexpr int NM = CM::kParts + 1, MS = C * MTile::kPitch;
    constexpr uint32_t SZ = sizeof(raw);
    extern __shared__ __attribute__((aligned(16))) char lds[];
    raw* sK = reinterpret_cast<raw*>(lds);
    raw* sQ = sK + C * KTile::kPitch;
    raw* sT = sQ + C * KTile::kPitch;  // T - I (its parts), P
    raw* sP = sT + CM::kParts * MS;
    float* sV = reinterpret_cast<float*>(sT + NM * MS);

    const int nblk = (p.dv + WG - 1) / WG;
    const int blk = blockIdx.x % nblk, h = blockIdx.x / nblk % p.H, b = blockIdx.x / nblk / p.H;
    const int end = seq_end(p.seqlens, b, p.L), kh = h / (p.H / p.Hk);
    const int tid = threadIdx.x, l16 = lane16(), g4 = group4();
    const int n0 = blk * WG + (tid >> 6) * 16 * COLS + l16;  // the first of a lane's columns, the others 16 apart
    const bool wave_on = n0 - l16 < p.dv;

    const raw* K = static_cast<const raw*>(p.k) + b * p.sk.batch + kh * p.sk.head;
    const raw* Q = static_cast<const raw*>(p.q) + b * p.sq.batch + kh * p.sq.head;
    const raw* V = static_cast<const raw*>(p.v) + b * p.sv.batch + h * p.sv.head;
    const int64_t row = int64_t(p.H) * p.dv;  // of a token of y
    const int64_t out = int64_t(b) * p.L * row + int64_t(h) * p.dv;
    raw* Y = static_cast<raw*>(p.y) + out;

    f32x4 S[COLS][KT];
    bool on[COLS];
#pragma unroll
    for (int u = 0; u < COLS; ++u) {
        const int n = n0 + 16 * u;
        on[u] = n < p.dv;
        const float* from = p.h0 + ((int64_t(b) * p.H + h) * p.dv + n) * p.dk;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = 16 * t + 4 * g4 + r;
                S[u][t][r] = p.h0 && on[u] && d < p.dk ? from[d] : 0.0f;
            }
    }

    // offsets of a lane in a chunk: of its vectors of K, Q and the matrices, of its elements of V and Y
    typedef TileRegs<E, C, DK, THREADS> KRegs;
    typedef TileRegs<E, C, C, THREADS> MRegs;
    const KTile kt;
    const MTile mt;
    const uint32_t ok = KRegs::offset(p.sk.token, p.dk), oq = KRegs::offset(p.sq.token, p.dk), om = MRegs::offset(C, C);
    const uint32_t vrow = uint32_t(p.sv.token) * SZ, yrow = uint32_t(row) * SZ;
    uint32_t ov[COLS], oy[COLS];
#pragma unroll
    for (int u = 0; u < COLS; ++u) {
        ov[u] = on[u] ? 4 * g4 * vrow + (n0 + 16 * u) * SZ : kOutside;
        oy[u] = on[u] ? 4 * g4 * yrow + (n0 + 16 * u) * SZ : kOutside;
    }
    KRegs rk, rq;
    MRegs rm[NM];
    float rv = 0.0f;
    raw v[COLS][NT][4];
    const int chunks = (end + C - 1) / C;
    const auto fetch = [&](int c) {
        const int t0 = c * C, left = end - t0;
        rk.load(buffer(K + t0 * p.sk.token, left * p.sk.token * SZ), ok, p.sk.token);
        rq.load(buffer(Q + t0 * p.sq.token, left * p.sq.token * SZ), oq, p.sq.token);
        const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
        const raw* mats = static_cast<const raw*>(p.mats) + chunk * CM::kAll * CM::kSize;
#pragma unroll
        for (int m = 0; m < NM; ++m) rm[m].load(buffer(mats + m * CM::kSize), om, C);
        if (tid < 3 * C) rv = p.vecs[chunk * 3 * C + tid];
        const Buffer bv = buffer(V + t0 * p.sv.token, left * p.sv.token * SZ);
#pragma unroll
        for (int u = 0; u < COLS; ++u) {
            const uint32_t at = here(ov[u]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[u][t][r] = load_one<E>(bv, at + (16 * t + r) * vrow);
        }
    };
    if (chunks > 0) fetch(0);
    for (int c = 0; c < chunks; ++c) {
        const int t0 = c * C;
        lds_meet();  // the chunk before is read
        rk.template store<KTile>(sK);
        rq.template store<KTile>(sQ);
#pragma unroll
        for (int m = 0; m < NM; ++m) rm[m].template store<MTile>(sT + m * MS);
        if (tid < 3 * C) sV[tid] = rv;
        f32x4 R[COLS][NT];
#pragma unroll
        for (int u = 0; u < COLS; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) R[u][t][r] = E::get(v[u][t][r]);
        lds_meet();
        if (c + 1 < chunks) fetch(c + 1);
        if (!wave_on) continue;

        if (p.states) {
            const Buffer bs = buffer(p.states + ((int64_t(b) * p.nchunk + c) * p.H + h) * p.dk * p.dv,
                                     int64_t(p.dk) * p.dv * 4);
#pragma unroll
            for (int u = 0; u < COLS; ++u) {
                const uint32_t at = here(on[u] ? (4 * g4 * p.dv + n0 + 16 * u) * 4 : kOutside);
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) store_one<ElemF32>(bs, at + (16 * t + r) * p.dv * 4, S[u][t][r]);
            }
        }
        f32x4 ks[COLS][NT], O[COLS][NT];
#pragma unroll
        for (int u = 0; u < COLS; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t) ks[u][t] = O[u][t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) {
            Two<E> st[COLS];
#pragma unroll
            for (int u = 0; u < COLS; ++u) st[u] = two<E>(S[u][2 * s], S[u][2 * s + 1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const frag k = kt.rows(sK, t, s), q = kt.rows(sQ, t, s);
#pragma unroll
                for (int u = 0; u < COLS; ++u) {
                    ks[u][t] = mma2<E>(k, st[u], ks[u][t]);
                    O[u][t] = M::mma(q, st[u].hi, O[u][t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 e = *reinterpret_cast<const f32x4*>(sV + 16 * t + 4 * g4);
            const f32x4 be = *reinterpret_cast<const f32x4*>(sV + 2 * C + 16 * t + 4 * g4);
#pragma unroll
            for (int u = 0; u < COLS; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    R[u][t][r] = be[r] * fmaf(-e[r], ks[u][t][r], R[u][t][r]);
                    O[u][t][r] *= e[r];
                }
        }
        // N = R + (T - I) R: tokens up to 32 (t / 2 + 1) reach tile t
        f32x4 N[COLS][NT];
        {
            Two<E> rr[COLS][NT / 2];
#pragma unroll
            for (int u = 0; u < COLS; ++u)
#pragma unroll
                for (int s = 0; s < NT / 2; ++s) rr[u][s] = two<E>(R[u][2 * s], R[u][2 * s + 1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int u = 0; u < COLS; ++u) N[u][t] = R[u][t];
#pragma unroll
                for (int s = 0; s <= t / 2; ++s) {
                    Two<E> T;
                    T.hi = mt.rows(sT, t, s);
                    if constexpr (M::kSplit) T.lo = mt.rows(sT + MS, t, s);
#pragma unroll
                    for (int u = 0; u < COLS; ++u) N[u][t] = mma3<E>(T, rr[u][s], N[u][t]);
                }
            }
        }
        const int64_t at = out + t0 * row;
        const Buffer by = buffer(Y + t0 * row, int64_t(p.L - t0) * row * SZ);
        {
            frag nf[COLS][NT / 2];
#pragma unroll
            for (int u = 0; u < COLS; ++u)
#pragma unroll
                for (int s = 0; s < NT / 2; ++s) nf[u][s] = M::cvt(N[u][2 * s], N[u][2 * s + 1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int s = 0; s <= t / 2; ++s) {
                    const frag P = mt.rows(sP, t, s);
#pragma unroll
                    for (int u = 0; u < COLS; ++u) O[u][t] = M::mma(P, nf[u][s], O[u][t]);
                }
            }
        }
        if (t0 + C > end)  // padding within the chunk
#pragma unroll
            for (int u = 0; u < COLS; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (t0 + 16 * t + 4 * g4 + r >= end) O[u][t][r] = 0.0f;
#pragma unroll
        for (int u = 0; u < COLS; ++u) {
            const uint32_t to = here(oy[u]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) store_one<E>(by, to + (16 * t + r) * yrow, p.scale * O[u][t][r]);
        }
        if (p.fixes) {
            const Buffer bf = buffer(p.fixes + at, int64_t(p.L - t0) * row * 4);
#pragma unroll
            for (int u = 0; u < COLS; ++u) {
                const uint32_t of = here(on[u] ? (4 * g4 * uint32_t(row) + n0 + 16 * u) * 4 : kOutside);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) store_one<ElemF32>(bf, of + (16 * t + r) * uint32_t(row) * 4, N[u][t][r]);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 e = *reinterpret_cast<const f32x4*>(sV + C + 16 * t + 4 * g4);
#pragma unroll
            for (int u = 0; u < COLS; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) N[u][t][r] *= e[r];
        }
        const float fade = sV[C - 1];
        Two<E> nn[COLS][NT / 2];
#pragma unroll
        for (int u = 0; u < COLS; ++u)
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) nn[u][s] = two<E>(N[u][2 * s], N[u][2 * s + 1]);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
#pragma unroll
            for (int u = 0; u < COLS; ++u) S[u][t] *= fade;
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) {
                const frag k = kt.cols(sK, s, t);
#pragma unroll
                for (int u = 0; u < COLS; ++u) S[u][t] = mma2<E>(k, nn[u][s], S[u][t]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < COLS; ++u) {
        if (!on[u]) continue;
        for (int tok = chunks * C + g4; tok < p.L; tok += 4) Y[tok * row + n0 + 16 * u] = raw(0);
        if (!p.h_last) continue;
        float* to = p.h_last + ((int64_t(b) * p.H + h) * p.dv + n0 + 16 * u) * p.dk;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = 16 * t + 4 * g4 + r;
                if (d < p.dk) to[d] = S[u][t][r];
            }
    }
}

template <typename E, int DK, int COLS, int WAVES>
int launch(const DeltaParams& p, hipStream_t stream) {
    typedef Mat<E> M;
    typedef ChunkMats<E> CM;
    constexpr size_t bytes = (2 * M::kChunk * LdsTile<E, DK>::kPitch + (CM::kParts + 1) * M::kChunk * LdsTile<E, M::kChunk>::kPitch) *
                                 sizeof(typename M::raw) + 3 * M::kChunk * sizeof(float);
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_fwd_kernel<E, DK, COLS, WAVES>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    constexpr int WG = 16 * COLS * WAVES;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + WG - 1) / WG));
    delta_fwd_kernel<E, DK, COLS, WAVES><<<wgs, 64 * WAVES, bytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_fwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        return cls::launch<decltype(e), decltype(dk)::value, 1, 4>(p, stream);
    });
}
