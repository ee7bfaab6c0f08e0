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

// COLS tiles of 16 columns to a wave, WAVES waves to a workgroup.
template <typename E, int DK, int COLS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, DK == 256 ? 1 : 2) void delta_bwd_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef ChunkMats<E> CM;
    typedef LdsTile<E, DK> KTile;
    typedef LdsTile<E, M::kChunk> MTile;
    typedef typename M::frag frag;
    constexpr int C = M::kChunk, NT = C / 16, KT = DK / 16, THREADS = 64 * WAVES, WG = 16 * COLS * WAVES;
    constexpr int NM = CM::kAll, MS = C * MTile::kPitch;
    constexpr uint32_t SZ = sizeof(raw);
    extern __shared__ __attribute__((aligned(16))) char lds[];
    raw* sK = reinterpret_cast<raw*>(lds);
    raw* sQ = sK + C * KTile::kPitch;
    raw* sT = sQ + C * KTile::kPitch;  // T - I, P (their parts)
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
    const raw* dY = static_cast<const raw*>(p.dy) + b * p.sdy.batch + h * p.sdy.head;
    const int64_t row = int64_t(p.H) * p.dv;  // of a token of dv
    const int64_t out = int64_t(b) * p.L * row + int64_t(h) * p.dv;
    raw* dV = static_cast<raw*>(p.dv_) + out;

    f32x4 S[COLS][KT];
    bool on[COLS];
#pragma unroll
    for (int u = 0; u < COLS; ++u) {
        const int n = n0 + 16 * u;
        on[u] = n < p.dv;
        const float* from = p.dh_last + ((int64_t(b) * p.H + h) * p.dv + n) * p.dk;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = 16 * t + 4 * g4 + r;
                S[u][t][r] = p.dh_last && on[u] && d < p.dk ? from[d] : 0.0f;
            }
    }

    typedef TileRegs<E, C, DK, THREADS> KRegs;
    typedef TileRegs<E, C, C, THREADS> MRegs;
    const KTile kt;
    const MTile mt;
    const uint32_t ok = KRegs::offset(p.sk.token, p.dk), oq = KRegs::offset(p.sq.token, p.dk), om = MRegs::offset(C, C);
    const uint32_t vrow = uint32_t(p.sdy.token) * SZ, yrow = uint32_t(row) * SZ;
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
        const Buffer bv = buffer(dY + t0 * p.sdy.token, left * p.sdy.token * SZ);
#pragma unroll
        for (int u = 0; u < COLS; ++u) {
            const uint32_t at = here(ov[u]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[u][t][r] = load_one<E>(bv, at + (16 * t + r) * vrow);
        }
    };
    if (chunks > 0) fetch(chunks - 1);
    for (int c = chunks - 1; c >= 0; --c) {
        const int t0 = c * C;
        lds_meet();  // the chunk before is read
        rk.template store<KTile>(sK);
        rq.template store<KTile>(sQ);
#pragma unroll
        for (int m = 0; m < NM; ++m) rm[m].template store<MTile>(sT + m * MS);
        if (tid < 3 * C) sV[tid] = rv;
        f32x4 dy[COLS][NT];
#pragma unroll
        for (int u = 0; u < COLS; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) dy[u][t][r] = E::get(v[u][t][r]);
        lds_meet();
        if (c > 0) fetch(c - 1);
        if (!wave_on) continue;

        const Buffer bs = buffer(p.dstates + ((int64_t(b) * p.nchunk + c) * p.H + h) * p.dk * p.dv, int64_t(p.dk) * p.dv * 4);
#pragma unroll
        for (int u = 0; u < COLS; ++u) {
            const uint32_t at = here(on[u] ? (4 * g4 * p.dv + n0 + 16 * u) * 4 : kOutside);
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) store_one<ElemF32>(bs, at + (16 * t + r) * p.dv * 4, S[u][t][r]);
        }
        f32x4 dN[COLS][NT];
#pragma unroll
        for (int u = 0; u < COLS; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t) dN[u][t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) {
            Two<E> st[COLS];
#pragma unroll
            for (int u = 0; u < COLS; ++u) st[u] = two<E>(S[u][2 * s], S[u][2 * s + 1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const frag k = kt.rows(sK, t, s);
#pragma unroll
                for (int u = 0; u < COLS; ++u) dN[u][t] = mma2<E>(k, st[u], dN[u][t]);
            }
        }
        {
            frag df[COLS][NT / 2];
#pragma unroll
            for (int u = 0; u < COLS; ++u)
#pragma unroll
                for (int s = 0; s < NT / 2; ++s) df[u][s] = M::cvt(dy[u][2 * s], dy[u][2 * s + 1]);  // exact
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 later[COLS];
#pragma unroll
                for (int u = 0; u < COLS; ++u) later[u] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = t / 2; s < NT / 2; ++s) {  // later tokens' outputs
                    Two<E> P;
                    P.hi = mt.cols(sP, s, t);
                    if constexpr (M::kSplit) P.lo = mt.cols(sP + MS, s, t);
#pragma unroll
                    for (int u = 0; u < COLS; ++u) later[u] = mma2<E>(P, df[u][s], later[u]);
                }
                const f32x4 e = *reinterpret_cast<const f32x4*>(sV + C + 16 * t + 4 * g4);
#pragma unroll
                for (int u = 0; u < COLS; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) dN[u][t][r] = fmaf(dN[u][t][r], e[r], p.scale * later[u][r]);
            }
        }
        // Z = dN + (T - I)^T dN; then dR = beta Z, and what it and dY add to dS
        const Buffer by = buffer(dV + t0 * row, int64_t(p.L - t0) * row * SZ);
        const Buffer bz = buffer(p.z + out + t0 * row, int64_t(p.L - t0) * row * 4);
        {
            Two<E> dn[COLS][NT / 2];
#pragma unroll
            for (int u = 0; u < COLS; ++u)
#pragma unroll
                for (int s = 0; s < NT / 2; ++s) dn[u][s] = two<E>(dN[u][2 * s], dN[u][2 * s + 1]);
            uint32_t oz[COLS], to[COLS];
#pragma unroll
            for (int u = 0; u < COLS; ++u) {
                oz[u] = here(on[u] ? (4 * g4 * uint32_t(row) + n0 + 16 * u) * 4 : kOutside);
                to[u] = here(oy[u]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 Z[COLS];
#pragma unroll
                for (int u = 0; u < COLS; ++u) Z[u] = dN[u][t];
#pragma unroll
                for (int s = t / 2; s < NT / 2; ++s) {
                    Two<E> T;
                    T.hi = mt.cols(sT, s, t);
                    if constexpr (M::kSplit) T.lo = mt.cols(sT + MS, s, t);
#pragma unroll
                    for (int u = 0; u < COLS; ++u) Z[u] = mma3<E>(T, dn[u][s], Z[u]);
                }
                const f32x4 e = *reinterpret_cast<const f32x4*>(sV + 16 * t + 4 * g4);
                const f32x4 be = *reinterpret_cast<const f32x4*>(sV + 2 * C + 16 * t + 4 * g4);
#pragma unroll
                for (int u = 0; u < COLS; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float z = Z[u][r], dr = t0 + 16 * t + 4 * g4 + r < end ? be[r] * z : 0.0f;
                        dN[u][t][r] = -e[r] * dr;
                        dy[u][t][r] *= p.scale * e[r];
                        store_one<E>(by, to[u] + (16 * t + r) * yrow, dr);
                        store_one<ElemF32>(bz, oz[u] + (16 * t + r) * uint32_t(row) * 4, z);
                    }
            }
        }
        const float fade = sV[C - 1];
        Two<E> a[COLS][NT / 2], q[COLS][NT / 2];
#pragma unroll
        for (int u = 0; u < COLS; ++u)
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) {
                a[u][s] = two<E>(dN[u][2 * s], dN[u][2 * s + 1]);
                q[u][s] = two<E>(dy[u][2 * s], dy[u][2 * s + 1]);
            }
#pragma unroll
        for (int t = 0; t < KT; ++t) {
#pragma unroll
            for (int u = 0; u < COLS; ++u) S[u][t] *= fade;
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) {
                const frag qc = kt.cols(sQ, s, t), kc = kt.cols(sK, s, t);
#pragma unroll
                for (int u = 0; u < COLS; ++u) {
                    S[u][t] = mma2<E>(qc, q[u][s], S[u][t]);
                    S[u][t] = mma2<E>(kc, a[u][s], S[u][t]);
                }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < COLS; ++u) {
        if (!on[u]) continue;
        for (int tok = chunks * C + g4; tok < p.L; tok += 4) dV[tok * row + n0 + 16 * u] = raw(0);
        if (!p.dh0) continue;
        float* to = p.dh0 + ((int64_t(b) * p.H + h) * p.dv + n0 + 16 * u) * p.dk;
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
    constexpr size_t bytes = (2 * M::kChunk * LdsTile<E, DK>::kPitch + CM::kAll * M::kChunk * LdsTile<E, M::kChunk>::kPitch) *
                                 sizeof(typename M::raw) + 3 * M::kChunk * sizeof(float);
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_bwd_kernel<E, DK, COLS, WAVES>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    constexpr int WG = 16 * COLS * WAVES;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.H * ((p.dv + WG - 1) / WG));
    delta_bwd_kernel<E, DK, COLS, WAVES><<<wgs, 64 * WAVES, bytes, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_bwd_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        return cls::launch<decltype(e), decltype(dk)::value, 1, 4>(p, stream);
    });
}
