// Gradients of the gated delta rule, the part that takes all chunks at once: dq,
// dk, dbeta and dg from the state S before each chunk and the gradient dS of the
// one behind it, the corrections N and Z = (I + A)^-T dN.  With dP = dY N^T (j <= i),
// M = Z N^T (j < i), pP_ij = scale D_ij dP_ij and pB_ij = -beta_i D_ij M_ij:
//     dQ = scale e^gamma dY S^T + pP K
//     dK = -beta e^gamma Z S^T + pB K  +  e^(gamma_C - gamma) N dS^T + pB^T K + pP^T Q
//     dbeta_i = Z_i.V_i - e^gamma_i (S^T k_i).Z_i - sum_j D_ij k_i.k_j M_ij
// (no division by beta, which may be zero).  g_t stands in every product between a token
// before t and one from t on, so with F_ij = pP_ij q_i.k_j + pB_ij k_i.k_j
//     dg_t = sum_{i >= t > j} F_ij + sum_{i >= t} read_i + sum_{j < t} write_j + e^gamma_C <S, dS>
// where read and write are the state's parts of dQ.q + dK.k and of dK.k.  (Differences
// q.dQ - k.dK of whole gradients would be shorter, but cancel and carry the operands'
// rounding; sums of F are of the same numbers by rows and by columns.)
// A wave has 16 tokens; products run transposed (tokens in the columns), so dQ and dK
// leave as four adjacent values of a token, and the decays are factors of a lane.
// What reaches dg and dbeta, fp32 outputs, takes computed operands in two parts;
// pP and pB only reach dQ and dK and go in as one.
#include <hip/hip_runtime.h>

#include "delta.hpp"
#include "device_once.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// 32 rows (of dv) of a matrix [dv, cols] of fp32 values, padded to COLS columns, held by the workgroup's threads between
// memory and LDS, where they are an operand's parts.
template <typename E, int COLS, int THREADS>
struct Tile32 {
    typedef LdsTile<E, COLS> Lds;
    static constexpr int PER_ROW = COLS / 4, STEP = THREADS / PER_ROW, N = 32 / STEP;
    static_assert(THREADS % PER_ROW == 0 && 32 % STEP == 0, "");
    static constexpr int kPart = 32 * Lds::kPitch;
    f32x4 r[N];
    __device__ __forceinline__ void load(const float* m, int64_t dv, int row0, int cols) {
        const Buffer b = buffer(m, dv * cols * 4);
        const int col = threadIdx.x % PER_ROW * 4;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int row = row0 + int(threadIdx.x) / PER_ROW + n * STEP;
            const uint32_t at = uint32_t(row * cols + col) * 4;
            if (cols % 4 == 0) {
                r[n] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, int(col < cols ? at : kOutside), 0, 0));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) r[n][e] = as_float(load_one<ElemF32>(b, col + e < cols ? at + 4 * e : kOutside));
            }
        }
    }
    __device__ __forceinline__ void store(typename E::raw* to) const {
        const int col = threadIdx.x % PER_ROW * 4;
#pragma unroll
        for (int n = 0; n < N; ++n) put4<E>(to + Lds::quad(int(threadIdx.x) / PER_ROW + n * STEP, col), kPart, r[n]);
    }
    // times a factor of each column
    __device__ __forceinline__ void scale(const f32x4& f) {
#pragma unroll
        for (int n = 0; n < N; ++n) r[n] *= f;
    }
    __device__ __forceinline__ float dot(const Tile32& o) const {
        float v = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) v = fmaf(r[n][e], o.r[n][e], v);
        return v;
    }
};

// 16 columns of such a tile as an operand.
template <typename E, typename T>
__device__ __forceinline__ Two<E> two_cols(const T& tile, const typename E::raw* m, int t) {
    Two<E> x;
    x.hi = tile.cols(m, 0, t);
    if constexpr (Mat<E>::kSplit) x.lo = tile.cols(m + 32 * T::kPitch, 0, t);
    return x;
}

template <typename E, int DK>
struct GradSize {
    typedef Mat<E> M;
    static constexpr int C = M::kChunk, KP = LdsTile<E, DK>::kPitch, MP = LdsTile<E, C>::kPitch;
    static constexpr int kParts = ChunkMats<E>::kParts;
    static constexpr int kTiles = kParts * 32 * (KP + 2 * MP);  // tiles of S or dS, of N and of Z
    static constexpr int kPairs = 2 * C * MP;                   // pB and pP, in the same place
    static constexpr int kUnion = kTiles > kPairs ? kTiles : kPairs;
    static constexpr size_t bytes = (2 * C * KP + kUnion) * sizeof(typename M::raw) + (Decays<C>::kFloats + (2 + C / 16) * C + C / 16) * sizeof(float);
};

template <typename E, int DK>
__global__ __launch_bounds__(Mat<E>::kChunk * 4, DK <= 128 ? 2 : 1) void delta_grad_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef GradSize<E, DK> G;
    constexpr int C = G::C, NT = C / 16, KT = DK / 16, THREADS = 64 * NT, KP = G::KP, MP = G::MP;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    raw* sK = reinterpret_cast<raw*>(lds);
    raw* sQ = sK + C * KP;
    raw* sS = sQ + C * KP;
    raw* sN = sS + G::kParts * 32 * KP;
    raw* sZ = sN + G::kParts * 32 * MP;
    raw* sB = sS;  // once the tiles are done with
    raw* sP = sB + C * MP;
    float* sG = reinterpret_cast<float*>(sS + G::kUnion);
    float* sRow = sG + Decays<C>::kFloats;  // read_i + sum_j F_ij
    float* sWrite = sRow + C;   // write_j
    float* sCol = sWrite + C;   // [NT][C]: sums of F over a wave's tokens
    float* sDot = sCol + NT * C;

    const int rep = p.H / p.Hk;
    const UnitPart u = unit_part(p.batch * p.nchunk * p.Hk, rep);
    const int kh = u.unit % p.Hk, h = kh * rep + u.part, c = u.unit / p.Hk % p.nchunk, b = u.unit / p.Hk / p.nchunk;
    const int end = seq_end(p.seqlens, b, p.L), t0 = c * C;
    const int tid = threadIdx.x, w = tid >> 6, l16 = lane16(), g4 = group4();
    const int i = 16 * w + l16, tok = t0 + i;  // this lane's token
    const bool in = tok < end;
    // rows of the outputs: of a token's head, or its part of a key head's sum
    raw* dQ = static_cast<raw*>(p.dq) + ((int64_t(b) * p.L + tok) * p.Hk + kh) * p.dk;
    raw* dK = static_cast<raw*>(p.dk_) + ((int64_t(b) * p.L + tok) * p.Hk + kh) * p.dk;
    float* partQ = p.part_q + ((int64_t(b) * p.L + tok) * p.H + h) * p.dk;
    float* partK = p.part_k + ((int64_t(b) * p.L + tok) * p.H + h) * p.dk;
    const int64_t gat = (int64_t(b) * p.L + tok) * p.H + h;

    const auto put_row = [&](raw* one, float* part, int d, const f32x4& v) {
        if (tok >= p.L) return;
        if (rep > 1) {
            if (p.dk % 4 == 0) {
                if (d < p.dk) *reinterpret_cast<f32x4*>(part + d) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (d + e < p.dk) part[d + e] = v[e];
            }
        } else if (p.dk % 4 == 0 && p.vec_dqk) {
            if (d < p.dk) put4<E>(one + d, 0, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < p.dk) one[d + e] = E::put(v[e]);
        }
    };
    if (t0 >= end) {  // padding
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            put_row(dQ, partQ, 16 * t + 4 * g4, f32x4{0, 0, 0, 0});
            put_row(dK, partK, 16 * t + 4 * g4, f32x4{0, 0, 0, 0});
        }
        if (g4 == 0 && tok < p.L) p.dg[gat] = p.dbeta[gat] = 0.0f;
        return;
    }

    const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
    const float* vecs = p.vecs + chunk * kVecs * C;
    const float start = vecs[kStart * C + i], beta = vecs[kBeta * C + i], fade = vecs[kStart * C + C - 1];
    const float* S0 = p.states + chunk * p.dk * p.dv;
    const float* dS = p.dstates + chunk * p.dk * p.dv;
    const float* N = p.fixes + chunk * p.dv * C;
    const float* Z = p.z + chunk * p.dv * C;
    const raw* Yi = static_cast<const raw*>(p.dy) + b * p.sdy.batch + h * p.sdy.head + tok * p.sdy.token;
    const raw* Vi = static_cast<const raw*>(p.v) + b * p.sv.batch + h * p.sv.head + tok * p.sv.token;
    const int left = end - t0 < C ? end - t0 : C;  // tokens of the chunk
    typedef LdsTile<E, DK> KTile;
    typedef LdsTile<E, C> MTile;
    const KTile kt;
    const MTile mt;
    {
        typedef TileRegs<E, C, DK, THREADS> Regs;
        Regs k, q;
        const raw* K = static_cast<const raw*>(p.k) + b * p.sk.batch + t0 * p.sk.token + kh * p.sk.head;
        const raw* Q = static_cast<const raw*>(p.q) + b * p.sq.batch + t0 * p.sq.token + kh * p.sq.head;
        k.load(buffer(K, left * p.sk.token * sizeof(raw)), Regs::offset(p.sk.token, p.dk, tid), p.sk.token);
        q.load(buffer(Q, left * p.sq.token * sizeof(raw)), Regs::offset(p.sq.token, p.dk, tid), p.sq.token);
        if (tid < C) Decays<C>::put(sG, t0 + tid < end ? p.g[b * p.g_batch + int64_t(t0 + tid) * p.g_token + h] : 0.0f);
        k.template store<KTile>(sK, tid);
        q.template store<KTile>(sQ, tid);
    }

    // with the state before the chunk: X1 = S dY^T, X2 = S Z^T; with the corrections: dP^T and M^T
    f32x4 X1[KT], X2[KT], dP[NT], Mz[NT];
#pragma unroll
    for (int t = 0; t < KT; ++t) X1[t] = X2[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < NT; ++t) dP[t] = Mz[t] = f32x4{0, 0, 0, 0};
    float zv = 0.0f;  // Z_i.V_i
    typedef Tile32<E, DK, THREADS> STile;
    typedef Tile32<E, C, THREADS> NTile;
    STile rs;
    NTile rn, rz;
    rs.load(S0, p.dv, 0, p.dk);
    rn.load(N, p.dv, 0, C);
    rz.load(Z, p.dv, 0, C);
    f32x4 y1[2], v1[2];  // of dY and V, of the columns to come
    const auto ahead = [&](int d0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int col = d0 + 16 * u + 4 * g4;
            y1[u] = in ? load4<E>(Yi, col, p.dv, true) : f32x4{0, 0, 0, 0};
            v1[u] = in ? load4<E>(Vi, col, p.dv, true) : f32x4{0, 0, 0, 0};
        }
    };
    ahead(0);
    for (int d0 = 0; d0 < p.dv; d0 += 32) {
        lds_meet();
        rs.store(sS);
        rn.store(sN);
        rz.store(sZ);
        const f32x4 y[2] = {y1[0], y1[1]}, v[2] = {v1[0], v1[1]};
        lds_meet();
        if (d0 + 32 < p.dv) {
            rs.load(S0, p.dv, d0 + 32, p.dk);
            rn.load(N, p.dv, d0 + 32, C);
            rz.load(Z, p.dv, d0 + 32, C);
            ahead(d0 + 32);
        }
        const Two<E> zf = two_cols<E>(mt, sZ, w);
        const typename M::frag yf = M::cvt(y[0], y[1]);  // exact
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float z = M::at(zf.hi, e);
            if constexpr (M::kSplit) z += M::at(zf.lo, e);
            zv = fmaf(z, v[e >> 2][e & 3], zv);
        }
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const Two<E> s = two_cols<E>(kt, sS, t);
            X1[t] = mma2<E>(s, yf, X1[t]);
            X2[t] = mma3<E>(s, zf, X2[t]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t > w) break;
            const Two<E> nj = two_cols<E>(mt, sN, t);
            dP[t] = mma2<E>(nj, yf, dP[t]);
            Mz[t] = mma3<E>(nj, zf, Mz[t]);
        }
    }
    zv = sum_groups(zv);
    const auto dot_row = [&](const raw* m, const f32x4 (&x)[KT]) {
        float v = 0.0f;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const f32x4 a = load4<E>(m, KTile::quad(i, 16 * t + 4 * g4), 1 << 30, true);
#pragma unroll
            for (int r = 0; r < 4; ++r) v = fmaf(a[r], x[t][r], v);
        }
        return sum_groups(v);
    };
    const float qx = p.scale * start * dot_row(sQ, X1), kx = start * dot_row(sK, X2);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        X1[t] *= p.scale * start;
        X2[t] *= -beta * start;
    }

    // with the gradient of the state behind it: + dS (e^(gamma_C - gamma) N)^T, and <S, dS>
    float both = 0.0f;
    {
        STile r0;
        const f32x4 after = *reinterpret_cast<const f32x4*>(vecs + kWrite * C + threadIdx.x % NTile::PER_ROW * 4);
        rs.load(dS, p.dv, 0, p.dk);
        r0.load(S0, p.dv, 0, p.dk);
        rn.load(N, p.dv, 0, C);
        for (int d0 = 0; d0 < p.dv; d0 += 32) {
            lds_meet();
            rs.store(sS);
            rn.scale(after);
            rn.store(sN);
            both += rs.dot(r0);
            lds_meet();
            if (d0 + 32 < p.dv) {
                rs.load(dS, p.dv, d0 + 32, p.dk);
                r0.load(S0, p.dv, d0 + 32, p.dk);
                rn.load(N, p.dv, d0 + 32, C);
            }
            const Two<E> nf = two_cols<E>(mt, sN, w);
#pragma unroll
            for (int t = 0; t < KT; ++t) X2[t] = mma3<E>(two_cols<E>(kt, sS, t), nf, X2[t]);
        }
    }
    const float write = dot_row(sK, X2) + beta * kx;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) both += __shfl_xor(both, d, 64);
    if ((tid & 63) == 0) sDot[w] = both;

    // pairs of tokens
    f32x4 kk[NT], qk[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) kk[t] = qk[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
        const typename M::frag ki = kt.rows(sK, w, ks), qi = kt.rows(sQ, w, ks);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t > w) break;
            const typename M::frag kj = kt.rows(sK, t, ks);
            kk[t] = M::mma(kj, ki, kk[t]);
            qk[t] = M::mma(kj, qi, qk[t]);
        }
    }
    float rows = 0.0f, db = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
        if (t > w)
            for (int r = 0; r < 4; ++r) kk[t][r] = 0.0f;
    Decays<C>::each(sG, w, [&](int t, const f32x4& d) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = 16 * t + 4 * g4 + r;
            const float m = j < i ? d[r] * Mz[t][r] : 0.0f;
            dP[t][r] = j <= i ? p.scale * d[r] * dP[t][r] : 0.0f;
            Mz[t][r] = -beta * m;
            db = fmaf(m, kk[t][r], db);
            const float f = j < i ? fmaf(dP[t][r], qk[t][r], Mz[t][r] * kk[t][r]) : 0.0f;
            rows += f;
            kk[t][r] = f;  // kk becomes F
        }
    });
    rows = sum_groups(rows);
    db = sum_groups(db);
    // sums of F over the wave's tokens
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float v = row_total(kk[t][r]);
            if (l16 == 0) sCol[w * C + 16 * t + 4 * g4 + r] = v;
        }
    if (g4 == 0) {
        sRow[i] = rows + qx - beta * kx;
        sWrite[i] = write;
        if (tok < p.L) p.dbeta[gat] = in ? zv - kx - db : 0.0f;
    }
    __syncthreads();  // the tiles are read
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        put4<E>(sB + MTile::quad(i, 16 * t + 4 * g4), 0, Mz[t]);  // zeros for the tiles behind w
        put4<E>(sP + MTile::quad(i, 16 * t + 4 * g4), 0, dP[t]);
    }
    __syncthreads();
    if (tid < 64) {  // dg of token tid, by the first wave
        float both = 0.0f, row = 0.0f, put = 0.0f;
#pragma unroll
        for (int k = 0; k < NT; ++k) both += fade * sDot[k];
        if (tid < C) {
            row = sRow[tid];
            put = sWrite[tid];
#pragma unroll
            for (int k = 0; k < NT; ++k) row -= sCol[k * C + tid];
        }
        // from tid on, and before tid: sums over 16 lanes, then over their rows
        float from = row + row_behind(row), before = row_prefix(row_move<0x111>(put));  // of those before it
        const float rows16 = row_total(row), puts16 = row_total(put);
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            const float a = __shfl(rows16, 16 * k, 64), c = __shfl(puts16, 16 * k, 64);
            from += k > tid >> 4 ? a : 0.0f;
            before += k < tid >> 4 ? c : 0.0f;
        }
        float v = both + from + before;
        if (tid < C && t0 + tid < p.L) {
            if (fexp(sG[tid]) == 0.0f) v = 0.0f;  // nothing passes: not the sums' roundings either
            p.dg[(int64_t(b) * p.L + t0 + tid) * p.H + h] = t0 + tid < end ? v : 0.0f;
        }
    }
    // the pairs' parts: as the later token (operands from the lanes), as the earlier one (from LDS)
    typename M::frag bi[NT / 2], pi[NT / 2], bj[NT / 2], pj[NT / 2];
#pragma unroll
    for (int s = 0; s < NT / 2; ++s) {
        bi[s] = M::cvt(Mz[2 * s], Mz[2 * s + 1]);
        pi[s] = M::cvt(dP[2 * s], dP[2 * s + 1]);
        bj[s] = mt.cols(sB, s, w);
        pj[s] = mt.cols(sP, s, w);
    }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) {
            const typename M::frag kc = kt.cols(sK, s, t), qc = kt.cols(sQ, s, t);
            X1[t] = M::mma(kc, pi[s], X1[t]);
            X2[t] = M::mma(kc, bi[s], X2[t]);
            X2[t] = M::mma(kc, bj[s], X2[t]);
            X2[t] = M::mma(qc, pj[s], X2[t]);
        }
        if (!in) X1[t] = X2[t] = f32x4{0, 0, 0, 0};
        put_row(dQ, partQ, 16 * t + 4 * g4, X1[t]);
        put_row(dK, partK, 16 * t + 4 * g4, X2[t]);
    }
}

// Sums over the heads of a key head.
template <typename E>
__global__ __launch_bounds__(256) void delta_heads_kernel(const float* part_q, const float* part_k, typename E::raw* dq,
                                                          typename E::raw* dk, int64_t n, int dim, int rep) {
    const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (at >= n) return;
    const int64_t from = at / dim * rep * dim + at % dim;
    float q = 0.0f, k = 0.0f;
    for (int r = 0; r < rep; ++r) {
        q += part_q[from + int64_t(r) * dim];
        k += part_k[from + int64_t(r) * dim];
    }
    dq[at] = E::put(q);
    dk[at] = E::put(k);
}

template <typename E, int DK>
int launch(const DeltaParams& p, hipStream_t stream) {
    constexpr size_t bytes = GradSize<E, DK>::bytes;
    static DeviceOnce once;
    const int st = run_once_per_device(once, [] {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&delta_grad_kernel<E, DK>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) == hipSuccess ? 0 : -7;
    });
    if (st != 0) return st;
    const unsigned wgs = unsigned(int64_t(p.batch) * p.nchunk * p.H);
    delta_grad_kernel<E, DK><<<wgs, 4 * Mat<E>::kChunk, bytes, stream>>>(p);
    if (hipGetLastError() != hipSuccess) return -7;
    if (p.H == p.Hk) return 0;
    typedef typename E::raw raw;
    const int64_t n = int64_t(p.batch) * p.L * p.Hk * p.dk;
    delta_heads_kernel<E><<<unsigned((n + 255) / 256), 256, 0, stream>>>(
        p.part_q, p.part_k, static_cast<raw*>(p.dq), static_cast<raw*>(p.dk_), n, p.dk, p.H / p.Hk);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_grad_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        return cls::launch<decltype(e), decltype(dk)::value>(p, stream);
    });
}
