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
// All computed operands go in as two parts, so 16-bit gradients are off by their own rounding and little else.
// Bound by memory: a chunk's states and corrections (192 KB of the 288 KB that it moves for 64 tokens, keys and values of 128)
// are read once, 32 of dv at a time, past the caches: 4 x 2048 x 16 heads 152 us, 4.0 TB/s; through the caches 163 (with the
// products with S and with dS in two walks over dv, a fifth longer).  LDS has K and those tiles, and Q and the pairs in the
// tiles' place afterwards, so that two workgroups fit a compute unit.
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
    // cols: a multiple of 4
    __device__ __forceinline__ void load(Buffer b, int row0, int cols) {
        const int col = threadIdx.x % PER_ROW * 4, row = row0 + int(threadIdx.x) / PER_ROW;
        const uint32_t at = col < cols ? uint32_t(row * cols + col) * 4 : kOutside;
#pragma unroll
        for (int n = 0; n < N; ++n)
            r[n] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, int(at + uint32_t(n * STEP * cols * 4)), 0, kStream));
    }
    __device__ __forceinline__ void store(typename E::raw* to) const {
        const int col = threadIdx.x % PER_ROW * 4;
#pragma unroll
        for (int n = 0; n < N; ++n) put4<E>(to + Lds::quad(int(threadIdx.x) / PER_ROW + n * STEP, col), kPart, r[n]);
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
    static constexpr int kTiles = kParts * 32 * (2 * KP + 2 * MP);  // tiles of S, dS, N and Z
    static constexpr int kPairs = C * KP + 2 * kParts * C * MP;     // Q, pB and pP, in the same place
    static constexpr int kUnion = kTiles > kPairs ? kTiles : kPairs;
    static constexpr size_t bytes = (C * KP + kUnion) * sizeof(typename M::raw) + (Decays<C>::kFloats + (2 + C / 16) * C + 2 * (C / 16)) * sizeof(float);
};

template <typename E, int DK>
__global__ __launch_bounds__(Mat<E>::kChunk * 4, Mat<E>::kSplit && DK <= 128 ? 2 : 1) void delta_grad_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef GradSize<E, DK> G;
    constexpr int C = G::C, NT = C / 16, KT = DK / 16, THREADS = 64 * NT, KP = G::KP, MP = G::MP;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    raw* sK = reinterpret_cast<raw*>(lds);
    raw* sS = sK + C * KP;
    raw* sD = sS + G::kParts * 32 * KP;
    raw* sN = sD + G::kParts * 32 * KP;
    raw* sZ = sN + G::kParts * 32 * MP;
    raw* sQ = sS;  // once the tiles are done with
    raw* sB = sQ + C * KP;
    raw* sP = sB + G::kParts * C * MP;
    float* sG = reinterpret_cast<float*>(sS + G::kUnion);
    float* sRow = sG + Decays<C>::kFloats;  // read_i + sum_j F_ij
    float* sWrite = sRow + C;   // write_j
    float* sCol = sWrite + C;   // [NT][C]: sums of F over a wave's tokens
    float* sDot = sCol + NT * C;
    float* sMost = sDot + NT;  // the waves' largest pairs

    const int rep = p.H / p.Hk;
    const UnitPart u = unit_part(p.batch * p.nchunk * p.Hk, rep);
    const int kh = u.unit % p.Hk, h = kh * rep + u.part, c = u.unit / p.Hk % p.nchunk, b = u.unit / p.Hk / p.nchunk;
    const int end = seq_end(p.seqlens, b, p.L), t0 = c * C;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane16(), g4 = group4();
    const int i = 16 * w + l16, tok = t0 + i;  // this lane's token
    const bool in = tok < end;

    // rows of the outputs: of a token's head, or its part of a key head's sum
    const auto put_rows = [&](auto&& q, auto&& k) {
        int at = tok;
        asm volatile("" : "+v"(at));  // addresses from here: those of all tiles would be kept from the padding's on
        if (at >= p.L) return;
        const int64_t one = ((int64_t(b) * p.L + at) * p.Hk + kh) * p.dk, part = ((int64_t(b) * p.L + at) * p.H + h) * p.dk;
        const auto put = [&](raw* whole, float* parts, int d, const f32x4& v) {
            if (rep > 1) {
                if (p.dk % 4 == 0) {
                    if (d < p.dk) *reinterpret_cast<f32x4*>(parts + part + d) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (d + e < p.dk) parts[part + d + e] = v[e];
                }
            } else if (p.dk % 4 == 0 && p.vec_dqk) {
                if (d < p.dk) put4<E>(whole + one + d, 0, v);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (d + e < p.dk) whole[one + d + e] = E::put(v[e]);
            }
        };
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            put(static_cast<raw*>(p.dq), p.part_q, 16 * t + 4 * g4, q(t));
            put(static_cast<raw*>(p.dk_), p.part_k, 16 * t + 4 * g4, k(t));
        }
    };
    if (t0 >= end) {  // padding
        const auto none = [](int) { return f32x4{0, 0, 0, 0}; };
        put_rows(none, none);
        if (g4 == 0 && tok < p.L) p.dg[(int64_t(b) * p.L + tok) * p.H + h] = p.dbeta[(int64_t(b) * p.L + tok) * p.H + h] = 0.0f;
        return;
    }

    // dS, Z and what comes of them are times a power of two, and so are products with dY times `scale`
    const GradPower size = grad_power<E>(p, int64_t(b) * p.H + h);
    const float scale = p.scale * size.ratio;
    const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
    const float* vecs = p.vecs + chunk * kVecs * C;
    const Buffer bS = buffer(p.states + chunk * p.dv * p.kpitch, int64_t(p.dv) * p.kpitch * 4);
    const Buffer bD = buffer(p.dstates + chunk * p.dv * p.kpitch, int64_t(p.dv) * p.kpitch * 4);
    const Buffer bN = buffer(p.fixes + chunk * p.dv * C, int64_t(p.dv) * C * 4);
    const Buffer bZ = buffer(p.z + chunk * p.dv * C, int64_t(p.dv) * C * 4);
    const int left = end - t0 < C ? end - t0 : C;  // tokens of the chunk
    // dY and V, of the lane's token
    constexpr int SZ = sizeof(raw);
    const auto rows_of = [&](const void* m, const Strided3& s) {
        return buffer(static_cast<const raw*>(m) + b * s.batch + h * s.head + t0 * s.token, left * s.token * SZ);
    };
    const Buffer bY = rows_of(p.dy, p.sdy), bV = rows_of(p.v, p.sv);
    const uint32_t oy = uint32_t(i * p.sdy.token * SZ), ov = uint32_t(i * p.sv.token * SZ);
    typedef LdsTile<E, DK> KTile;
    typedef LdsTile<E, C> MTile;
    const KTile kt;
    const MTile mt, mw(16 * w);  // mw: of the wave's tokens
    typedef TileRegs<E, C, DK, THREADS> Regs;
    const raw* Q = static_cast<const raw*>(p.q) + b * p.sq.batch + t0 * p.sq.token + kh * p.sq.head;
    {
        Regs k;
        const raw* K = static_cast<const raw*>(p.k) + b * p.sk.batch + t0 * p.sk.token + kh * p.sk.head;
        k.load(buffer(K, left * p.sk.token * sizeof(raw)), Regs::offset(p.sk.token, p.dk, tid), p.sk.token);
        if (tid < C) Decays<C>::put(sG, t0 + tid < end ? p.g[b * p.g_batch + int64_t(t0 + tid) * p.g_token + h] : 0.0f);
        k.template store<KTile>(sK, tid);
    }

    // 32 of dv at a time: X1 = S dY^T, X2 = S Z^T, X3 = dS N^T, <S, dS>, dP^T and M^T
    f32x4 X1[KT], X2[KT], X3[KT], dP[NT], Mz[NT];
#pragma unroll
    for (int t = 0; t < KT; ++t) X1[t] = X2[t] = X3[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < NT; ++t) dP[t] = Mz[t] = f32x4{0, 0, 0, 0};
    float zv = 0.0f, both = 0.0f;  // Z_i.V_i
    typedef Tile32<E, DK, THREADS> STile;
    typedef Tile32<E, C, THREADS> NTile;
    STile rs, rd;
    NTile rn, rz;
    typename M::frag y1, v1;  // of dY and V
    const auto ahead = [&](int d0) {
        rs.load(bS, d0, p.kpitch);
        rd.load(bD, d0, p.kpitch);
        rn.load(bN, d0, C);
        rz.load(bZ, d0, C);
        y1 = load_frag<E>(bY, oy, d0, p.dv);
        v1 = load_frag<E>(bV, ov, d0, p.dv);
    };
    ahead(0);
    for (int d0 = 0; d0 < p.dv; d0 += 32) {
        lds_meet();
        rs.store(sS);
        rd.store(sD);
        rn.store(sN);
        rz.store(sZ);
        both += rs.dot(rd);
        typename M::frag yf = y1;
        const typename M::frag v = v1;
        if constexpr (kSized<E>) yf = times<E>(yf, size.dy);
        lds_meet();
        if (d0 + 32 < p.dv) {
            ahead(d0 + 32);
        } else {  // Q, in registers of S
            Regs q;
            q.load(buffer(Q, left * p.sq.token * sizeof(raw)), Regs::offset(p.sq.token, p.dk, tid), p.sq.token);
#pragma unroll
            for (int n = 0; n < STile::N; ++n) rs.r[n] = __builtin_bit_cast(f32x4, q.r[n]);
        }
        const Two<E> zf = two_cols<E>(mw, sZ, 0), nf = two_cols<E>(mw, sN, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float z = M::at(zf.hi, e);
            if constexpr (M::kSplit) z += M::at(zf.lo, e);
            zv = fmaf(z, M::at(v, e), zv);
        }
        // operands are read a tile at a time and not further ahead: registers are what is short
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const Two<E> s = two_cols<E>(kt, sS, t), d = two_cols<E>(kt, sD, t);
            X1[t] = mma2<E>(s, yf, X1[t]);
            X2[t] = mma3<E, small_parts(DK)>(s, zf, X2[t]);
            X3[t] = mma3<E, small_parts(DK)>(d, nf, X3[t]);
            fence();
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {  // without a branch: those of later tokens are not used
            const Two<E> nj = two_cols<E>(mt, sN, t);
            dP[t] = mma2<E>(nj, yf, dP[t]);
            Mz[t] = mma3<E, small_parts(DK)>(nj, zf, Mz[t]);
            fence();
        }
        settle();
    }
    lds_meet();  // the tiles are read
    {
        static_assert(Regs::N == STile::N, "");
        Regs q;
#pragma unroll
        for (int n = 0; n < STile::N; ++n) q.r[n] = __builtin_bit_cast(u32x4, rs.r[n]);
        q.template store<KTile>(sQ, tid);
    }
    lds_meet();
    zv = sum_groups(zv);
    const auto dot_row = [&](const raw* m, const f32x4 (&x)[KT]) {
        float v = 0.0f;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const f32x4 a = load4<E>(m + KTile::quad(i, 16 * t + 4 * g4));
#pragma unroll
            for (int r = 0; r < 4; ++r) v = fmaf(a[r], x[t][r], v);
        }
        return sum_groups(v);
    };
    const float start = vecs[kStart * C + i], beta = vecs[kBeta * C + i], fade = vecs[kStart * C + C - 1];
    const float after = vecs[kWrite * C + i];
    const float qx = scale * start * dot_row(sQ, X1), kx = start * dot_row(sK, X2), write = after * dot_row(sK, X3);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        X1[t] *= scale * start;
        X2[t] = after * X3[t] - beta * start * X2[t];
        // here, not where it is used: both are kept until then otherwise
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v = X2[t][r], u = X1[t][r];
            asm volatile("" : "+v"(v), "+v"(u));
            X2[t][r] = v;
            X1[t][r] = u;
        }
    }
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
        if (t > w) kk[t] = dP[t] = Mz[t] = f32x4{0, 0, 0, 0};
    Decays<C>::each(sG, w, [&](int t, const f32x4& d) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = 16 * t + 4 * g4 + r;
            const float m = j < i ? d[r] * Mz[t][r] : 0.0f;
            dP[t][r] = j <= i ? scale * d[r] * dP[t][r] : 0.0f;
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
        if (tok < p.L) p.dbeta[(int64_t(b) * p.L + tok) * p.H + h] = in ? size.down * (zv - kx - db) : 0.0f;
    }
    // The pairs are products of dY or Z with the corrections, which may be of any size: a power of two of the chunk's
    // own brings them to 2^10, at most 2^15 as they only add to the states' parts.
    Power pairs{1.0f, 1.0f};
    if constexpr (kSized<E>) {
        float most = 0.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) most = larger(larger(most, dP[t][r]), Mz[t][r]);
        most = wave_max(most);
        if ((tid & 63) == 0) sMost[w] = most;
        lds_meet();
#pragma unroll
        for (int k = 0; k < NT; ++k) most = fmaxf(most, sMost[k]);
        pairs = power_to(most, 10, 15);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dP[t] *= pairs.up;
            Mz[t] *= pairs.up;
        }
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            X1[t] *= pairs.up;
            X2[t] *= pairs.up;
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        put4<E>(sB + MTile::quad(i, 16 * t + 4 * g4), C * MP, Mz[t]);  // zeros for the tiles behind w
        put4<E>(sP + MTile::quad(i, 16 * t + 4 * g4), C * MP, dP[t]);
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
            p.dg[(int64_t(b) * p.L + t0 + tid) * p.H + h] = t0 + tid < end ? size.down * v : 0.0f;
        }
    }
    // the pairs' parts: as the later token (operands from the lanes), as the earlier one (from LDS)
#pragma unroll
    for (int s = 0; s < NT / 2; ++s) {
        const Two<E> bi = two<E>(Mz[2 * s], Mz[2 * s + 1]), pi = two<E>(dP[2 * s], dP[2 * s + 1]);
        const auto earlier = [&](const raw* m) {
            Two<E> x;
            x.hi = mw.cols(m, s, 0);
            if constexpr (M::kSplit) x.lo = mw.cols(m + C * MP, s, 0);
            return x;
        };
        const Two<E> bj = earlier(sB), pj = earlier(sP);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const typename M::frag kc = kt.cols(sK, s, t), qc = kt.cols(sQ, s, t);
            X1[t] = mma2<E>(kc, pi, X1[t]);
            X2[t] = mma2<E>(kc, bi, X2[t]);
            X2[t] = mma2<E>(kc, bj, X2[t]);
            X2[t] = mma2<E>(qc, pj, X2[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
        if (!in) X1[t] = X2[t] = f32x4{0, 0, 0, 0};
    put_rows([&](int t) { return size.down * (pairs.down * X1[t]); }, [&](int t) { return size.down * (pairs.down * X2[t]); });
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
