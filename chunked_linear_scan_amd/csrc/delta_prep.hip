// Gated delta rule: what a chunk of C tokens needs that no state enters, for all
// chunks at once.  With D_ij = e^(g_{j+1} + .. + g_i) and A_ij = beta_i D_ij k_i.k_j
// (j < i), the corrections N of a chunk solve (I + A) N = diag(beta) (V - e^gamma K S0);
// here are T - I, T = (I + A)^-1, P_ij = D_ij q_i.k_j (j <= i) and the factors
// e^gamma_i and e^(gamma_C - gamma_j) of reads and writes of the state.  The ones
// of T's diagonal are left out so that what they multiply stays in fp32 (with two
// bf16 numbers to an operand half of the states' error came from them).  P is without
// the scale, so that with fp16 fewer entries are subnormal.
//
// T by blocks: the 16x16 diagonal blocks by forward substitution (a column to a
// lane, in registers), then T10 = -T11 A10 T00 for pairs of blocks and pairs of
// pairs, in fp32 matrix products.  The product form (I - A)(I + A^2)(I + A^4).. is
// shorter, but its powers grow with alike keys (binomially), and cancel.
#include <hip/hip_runtime.h>

#include "delta.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

// One 16x16 product in fp32: rows of a in LDS, columns held as a result tile is.
__device__ __forceinline__ f32x4 mul16(const float* a, int pitch, const f32x4& b, f32x4 c) {
    const f32x4 av = *reinterpret_cast<const f32x4*>(a + lane16() * pitch + 4 * group4());
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(av[r], b[r], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x4 tile16(const float* t, int pitch) {
    f32x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = t[(4 * group4() + r) * pitch + lane16()];
    return v;
}
__device__ __forceinline__ void put16(float* t, int pitch, const f32x4& v) {
#pragma unroll
    for (int r = 0; r < 4; ++r) t[(4 * group4() + r) * pitch + lane16()] = -v[r];
}

template <typename E, int DK>
__global__ __launch_bounds__(Mat<E>::kChunk * 4) void delta_prep_kernel(DeltaParams p) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    constexpr int C = M::kChunk, NT = C / 16, THREADS = 64 * NT;
    typedef LdsTile<E, DK> KT;
    constexpr int AP = C + 4;
    // K and Q, and once their products are taken A and T in the same place
    constexpr size_t kKeys = 2 * C * KT::kPitch * sizeof(raw), kTri = 2 * C * AP * sizeof(float);
    __shared__ __attribute__((aligned(16))) char lds[kKeys > kTri ? kKeys : kTri];
    __shared__ __attribute__((aligned(16))) float sG[Decays<C>::kFloats];
    raw* sK = reinterpret_cast<raw*>(lds);
    raw* sQ = sK + C * KT::kPitch;
    float* sA = reinterpret_cast<float*>(lds);
    float* sT = sA + C * AP;

    const int rep = p.H / p.Hk;
    const UnitPart u = unit_part(p.batch * p.nchunk * p.Hk, rep);
    const int kh = u.unit % p.Hk, h = kh * rep + u.part, c = u.unit / p.Hk % p.nchunk, b = u.unit / p.Hk / p.nchunk;
    const int end = seq_end(p.seqlens, b, p.L), t0 = c * C;
    if (t0 >= end) return;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane16(), g4 = group4();
    {
        typedef TileRegs<E, C, DK, THREADS> Regs;
        Regs k, q;
        const int left = end - t0;
        const raw* K = static_cast<const raw*>(p.k) + b * p.sk.batch + t0 * p.sk.token + kh * p.sk.head;
        const raw* Q = static_cast<const raw*>(p.q) + b * p.sq.batch + t0 * p.sq.token + kh * p.sq.head;
        k.load(buffer(K, left * p.sk.token * sizeof(raw)), Regs::offset(p.sk.token, p.dk, tid), p.sk.token);
        q.load(buffer(Q, left * p.sq.token * sizeof(raw)), Regs::offset(p.sq.token, p.dk, tid), p.sq.token);
        if (tid < C) Decays<C>::put(sG, t0 + tid < end ? p.g[b * p.g_batch + int64_t(t0 + tid) * p.g_token + h] : 0.0f);
        k.template store<KT>(sK, tid);
        q.template store<KT>(sQ, tid);
    }
    const int i = 16 * w + l16;  // this lane's token: the row of A and P
    const float beta = t0 + i < end ? p.beta[b * p.b_batch + int64_t(t0 + i) * p.b_token + h] : 0.0f;
    __syncthreads();

    const KT kt;
    // products of keys, and of keys with queries, for tokens j = 16 t + 4 g4 + r before i
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

    __syncthreads();
    const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
    raw* mats = static_cast<raw*>(p.mats) + chunk * ChunkMats<E>::kAll * ChunkMats<E>::kSize;
    raw* P = mats + ChunkMats<E>::kParts * ChunkMats<E>::kSize;
    if (!(w & 1)) {  // above the diagonal, but within the 32 columns that products read
#pragma unroll
        for (int part = 0; part < ChunkMats<E>::kParts; ++part)
            put4<E>(P + part * ChunkMats<E>::kSize + i * C + 16 * (w + 1) + 4 * g4, 0, f32x4{0, 0, 0, 0});
    }
    Decays<C>::each(sG, w, [&](int t, const f32x4& d) {
        f32x4 a, q;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = 16 * t + 4 * g4 + r;
            a[r] = j < i ? beta * d[r] * kk[t][r] : 0.0f;
            q[r] = j <= i ? d[r] * qk[t][r] : 0.0f;
        }
        *reinterpret_cast<f32x4*>(sA + i * AP + 16 * t + 4 * g4) = a;
        put4<E>(P + i * C + 16 * t + 4 * g4, ChunkMats<E>::kSize, q);
    });
    if (g4 == 0) {
        float* vecs = p.vecs + chunk * kVecs * C;
        const float start = Decays<C>::start(sG, w);
        vecs[kRead * C + i] = p.scale * start;
        vecs[kWrite * C + i] = Decays<C>::behind(sG, w);
        vecs[kBeta * C + i] = beta;
        vecs[kBetaStart * C + i] = beta * start;
        vecs[kStart * C + i] = start;
    }
    __syncthreads();

    // the diagonal blocks' inverses: column l16 of block g4 to a lane
    if (tid < 16 * NT) {
        const float* a = sA + 16 * g4 * AP + 16 * g4;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float v = r == l16 ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < r; ++j) v = fmaf(-a[r * AP + j], x[j], v);
            x[r] = v;
            sT[(16 * g4 + r) * AP + 16 * g4 + l16] = v;
        }
    }
    __syncthreads();
    if (w < NT / 2) {  // T10 = -T11 (A10 T00) of each pair of blocks
        const int o = 32 * w;
        const f32x4 zero{0, 0, 0, 0};
        const f32x4 x = mul16(sA + (o + 16) * AP + o, AP, tile16(sT + o * AP + o, AP), zero);
        put16(sT + (o + 16) * AP + o, AP, mul16(sT + (o + 16) * AP + o + 16, AP, x, zero));
    }
    if constexpr (NT == 4) {  // the same of the two pairs; a wave to a 16x16 block of the result
        __syncthreads();
        const int mi = 2 + (w >> 1), ni = w & 1;
        f32x4 x[2], out{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            x[k] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (j >= ni)
                    x[k] = mul16(sA + 16 * (2 + k) * AP + 16 * j, AP, tile16(sT + 16 * j * AP + 16 * ni, AP), x[k]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (2 + k <= mi) out = mul16(sT + 16 * mi * AP + 16 * (2 + k), AP, x[k], out);
        put16(sT + 16 * mi * AP + 16 * ni, AP, out);
    }
    __syncthreads();
    // rows of T, four columns to a thread
#pragma unroll
    for (int n = 0; n < C * C / 4 / THREADS; ++n) {
        const int at = tid + n * THREADS, row = at / (C / 4), col = at % (C / 4) * 4;
        if (C == 64 && row < 32 && col >= 32) continue;  // never read
        f32x4 v = *reinterpret_cast<const f32x4*>(sT + row * AP + col);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = col + r >= row ? 0.0f : v[r];  // less I; blocks above were not written
        put4<E>(mats + row * C + col, ChunkMats<E>::kSize, v);
    }
}

template <typename E, int DK>
int launch(const DeltaParams& p, hipStream_t stream) {
    const unsigned wgs = unsigned(int64_t(p.batch) * p.nchunk * p.H);
    delta_prep_kernel<E, DK><<<wgs, 4 * Mat<E>::kChunk, 0, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace
}  // namespace cls

int cls_delta_prep_launch(const cls::DeltaParams& p, int dtype, hipStream_t stream) {
    return cls::by_type(dtype, p.dk, [&](auto e, auto dk) {
        return cls::launch<decltype(e), decltype(dk)::value>(p, stream);
    });
}
