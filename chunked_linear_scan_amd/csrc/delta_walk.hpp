// What the forward and the backward walk over the chunks share: a workgroup of
// four waves that compute, 16 columns of a state each, and four that load.  The
// computing waves' work on a chunk is one long chain of products, so what
// bounds a walk is that chain's latency: the loading waves keep the loads and
// stores into LDS (56 registers and 60 instructions a chunk) out of it, and the registers that this
// frees hold the next operands while a product runs.
#pragma once

#include "delta.hpp"
#include "device_once.hpp"

namespace cls {

constexpr int kWalkCols = 64;      // columns to a workgroup
constexpr int kWalkThreads = 512;  // computing waves, then loading waves

// Asks for N matrix instructions with V vector ones behind each, of those between two scheduling barriers: left to
// itself the compiler issues products in blocks, during which the vector unit waits, and the other way round.
template <int N, int V>
__device__ __forceinline__ void interleave() {
    if constexpr (N > 0) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
        interleave<N - 1, V>();
    }
}
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// LDS of a walk: K, Q, NM matrices of a chunk and its factors, twice where that fits.
template <typename E, int DK, int NM>
struct WalkLds {
    typedef typename Mat<E>::raw raw;
    static constexpr int C = Mat<E>::kChunk;
    static constexpr int KS = C * LdsTile<E, DK>::kPitch, MS = C * LdsTile<E, C>::kPitch;
    static constexpr int kBuffer = int((2 * KS + NM * MS) * sizeof(raw) + 3 * C * sizeof(float));
    static constexpr bool kTwice = 2 * kBuffer <= 160 * 1024;
    static constexpr int kBytes = kTwice ? 2 * kBuffer : kBuffer;
    raw *k, *q, *m;
    float* v;  // e^gamma, e^(gamma_C - gamma), beta
    __device__ __forceinline__ WalkLds(char* lds, int at) {
        k = reinterpret_cast<raw*>(lds + (kTwice ? (at & 1) * kBuffer : 0));
        q = k + KS;
        m = q + KS;
        v = reinterpret_cast<float*>(m + NM * MS);
    }
};

// The loading waves' part: chunks first, first + step, .. (n of them).
template <typename E, int DK, int NM>
__device__ __forceinline__ void walk_load(const DeltaParams& p, char* lds, int b, int h, int end, int first, int step, int n) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef ChunkMats<E> CM;
    typedef WalkLds<E, DK, NM> Lds;
    constexpr int C = M::kChunk, THREADS = 256;
    constexpr int64_t SZ = sizeof(raw);
    typedef TileRegs<E, C, DK, THREADS> KRegs;
    typedef TileRegs<E, C, C, THREADS> MRegs;
    const int kh = h / (p.H / p.Hk), tid = threadIdx.x % THREADS;
    const raw* K = static_cast<const raw*>(p.k) + b * p.sk.batch + kh * p.sk.head;
    const raw* Q = static_cast<const raw*>(p.q) + b * p.sq.batch + kh * p.sq.head;
    const uint32_t ok = KRegs::offset(p.sk.token, p.dk), oq = KRegs::offset(p.sq.token, p.dk), om = MRegs::offset(C, C);
    // two chunks in flight: a chunk takes less time than a load from memory
    struct Set {
        KRegs k, q;
        MRegs m[NM];
        float v;
    } set[2];
    const auto fetch = [&](Set& r, int i) {
        const int c = first + i * step, t0 = c * C, left = end - t0;
        r.k.load(buffer(K + t0 * p.sk.token, left * p.sk.token * SZ), ok, p.sk.token);
        r.q.load(buffer(Q + t0 * p.sq.token, left * p.sq.token * SZ), oq, p.sq.token);
        const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
        const raw* mats = static_cast<const raw*>(p.mats) + chunk * CM::kAll * CM::kSize;
#pragma unroll
        for (int m = 0; m < NM; ++m) r.m[m].load(buffer(mats + m * CM::kSize), om, C);
        r.v = p.vecs[chunk * 3 * C + (tid < 3 * C ? tid : 0)];
    };
    const auto put = [&](const Set& r, int i) {
        const Lds to(lds, i);
        r.k.template store<LdsTile<E, DK>>(to.k);
        r.q.template store<LdsTile<E, DK>>(to.q);
#pragma unroll
        for (int m = 0; m < NM; ++m) r.m[m].template store<LdsTile<E, C>>(to.m + m * Lds::MS);
        if (tid < 3 * C) to.v[tid] = r.v;
    };
    const auto last = [&](int i) { return i < n ? i : n - 1; };  // past the end: loaded again, not used
    if (n == 0) {
        if (Lds::kTwice) lds_meet();
        return;
    }
    fetch(set[0], 0);
    fetch(set[1], last(1));
    if constexpr (Lds::kTwice) {
        put(set[0], 0);
        fetch(set[0], last(2));
        lds_meet();
        for (int i = 0; i < n; i += 2) {
            if (i + 1 < n) put(set[1], i + 1);
            fetch(set[1], last(i + 3));
            lds_meet();
            if (i + 1 == n) break;
            if (i + 2 < n) put(set[0], i + 2);
            fetch(set[0], last(i + 4));
            lds_meet();
        }
    } else {
        for (int i = 0; i < n; i += 2) {
            lds_meet();
            put(set[0], i);
            lds_meet();
            if (i + 1 == n) break;
            fetch(set[0], last(i + 2));
            lds_meet();
            put(set[1], i + 1);
            lds_meet();
            fetch(set[1], last(i + 3));
        }
    }
}

// The computing waves' part: f(i, lds) for every chunk that the loading waves bring.
template <typename Lds, typename F>
__device__ __forceinline__ void walk(char* lds, int n, F&& f) {
    if constexpr (Lds::kTwice) {
        lds_meet();
        for (int i = 0; i < n; ++i) {
            f(i, Lds(lds, i));
            lds_meet();
        }
    } else {
        for (int i = 0; i < n; ++i) {
            lds_meet();
            lds_meet();
            f(i, Lds(lds, i));
        }
    }
}

// A lane's part of a state [dv, dk] in memory: column n, rows 4 (l/16) + r of each tile; `of` is the state's place
// among those of all sequences and heads.
template <int KT>
__device__ __forceinline__ void load_state(f32x4 (&S)[KT], const float* from, int64_t of, int n, const DeltaParams& p) {
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] = f32x4{0, 0, 0, 0};
    if (from) {
        const Buffer b = buffer(from + of * p.dv * p.dk, int64_t(p.dv) * p.dk * 4);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const int d = 16 * t + 4 * group4();
            const uint32_t at = uint32_t(n * p.dk + d) * 4;
            if (p.dk % 4 == 0) {
                S[t] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, int(d < p.dk && n < p.dv ? at : kOutside), 0, 0));
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[t][r] = as_float(load_one<ElemF32>(b, d + r < p.dk && n < p.dv ? at + 4 * r : kOutside));
            }
        }
    }
    // waited for here, not in the loop, where a wait for loads is one for the stores before them
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v = S[t][r];
            asm volatile("" : "+v"(v));
            S[t][r] = v;
        }
}
template <int KT>
__device__ __forceinline__ void store_state(const f32x4 (&S)[KT], float* to, int64_t of, int n, const DeltaParams& p) {
    const Buffer b = buffer(to + of * p.dv * p.dk, int64_t(p.dv) * p.dk * 4);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const int d = 16 * t + 4 * group4();
        const uint32_t at = uint32_t(n * p.dk + d) * 4;
        if (p.dk % 4 == 0) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[t]), b, int(d < p.dk && n < p.dv ? at : kOutside), 0, 0);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) store_one<ElemF32>(b, d + r < p.dk && n < p.dv ? at + 4 * r : kOutside, S[t][r]);
        }
    }
}
// The same as a chunk's [dk, dv] for the kernel of the gradients.
template <int KT>
__device__ __forceinline__ void keep_state(const f32x4 (&S)[KT], float* states, int64_t chunk, uint32_t offset, const DeltaParams& p) {
    const Buffer b = buffer(states + chunk * p.dk * p.dv, int64_t(p.dk) * p.dv * 4);
    const uint32_t at = here(offset);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) store_one<ElemF32>(b, at + uint32_t((16 * t + r) * p.dv) * 4, S[t][r]);
}

}  // namespace cls
