// What the forward and the backward walk over the chunks share: a workgroup of
// two or four waves that compute, 16 columns of a state each, and four that load.  The
// computing waves' work on a chunk is one long chain of products, so what
// bounds a walk is that chain's latency: the loading waves keep the traffic with memory
// (but for kept states) out of it, and the registers that this
// frees hold the next operands while a product runs.  V (or dY) comes and y (or
// dV) leaves through LDS as whole rows, too.
#pragma once

#include "delta.hpp"
#include "device_once.hpp"

namespace cls {

// The computing waves of a workgroup: what bounds four is LDS, from which each reads the chunk's matrices for itself
// (3200 cycles a chunk of 128-element keys, of which the products take 1700), so while a compute unit is free for every
// 32 columns there are two.
inline int walk_waves(const DeltaParams& p) {
    return int64_t(p.batch) * p.H * ((p.dv + 31) / 32) <= 256 ? 2 : 4;
}

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

// Lets the last product's result be written: the compiler's copies of it at a loop's end (v_mov_b64) were seen two
// instructions behind the product, without the wait for its last two registers.
__device__ __forceinline__ void settle(f32x4& x) {
    float a = x[0], b = x[1], c = x[2], d = x[3];
    asm volatile("s_nop 15" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
    x = f32x4{a, b, c, d};
}

// LDS of a walk: K, Q, NM matrices of a chunk, its columns of V and its factors, and those of y; twice where that fits.
template <typename E, int DK, int NM, int WAVES>
struct WalkLds {
    typedef typename Mat<E>::raw raw;
    typedef LdsTile<E, DK> KTile;
    typedef LdsTile<E, Mat<E>::kChunk> MTile;
    typedef LdsTile<E, 64> XTile;  // whose second half two waves do not use
    static constexpr int C = Mat<E>::kChunk, kCols = 16 * WAVES;
    static constexpr int kThreads = 64 * (WAVES + 4);  // computing waves, then loading waves
    static constexpr int KS = C * KTile::kPitch, MS = C * MTile::kPitch, XS = C * XTile::kPitch;
    static constexpr int YP = 64 + 16 / int(sizeof(raw));  // pitch of y: four rows touch every bank once
    static constexpr int kBuffer = int((2 * KS + NM * MS + XS) * sizeof(raw) + kVecs * C * sizeof(float));
    static constexpr int kOut = C * YP * int(sizeof(raw));
    static constexpr bool kTwice = 2 * (kBuffer + kOut) <= 160 * 1024;
    static constexpr int kBytes = (kTwice ? 2 : 1) * (kBuffer + kOut);
    raw *k, *q, *m, *x, *y;
    float* v;
    __device__ __forceinline__ WalkLds(char* lds, int at) {
        const int one = kTwice ? at & 1 : 0;
        k = reinterpret_cast<raw*>(lds + one * kBuffer);
        q = k + KS;
        m = q + KS;
        x = m + NM * MS;
        v = reinterpret_cast<float*>(x + XS);
        y = reinterpret_cast<raw*>(lds + (kTwice ? 2 : 1) * kBuffer + one * kOut);
    }
};

// Columns of V or dY in, of y or dV out.
struct WalkColumns {
    const void* x;
    Strided3 sx;
    void* y;
    bool vec_x, vec_y;
};

// The loading waves' part: chunks first, first + step, .. (n of them).
template <typename E, int DK, int NM, int WAVES>
__device__ __forceinline__ void walk_load(const DeltaParams& p, const WalkColumns& w, char* lds, int b, int h, int col0, int end,
                                          int first, int step, int n) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef ChunkMats<E> CM;
    typedef WalkLds<E, DK, NM, WAVES> Lds;
    constexpr int C = M::kChunk, THREADS = 256;
    constexpr int64_t SZ = sizeof(raw);
    typedef TileRegs<E, C, DK, THREADS> KRegs;
    typedef TileRegs<E, C, C, THREADS> MRegs;
    typedef TileRegs<E, C, 64, THREADS> XRegs;
    const int kh = h / (p.H / p.Hk), tid = (threadIdx.x - 64 * WAVES) % THREADS;
    const raw* K = static_cast<const raw*>(p.k) + b * p.sk.batch + kh * p.sk.head;
    const raw* Q = static_cast<const raw*>(p.q) + b * p.sq.batch + kh * p.sq.head;
    const raw* X = static_cast<const raw*>(w.x) + b * w.sx.batch + h * w.sx.head + col0;
    const int cols = p.dv - col0 < Lds::kCols ? p.dv - col0 : Lds::kCols;
    const uint32_t ok = KRegs::offset(p.sk.token, p.dk, tid), oq = KRegs::offset(p.sq.token, p.dk, tid);
    const uint32_t ox = XRegs::offset(w.sx.token, cols, tid), om = MRegs::offset(C, C, tid);
    const uint32_t om0 = MRegs::offset(C, 32, tid);  // of the first 32 rows only 32 columns are there
    // Two chunks in flight: a chunk may take less time than a load from memory.  (One where LDS holds one: dk above 128,
    // whose chunks are longer and whose vectors would be twice as many.)
    constexpr int SETS = Lds::kTwice ? 2 : 1;
    struct Set {
        KRegs k, q;
        MRegs m[NM];
        XRegs x;
        u32x4 v;
    } set[SETS];
    const auto fetch = [&](Set& r, int i) {
        const int c = first + i * step, t0 = c * C, left = end - t0;
        r.k.load(buffer(K + t0 * p.sk.token, left * p.sk.token * SZ), ok, p.sk.token);
        r.q.load(buffer(Q + t0 * p.sq.token, left * p.sq.token * SZ), oq, p.sq.token);
        const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
        const raw* mats = static_cast<const raw*>(p.mats) + chunk * CM::kAll * CM::kSize;
#pragma unroll
        for (int m = 0; m < NM; ++m) r.m[m].load(buffer(mats + m * CM::kSize), om, C, om0);
        const Buffer bx = buffer(X + t0 * w.sx.token, left * w.sx.token * SZ - col0 * SZ);
        if (w.vec_x) {
            r.x.load(bx, ox, w.sx.token);
        } else {
#pragma unroll
            for (int v = 0; v < XRegs::N; ++v) {
                const int at = tid + v * THREADS, row = at / XRegs::PER_ROW, col = at % XRegs::PER_ROW * XRegs::VE;
                r.x.r[v] = u32x4{0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < XRegs::VE; ++e) {
                    const uint32_t one = load_one<E>(bx, col + e < cols ? uint32_t((row * w.sx.token + col + e) * SZ) : kOutside);
                    if constexpr (SZ == 4) r.x.r[v][e] = one;
                    else r.x.r[v][e >> 1] |= one << (16 * (e & 1));
                }
            }
        }
        r.v = ldg_b128(p.vecs + chunk * kVecs * C + 4 * (tid < kVecs * C / 4 ? tid : 0));
    };
    const auto put = [&](const Set& r, int i) {
        const Lds to(lds, i);
        r.k.template store<typename Lds::KTile>(to.k, tid);
        r.q.template store<typename Lds::KTile>(to.q, tid);
#pragma unroll
        for (int m = 0; m < NM; ++m) r.m[m].template store<typename Lds::MTile>(to.m + m * Lds::MS, tid);
        r.x.template store<typename Lds::XTile>(to.x, tid);
        if (tid < kVecs * C / 4) *reinterpret_cast<u32x4*>(to.v + 4 * tid) = r.v;
    };
    const int64_t row = int64_t(p.H) * p.dv;  // of a token of y
    raw* Y = static_cast<raw*>(w.y) + int64_t(b) * p.L * row + int64_t(h) * p.dv + col0;
    const auto out = [&](int i) {
        const Lds from(lds, i);
        const int t0 = (first + i * step) * C;
        const Buffer by = buffer(Y + t0 * row, int64_t(p.L - t0) * row * SZ - (int64_t(h) * p.dv + col0) * SZ);
#pragma unroll
        for (int v = 0; v < XRegs::N; ++v) {
            const int at = tid + v * THREADS, r = at / XRegs::PER_ROW, col = at % XRegs::PER_ROW * XRegs::VE;
            u32x4 x = *reinterpret_cast<const u32x4*>(from.y + r * Lds::YP + col);
            if (t0 + r >= end) x = u32x4{0, 0, 0, 0};  // padding
            const uint32_t to = uint32_t((r * row + col) * SZ);
            if (w.vec_y) {
                __builtin_amdgcn_raw_buffer_store_b128(x, by, int(col < cols ? to : kOutside), 0, 0);
            } else {
#pragma unroll
                for (int e = 0; e < XRegs::VE; ++e) {
                    const uint32_t word = x[SZ == 4 ? e : e >> 1], at2 = col + e < cols ? to + uint32_t(e * SZ) : kOutside;
                    if constexpr (SZ == 4) __builtin_amdgcn_raw_buffer_store_b32(word, by, int(at2), 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b16(uint16_t(word >> (16 * (e & 1))), by, int(at2), 0, 0);
                }
            }
        }
    };
    const auto last = [&](int i) { return i < n ? i : n - 1; };  // past the end: loaded again, not used
    if (n > 0) {
        fetch(set[0], 0);
        if constexpr (Lds::kTwice) {
            // while chunk i is computed: y of the one before leaves, the one behind it comes
            fetch(set[1], last(1));
            put(set[0], 0);
            fetch(set[0], last(2));
            lds_meet();
            for (int i = 0; i < n; i += 2) {
                if (i > 0) out(i - 1);
                if (i + 1 < n) put(set[1], i + 1);
                fetch(set[1], last(i + 3));
                lds_meet();
                if (i + 1 == n) break;
                out(i);
                if (i + 2 < n) put(set[0], i + 2);
                fetch(set[0], last(i + 4));
                lds_meet();
            }
        } else {
            for (int i = 0; i < n; ++i) {
                lds_meet();
                if (i > 0) out(i - 1);
                put(set[0], i);
                lds_meet();
                fetch(set[0], last(i + 1));
            }
            lds_meet();
        }
        out(n - 1);
    }
    // whole chunks of padding
    const int64_t t1 = (end + C - 1) / C * C;
    for (int64_t at = tid; at < (p.L - t1) * cols; at += THREADS) Y[(t1 + at / cols) * row + at % cols] = raw(0);
}

// The computing waves' part: f(i, lds) for every chunk that the loading waves bring.
template <typename Lds, typename F>
__device__ __forceinline__ void walk(char* lds, int n, F&& f) {
    if (n == 0) return;
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
        lds_meet();
    }
}

// A lane's part of a state [dv, dk] in memory: column n, rows 4 (l/16) + r of each tile; `of` is the state's place
// among those of all sequences and heads (and chunks).
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
// A column's values of the chunk's tokens: [dv, C].
template <int C>
__device__ __forceinline__ void store_tokens(const f32x4 (&x)[C / 16], float* to, int64_t chunk, int n, const DeltaParams& p) {
    const Buffer b = buffer(to + chunk * p.dv * C, int64_t(p.dv) * C * 4);
#pragma unroll
    for (int t = 0; t < C / 16; ++t)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x[t]), b,
                                               int(n < p.dv ? uint32_t(n * C + 16 * t + 4 * group4()) * 4 : kOutside), 0, 0);
}

// A result tile's rows to a column of y in LDS.
template <typename E, int YP>
__device__ __forceinline__ void put_column(typename E::raw* y, int t, const f32x4& v) {
    typename E::raw* to = y + 16 * t * YP;
    if constexpr (Mat<E>::kSplit) {
        const uint32_t a = Mat<E>::pack(v[0], v[1]), b = Mat<E>::pack(v[2], v[3]);
        to[0] = uint16_t(a);
        to[YP] = uint16_t(a >> 16);
        to[2 * YP] = uint16_t(b);
        to[3 * YP] = uint16_t(b >> 16);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) to[r * YP] = E::put(v[r]);
    }
}

}  // namespace cls
