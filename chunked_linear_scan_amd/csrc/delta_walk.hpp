// What the forward and the backward walk over the chunks share.  A chunk's work on a
// column of the state is one long chain of products, and of vector instructions on
// their results, of which a wave issues one in 8.5 cycles: that chain's latency
// bounds a walk, not any unit's rate.  So
//   - two waves have 16 columns of a state between them, each the rows of one half
//     of the keys' elements and the tokens of one half of a chunk.  Products with
//     the state are sums of two halves, which the waves exchange through LDS, as
//     they do what the other half's tokens add to the state: four meetings a chunk,
//     and half the instructions between them;
//   - four more waves load, and store what is not kept for the gradients, two
//     chunks ahead;
//   - operands are read from LDS a step before their products, and products are
//     interleaved with vector instructions.
// A workgroup has 32 columns: four computing waves, one to a SIMD, and four that
// load; or 16, and two.  A chunk of 64 tokens and keys of 128 takes 2.0 us, with 16
// columns 1.8 (0.2 more than with y's operands in one part each; then, one wave to
// 16 columns took 1.95 us with two computing waves to a workgroup, and 2.3 with
// four, where their reads of LDS took 3200 cycles of the 5500).
#pragma once

#include <type_traits>

#include "delta.hpp"
#include "device_once.hpp"

namespace cls {

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

// A workgroup of TILES has 16 TILES columns: computing waves (16 (w / 2).. of the columns, half w % 2), then four that load.
constexpr int walk_cols(int tiles) { return 16 * tiles; }
constexpr int walk_threads(int tiles) { return 128 * tiles + 256; }

// Calls f with the tiles of a walk's workgroups: two, or one, with the same rows of K, Q and matrices to load for half
// the columns, where all of those have a compute unit of their own (1 x 32768 x 32 heads of 128: 929 us instead of
// 1020; fp32 3 x 1000 x 8, values of 72: 69 instead of 75).
template <typename F>
int by_tiles(const DeltaParams& p, F&& f) {
    const int64_t columns = int64_t(p.batch) * p.H * ((p.dv + 15) / 16);
    return columns <= 256 ? f(std::integral_constant<int, 1>()) : f(std::integral_constant<int, 2>());
}

// LDS of a walk: K, Q, NM triangular matrices of a chunk (32 columns of all rows, then the others of the last 32), its
// columns of V and its factors; those of y; what waves exchange.  The first two twice where that fits.
template <typename E, int DK, int NM>
struct WalkLds {
    typedef typename Mat<E>::raw raw;
    typedef LdsTile<E, DK> KTile;
    typedef LdsTile<E, 32> MTile;  // of a block of 32 columns, and of V
    static constexpr int C = Mat<E>::kChunk;
    static constexpr int KS = C * KTile::kPitch, M1 = C * MTile::kPitch, MS = M1 + (C - 32) * MTile::kPitch;
    static constexpr int YP = 32 + 16 / int(sizeof(raw));  // pitch of y
    static constexpr int kBuffer = int((2 * KS + NM * MS + M1) * sizeof(raw) + kVecs * C * sizeof(float));
    static constexpr int kOut = C * YP * int(sizeof(raw));
    static constexpr int kSlots = 6, kExchange = 4 * kSlots * 1024;
    static constexpr bool kTwice = 2 * (kBuffer + kOut) + kExchange <= 160 * 1024;
    static constexpr int kBytes = (kTwice ? 2 : 1) * (kBuffer + kOut) + kExchange;
    raw *k, *q, *m, *x, *y;
    float* v;
    __device__ __forceinline__ WalkLds(char* lds, int at) {
        const int one = kTwice ? at & 1 : 0;
        k = reinterpret_cast<raw*>(lds + kExchange + one * kBuffer);
        q = k + KS;
        m = q + KS;
        x = m + NM * MS;
        v = reinterpret_cast<float*>(x + M1);
        y = reinterpret_cast<raw*>(lds + kExchange + (kTwice ? 2 : 1) * kBuffer + one * kOut);
    }
};

// ---------------------------------------------------------------------------
// operands whose depths are half a chunk's tokens: two tiles with 16-bit elements, one (half an operand) in fp32
// ---------------------------------------------------------------------------
template <typename E>
struct HalfOps {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef typename M::frag op;
    static constexpr int OT = M::kChunk / 32;  // tiles of half a chunk's tokens
    static __device__ __forceinline__ op cvt(const f32x4 (&x)[OT]) { return M::cvt(x[0], x[1]); }
    static __device__ __forceinline__ float at(const op& x, int t, int r) { return M::at(x, 4 * t + r); }
    static __device__ __forceinline__ f32x4 mma(const op& a, const op& b, f32x4 c) { return M::mma(a, b, c); }
    static __device__ __forceinline__ Two<E> two(const f32x4 (&x)[OT]) { return cls::two<E>(x[0], x[1]); }
    // Of a chunk's triangular matrix the rows of tile j of half h against the depths of half hd (h >= hd).
    template <typename T>
    static __device__ __forceinline__ op rows(const T& t, const raw* m, int m1, int h, int hd, int j) {
        return t.rows(m + (hd ? m1 : 32 * h * T::kPitch), j, 0);
    }
    // Its columns of tile j of half h against the depths of half hd (h <= hd).
    template <typename T>
    static __device__ __forceinline__ op cols(const T& t, const raw* m, int m1, int h, int hd, int j) {
        return t.cols(m + (h ? m1 : 32 * hd * T::kPitch), 0, j);
    }
    // Columns of tile j of a matrix whose rows are tokens, depths those of half hd.
    template <typename T>
    static __device__ __forceinline__ op tokens(const T& t, const raw* m, int hd, int j) {
        return t.cols(m + 32 * hd * T::kPitch, 0, j);
    }
};

template <>
struct HalfOps<ElemF32> {
    typedef Mat<ElemF32> M;
    typedef uint32_t raw;
    typedef f32x4 op;
    static constexpr int OT = 1;
    static __device__ __forceinline__ op cvt(const f32x4 (&x)[1]) { return x[0]; }
    static __device__ __forceinline__ float at(const op& x, int, int r) { return x[r]; }
    static __device__ __forceinline__ f32x4 mma(const op& a, const op& b, f32x4 c) {
#pragma unroll
        for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
        return c;
    }
    struct One { op hi, lo; };
    static __device__ __forceinline__ One two(const f32x4 (&x)[1]) { return {x[0], x[0]}; }
    template <typename T>
    static __device__ __forceinline__ op rows(const T&, const raw* m, int, int h, int hd, int) {
        return *reinterpret_cast<const f32x4*>(m + (16 * h + lane16()) * T::kPitch + 16 * hd + 4 * group4());
    }
    template <typename T>
    static __device__ __forceinline__ op cols(const T& t, const raw* m, int, int h, int hd, int) {
        return tokens(t, m, hd, h);
    }
    template <typename T>
    static __device__ __forceinline__ op tokens(const T& t, const raw* m, int hd, int j) {
        const raw* at = reinterpret_cast<const raw*>(reinterpret_cast<const char*>(m + 16 * hd * T::kPitch) + t.c[0]) + 16 * j;
        op x;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = as_float(at[k * T::kPitch]);
        return x;
    }
};

// A wave's place for what its partner reads: slots of 16 bytes to a lane.
struct Exchange {
    char *mine, *other;
    __device__ __forceinline__ Exchange(char* lds, int wave, int slots) {
        const int lane = 16 * (threadIdx.x & 63);
        mine = lds + wave * slots * 1024 + lane;
        other = lds + (wave ^ 1) * slots * 1024 + lane;
    }
    template <typename T>
    __device__ __forceinline__ void put(int slot, const T& x) const {
        static_assert(sizeof(T) == 16, "");
        *reinterpret_cast<u32x4*>(mine + slot * 1024) = __builtin_bit_cast(u32x4, x);
    }
    template <typename T>
    __device__ __forceinline__ void get(int slot, T& x) const {
        static_assert(sizeof(T) == 16, "");
        x = __builtin_bit_cast(T, *reinterpret_cast<const u32x4*>(other + slot * 1024));
    }
};

// ---------------------------------------------------------------------------
// the loading waves
// ---------------------------------------------------------------------------
// Columns of V or dY in, of y or dV out.
struct WalkColumns {
    const void* x;
    Strided3 sx;
    void* y;
    bool vec_y;
    float power;  // of X as an operand, where it is a gradient (GRADS)
};

// Chunks first, first + step, .. (n of them).
template <typename E, int DK, int NM, int TILES, bool GRADS>
__device__ __forceinline__ void walk_load(const DeltaParams& p, const WalkColumns& w, char* lds, int b, int h, int col0, int end,
                                          int first, int step, int n) {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    typedef ChunkMats<E> CM;
    typedef WalkLds<E, DK, NM> Lds;
    constexpr int C = M::kChunk, THREADS = 256;
    constexpr int64_t SZ = sizeof(raw);
    typedef TileRegs<E, C, DK, THREADS> KRegs;
    typedef TileRegs<E, C, 32, THREADS> XRegs;  // 32 columns: of a matrix, of V, of y
    static_assert(XRegs::N == 1, "");
    constexpr int LOW = (C - 32) * XRegs::PER_ROW;  // threads with a vector of the last 32 columns
    const int kh = h / (p.H / p.Hk), tid = threadIdx.x - 128 * TILES;
    const raw* K = static_cast<const raw*>(p.k) + b * p.sk.batch + kh * p.sk.head;
    const raw* Q = static_cast<const raw*>(p.q) + b * p.sq.batch + kh * p.sq.head;
    const raw* X = static_cast<const raw*>(w.x) + b * w.sx.batch + h * w.sx.head + col0;
    const int cols = p.dv - col0 < walk_cols(TILES) ? p.dv - col0 : walk_cols(TILES);
    const int xrow = tid / XRegs::PER_ROW, xcol = tid % XRegs::PER_ROW * XRegs::VE;  // a thread's vector of 32 columns
    const uint32_t ok = KRegs::offset(p.sk.token, p.dk, tid), oq = KRegs::offset(p.sq.token, p.dk, tid);
    // two chunks in flight, where LDS has two: a chunk may take less time than a load from memory
    constexpr int SETS = Lds::kTwice ? 2 : 1;
    struct Set {
        KRegs k, q;
        u32x4 m[NM], low[NM], x, v;
    } set[SETS];
    const auto fetch_keys = [&](KRegs& r, const raw* from, const Strided3& s, uint32_t at, int i) {
        const int t0 = (first + i * step) * C;
        r.load(buffer(from + t0 * s.token, (end - t0) * s.token * SZ), at, s.token);
        fence();
    };
    const auto fetch_k = [&](Set& r, int i) { fetch_keys(r.k, K, p.sk, ok, i); };
    const auto fetch_q = [&](Set& r, int i) { fetch_keys(r.q, Q, p.sq, oq, i); };
    const auto fetch_rest = [&](Set& r, int i) {
        const int c = first + i * step, t0 = c * C, left = end - t0;
        const int64_t chunk = (int64_t(b) * p.nchunk + c) * p.H + h;
        // A wait counts the loads behind the one that it is for.  So none is under a branch, or the other set's would be
        // waited for, too.
        const Buffer bm = buffer(static_cast<const raw*>(p.mats) + chunk * CM::kAll * CM::kSize);
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const uint32_t at = uint32_t((m * CM::kSize + xrow * C + xcol) * SZ);
            r.m[m] = __builtin_amdgcn_raw_buffer_load_b128(bm, int(at), 0, 0);
            if constexpr (LOW > 0)
                r.low[m] = __builtin_amdgcn_raw_buffer_load_b128(bm, int(tid < LOW ? at + uint32_t((32 * C + 32) * SZ) : kOutside), 0, 0);
        }
        const Buffer bx = buffer(X + t0 * w.sx.token, left * w.sx.token * SZ - col0 * SZ);
        r.x = __builtin_amdgcn_raw_buffer_load_b128(
            bx, int(xcol < cols ? uint32_t((xrow * w.sx.token + xcol) * SZ) : kOutside), 0, 0);
        r.v = ldg_b128(p.vecs + chunk * kVecs * C + 4 * (tid < kVecs * C / 4 ? tid : 0));
        fence();
    };
    const auto fetch = [&](Set& r, int i) {
        fetch_k(r, i);
        fetch_q(r, i);
        fetch_rest(r, i);
    };
    const auto put_keys = [&](const KRegs& r, raw* to) { r.template store<typename Lds::KTile>(to, tid); };
    const auto put_rest = [&](const Set& r, const Lds& to) {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            Lds::MTile::put(to.m + m * Lds::MS, xrow, xcol, r.m[m]);
            if (LOW > 0 && tid < LOW) Lds::MTile::put(to.m + m * Lds::MS + Lds::M1, xrow, xcol, r.low[m]);
        }
        Lds::MTile::put(to.x, xrow, xcol, GRADS ? times<E>(r.x, w.power) : r.x);
        if (tid < kVecs * C / 4) *reinterpret_cast<u32x4*>(to.v + 4 * tid) = r.v;
    };
    const int64_t row = int64_t(p.H) * p.dv;  // of a token of y
    raw* Y = static_cast<raw*>(w.y) + int64_t(b) * p.L * row + int64_t(h) * p.dv + col0;
    const auto out = [&](int i) {
        const Lds from(lds, i);
        const int t0 = (first + i * step) * C;
        const Buffer by = buffer(Y + t0 * row, int64_t(p.L - t0) * row * SZ - (int64_t(h) * p.dv + col0) * SZ);
        u32x4 x = *reinterpret_cast<const u32x4*>(from.y + xrow * Lds::YP + xcol);
        if (t0 + xrow >= end) x = u32x4{0, 0, 0, 0};  // padding
        const uint32_t to = uint32_t((xrow * row + xcol) * SZ);
        if (w.vec_y) {
            __builtin_amdgcn_raw_buffer_store_b128(x, by, int(xcol < cols ? to : kOutside), 0, 0);
        } else {
#pragma unroll
            for (int e = 0; e < XRegs::VE; ++e) {
                const uint32_t word = x[SZ == 4 ? e : e >> 1], at = xcol + e < cols ? to + uint32_t(e * SZ) : kOutside;
                if constexpr (SZ == 4) __builtin_amdgcn_raw_buffer_store_b32(word, by, int(at), 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b16(uint16_t(word >> (16 * (e & 1))), by, int(at), 0, 0);
            }
        }
    };
    const auto last = [&](int i) { return i < n ? i : n - 1; };  // past the end: loaded again, not used
    if (n > 0) {
        fetch(set[0], 0);
        if constexpr (Lds::kTwice) {
            const Lds lds0(lds, 0);
            fetch(set[1], last(1));
            put_keys(set[0].k, lds0.k);
            put_keys(set[0].q, lds0.q);
            put_rest(set[0], lds0);
            fetch(set[0], last(2));
            lds_meet();
            // While chunk i is computed the one behind it comes and y of the one before leaves, in pieces between the
            // computing waves' meetings.  A piece's registers are loaded again at once (1 x 32768 x 32 heads of 128: 891 us;
            // all loads behind the last piece: 1150).  Behind the last chunk there is one more that nobody reads.
            const auto turn = [&](Set& r, int i) {
                const Lds to(lds, i + 1);
                put_keys(r.k, to.k);
                fetch_k(r, last(i + 3));
                lds_meet();
                put_keys(r.q, to.q);
                fetch_q(r, last(i + 3));
                lds_meet();
                put_rest(r, to);
                fetch_rest(r, last(i + 3));
                lds_meet();
                if (i > 0) out(i - 1);
                lds_meet();
            };
            int i = 0;
            for (; i + 1 < n; i += 2) {  // no way from one set's turn to the same set's, for the waits' sake
                turn(set[1], i);
                turn(set[0], i + 1);
            }
            if (i < n) turn(set[1], i);
        } else {
            const Lds to(lds, 0);
            for (int i = 0; i < n; ++i) {
                lds_meet();
                if (i > 0) out(i - 1);
                put_keys(set[0].k, to.k);
                put_keys(set[0].q, to.q);
                put_rest(set[0], to);
                lds_meet();
                fetch(set[0], last(i + 1));
                lds_meet();
                lds_meet();
                lds_meet();
            }
            lds_meet();
        }
        out(n - 1);
    }
    // whole chunks of padding
    const int64_t t1 = (end + C - 1) / C * C;
    for (int64_t at = tid; at < (p.L - t1) * cols; at += THREADS) Y[(t1 + at / cols) * row + at % cols] = raw(0);
}

// The computing waves' part: f(i, lds) for every chunk that the loading waves bring, which meets three times.
template <typename Lds, typename F>
__device__ __forceinline__ void walk(char* lds, int n, F&& f) {
    if (n == 0) return;
    if constexpr (Lds::kTwice) {
        lds_meet();
        for (int i = 0; i < n; ++i) {
            f(i, Lds(lds, i));
            settle();
            lds_meet();
        }
    } else {
        for (int i = 0; i < n; ++i) {
            lds_meet();
            lds_meet();
            f(i, Lds(lds, i));
            settle();
        }
        lds_meet();
    }
}

// ---------------------------------------------------------------------------
// states in memory
// ---------------------------------------------------------------------------
// A lane's part of a state [dv, dk]: column n, keys' elements first + 16 t + 4 (l/16) + r; `of` is the state's place among
// those of all sequences and heads (and chunks).
template <int KT>
__device__ __forceinline__ void load_state(f32x4 (&S)[KT], const float* from, int64_t of, int n, int first, const DeltaParams& p) {
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] = f32x4{0, 0, 0, 0};
    if (from) {
        const Buffer b = buffer(from + of * p.dv * p.dk, int64_t(p.dv) * p.dk * 4);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const int d = first + 16 * t + 4 * group4();
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
// The same for the gradients: rows of kpitch elements.  Past the caches, as all of it is written before any of it is read
// (4 x 2048 x 16 heads of 128: the walks 128 and 135 -> 124 and 129 us, the gradients' kernel, which reads it once, 163 -> 152).
template <int KT>
__device__ __forceinline__ void keep_state(const f32x4 (&S)[KT], float* to, int64_t of, int n, int first, const DeltaParams& p) {
    const Buffer b = buffer(to + of * p.dv * p.kpitch, int64_t(p.dv) * p.kpitch * 4);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const int d = first + 16 * t + 4 * group4();
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[t]), b,
                                               int(d < p.kpitch && n < p.dv ? uint32_t(n * p.kpitch + d) * 4 : kOutside), 0, kStream);
    }
}
template <int KT>
__device__ __forceinline__ void store_state(const f32x4 (&S)[KT], float* to, int64_t of, int n, int first, const DeltaParams& p) {
    const Buffer b = buffer(to + of * p.dv * p.dk, int64_t(p.dv) * p.dk * 4);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const int d = first + 16 * t + 4 * group4();
        const uint32_t at = uint32_t(n * p.dk + d) * 4;
        if (p.dk % 4 == 0) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[t]), b, int(d < p.dk && n < p.dv ? at : kOutside), 0, 0);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) store_one<ElemF32>(b, d + r < p.dk && n < p.dv ? at + 4 * r : kOutside, S[t][r]);
        }
    }
}
// A column's values of half h of the chunk's tokens: [dv, C].
template <int C>
__device__ __forceinline__ void store_tokens(const f32x4 (&x)[C / 32], float* to, int64_t chunk, int n, int h, const DeltaParams& p) {
    const Buffer b = buffer(to + chunk * p.dv * C, int64_t(p.dv) * C * 4);
#pragma unroll
    for (int t = 0; t < C / 32; ++t)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x[t]), b,
                                               int(n < p.dv ? uint32_t(n * C + C / 2 * h + 16 * t + 4 * group4()) * 4 : kOutside), 0, kStream);
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
