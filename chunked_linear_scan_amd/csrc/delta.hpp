// Device helpers of the gated delta rule's kernels: operands of the matrix
// instructions for three element types, and the launch parameters.
//
// Every product is made of 16x16 tiles with a depth of 32.  Lane l holds of the
// left operand the row l%16 and of the right operand the column l%16, and of
// both the depths 16 (j/4) + 4 (l/16) + j%4, j = 0..7: the order in which two
// result tiles, one below the other, lie in the lanes (rows 4 (l/16) + r of
// column l%16).  So a result goes on as the right operand of the next product
// without leaving its lanes: in the walks LDS only has what waves that share
// columns exchange of them, and states stay in registers.
#pragma once

#include <type_traits>

#include "../../include/gated_delta.h"
#include "selective.hpp"

namespace cls {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int lane16() { return threadIdx.x & 15; }
__device__ __forceinline__ int group4() { return (threadIdx.x >> 4) & 3; }

template <typename E>
struct Mat;

template <typename E>
struct Mat16 {
    typedef typename E::raw raw;
    typedef u32x4 frag;
    static constexpr int kChunk = 64;
    static constexpr bool kSplit = true;  // computed operands are sums of two numbers

    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        if constexpr (std::is_same_v<E, ElemBF16>) {
            return pack_bf16x2(a, b);
        } else {
            typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
            f16x2 v;
            v[0] = (_Float16)a;
            v[1] = (_Float16)b;
            return __builtin_bit_cast(uint32_t, v);
        }
    }
    static __device__ __forceinline__ frag cvt(const f32x4& a, const f32x4& b) {
        return frag{pack(a[0], a[1]), pack(a[2], a[3]), pack(b[0], b[1]), pack(b[2], b[3])};
    }
    static __device__ __forceinline__ float part(uint32_t w, int hi) { return E::get(raw(hi ? w >> 16 : w & 0xffffu)); }
    static __device__ __forceinline__ float at(const frag& f, int j) { const uint32_t w = f[j >> 1]; return part(w, j & 1); }
};

template <>
struct Mat<ElemBF16> : Mat16<ElemBF16> {
    static __device__ __forceinline__ f32x4 mma(const frag& a, const frag& b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    }
};

template <>
struct Mat<ElemF16> : Mat16<ElemF16> {
    static __device__ __forceinline__ f32x4 mma(const frag& a, const frag& b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
    }
};

// fp32 elements: eight products of depth 4 with the same depths in the same lanes.
template <>
struct Mat<ElemF32> {
    typedef uint32_t raw;
    struct frag { f32x4 a, b; };
    static constexpr int kChunk = 32;
    static constexpr bool kSplit = false;
    static __device__ __forceinline__ frag cvt(const f32x4& a, const f32x4& b) { return frag{a, b}; }
    static __device__ __forceinline__ float at(const frag& f, int j) { return j < 4 ? f.a[j & 3] : f.b[j & 3]; }
    static __device__ __forceinline__ f32x4 mma(const frag& a, const frag& b, f32x4 c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[j], b.a[j], c, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[j], b.b[j], c, 0, 0, 0);
        return c;
    }
};

// A computed operand: with 16-bit elements x = hi + lo, hi the nearest number of
// the type and lo that of what is left, which leaves at most 2^-16 (bf16) of x; in fp32 x.
template <typename E>
struct Two {
    typename Mat<E>::frag hi, lo;
};

template <typename E>
__device__ __forceinline__ Two<E> two(const f32x4& a, const f32x4& b) {
    typedef Mat<E> M;
    Two<E> t;
    t.hi = M::cvt(a, b);
    if constexpr (M::kSplit) {
        // what is left is that of these very bits: the compiler may otherwise round a product to hi a second time, in
        // one step instead of two, and near a tie the two differ by a unit
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t bits = t.hi[w];
            asm("" : "+v"(bits));
            t.hi[w] = bits;
        }
        f32x4 ra, rb;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            ra[r] = a[r] - M::at(t.hi, r);
            rb[r] = b[r] - M::at(t.hi, 4 + r);
        }
        t.lo = M::cvt(ra, rb);
    }
    return t;
}

// exact x computed
template <typename E>
__device__ __forceinline__ f32x4 mma2(const typename Mat<E>::frag& a, const Two<E>& b, f32x4 c) {
    if constexpr (Mat<E>::kSplit) c = Mat<E>::mma(a, b.lo, c);
    return Mat<E>::mma(a, b.hi, c);
}
// computed x exact
template <typename E>
__device__ __forceinline__ f32x4 mma2(const Two<E>& a, const typename Mat<E>::frag& b, f32x4 c) {
    if constexpr (Mat<E>::kSplit) c = Mat<E>::mma(a.lo, b, c);
    return Mat<E>::mma(a.hi, b, c);
}
// Whether products of two computed operands have that of the small parts, at most 2^-16 of the whole (bf16).  With keys of
// few elements roundings average out less (of 8: dg up to 1.1e-5 off without it, 8.6e-6 with it; of 64: 5e-6).
constexpr bool small_parts(int dk) { return dk <= 64; }

// computed x computed
template <typename E, bool SMALL>
__device__ __forceinline__ f32x4 mma3(const Two<E>& a, const Two<E>& b, f32x4 c) {
    if constexpr (Mat<E>::kSplit) {
        if constexpr (SMALL) c = Mat<E>::mma(a.lo, b.lo, c);
        c = Mat<E>::mma(a.lo, b.hi, c);
        c = Mat<E>::mma(a.hi, b.lo, c);
    }
    return Mat<E>::mma(a.hi, b.hi, c);
}

// ---------------------------------------------------------------------------
// launch parameters and tiles
// ---------------------------------------------------------------------------
struct Strided3 { int64_t batch, token, head; };
constexpr int64_t kDeltaMaxToken = int64_t(1) << 23;  // elements from a token to the next

// q, k, v and dy have rows of whole 16-byte vectors: the caller's or, where those are off whole vectors or have rows that
// overlap or lie further apart than kDeltaMaxToken, copies with zeros behind a row's end.
struct DeltaParams {
    const void *q, *k, *v, *dy;
    const float *g, *beta, *h0, *dh_last;
    const int32_t* seqlens;
    void *y, *dq, *dk_, *dv_;
    float *h_last, *dg, *dbeta, *dh0;
    float* states;   // [batch, chunks, heads, dv, kpitch]: the state before each chunk (NULL = not kept)
    float* fixes;    // [batch, chunks, heads, dv, chunk]: N, the corrections (NULL = not kept)
    void* mats;      // per (batch, chunk, head): (I + A)^-1 - I and D QK^T, each in its parts
    float* vecs;     // per (batch, chunk, head): kVecs factors of each token
    float* dstates;  // as states: the gradient of the state behind each chunk, times grad_power
    float* z;        // as fixes: (I + A)^-T dN, likewise
    float *part_q, *part_k;  // [batch, L, heads, dk], where key heads are shared
    float* sizes;    // [batch, heads, 2, kSizes], the first nsize of each: largest values of parts of dY and of dh (fp16)
    Strided3 sq, sk, sv, sdy;
    int64_t g_batch, g_token, b_batch, b_token;
    int batch, L, Hk, H, dk, dv, nchunk;
    int nsize;
    int kpitch;  // of the kept states' rows: dk to whole vectors
    float scale;
    uint8_t vec_out;  // y or dv has rows of whole 16-byte vectors
    uint8_t vec_dqk;  // dq and dk start on 16 bytes
};

// Matrices of a chunk in `mats`: T hi, T lo, P hi, P lo (16-bit), T, P (fp32).
template <typename E>
struct ChunkMats {
    typedef Mat<E> M;
    static constexpr int kSize = M::kChunk * M::kChunk;
    static constexpr int kParts = M::kSplit ? 2 : 1;
    static constexpr int kAll = 2 * kParts;
};

// ---------------------------------------------------------------------------
// powers of two in front of fp16 operands
// ---------------------------------------------------------------------------
// Two fp16 numbers hold 22 bits of what is 2^-3 and more, and of less what is left above 2^-25; past 65504 they hold
// nothing.  Gradients are as large as the loss makes them, often far below that, so the backward pass multiplies a head's
// gradients of states, corrections and outputs by one power of two that brings the largest of scale dY and dh_final to
// 4..8, 2^13 below the type's end, and divides what it writes by it: exactly, so gradients of 2^n dy are 2^n times those
// of dy.  (Without it dg of dy about 1e-3 was 1.5e-4 off, of 1e-5 1.6e-2, and dh_final past 65504 gave NaN.)  dY itself
// goes in times another, at least 1, as products of subnormal operands lose bits where the unit adds them up (1e-8 of the
// sums for dy of 2^-14, 7e-7 for 2^-18).
template <typename E>
constexpr bool kSized = std::is_same_v<E, ElemF16>;
constexpr int kSizes = 64;  // at most, parts of a head that delta_size_kernel takes apart

// The larger of m and |x|; values that are not finite do not count.
__device__ __forceinline__ float larger(float m, float x) {
    const float a = fabsf(x);
    return a > m && a < __builtin_inff() ? a : m;
}
__device__ __forceinline__ float wave_max(float m) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    return m;
}

struct Power { float up, down; };
// 2^k, which brings m to 2^to up to twice that (k at most `most`), and 2^-k.
__device__ __forceinline__ Power power_to(float m, int to, int most = 126) {
    int k = to + 127 - int(as_uint(m) >> 23);
    k = m == 0.0f ? 0 : k > most ? most : k < -126 ? -126 : k;
    return {as_float(uint32_t(127 + k) << 23), as_float(uint32_t(127 - k) << 23)};
}
// Those of a head's gradients: of = batch * heads + head.
struct GradPower {
    float up, down;  // of all gradients
    float dy;        // of dY as an operand: up to 2^15, which is in the type's range and takes its smallest number to 2^-9
    float ratio;     // up / dy, of products with dY
};
template <typename E>
__device__ __forceinline__ GradPower grad_power(const DeltaParams& p, int64_t of) {
    if constexpr (kSized<E>) {
        const float* sizes = p.sizes + of * 2 * kSizes;
        const int lane = threadIdx.x & 63;
        const float dy = wave_max(lane < p.nsize ? sizes[lane] : 0.0f);
        const float dh = wave_max(lane < p.nsize ? sizes[kSizes + lane] : 0.0f);
        const Power all = power_to(larger(dh, dy * p.scale), 2), y = power_to(fminf(dy, 4.0f), 2, 15);
        return {all.up, all.down, y.up, all.up * y.down};
    }
    return {1.0f, 1.0f, 1.0f, 1.0f};
}
// Eight elements times such a power.
template <typename E>
__device__ __forceinline__ u32x4 times(const u32x4& x, float power) {
    if constexpr (kSized<E>) return __builtin_bit_cast(u32x4, __builtin_bit_cast(f16x8, x) * (_Float16)power);
    return x;
}

// Factors of a token in `vecs`, each for all of a chunk's: scale e^gamma, e^(gamma_C - gamma), beta, beta e^gamma, e^gamma.
enum { kRead, kWrite, kBeta, kBetaStart, kStart, kVecs };

// ---------------------------------------------------------------------------
// matrices in LDS
// ---------------------------------------------------------------------------
// With 16-bit elements a row's quads of four elements lie in the operands' order: of each 32 elements piece
// g (16 bytes) holds quads g and 4 + g, the depths of lane group g, so an operand of rows is one read.  Pieces are exchanged by an
// exclusive or with a number of the row instead of padding: reads of 16 rows touch every bank once, transposing
// reads of 16 columns (half a piece of 8 rows each) twice.  (With the quads in their natural order those are free of
// conflicts, too, but an operand of rows is two reads, which the compiler joins across tiles and takes apart by moves.)
// fp32 rows are padded by 16 bytes.  An object holds a lane's offsets, which do not change from tile to tile.
template <typename E, int DIM>
struct LdsTile {
    typedef Mat<E> M;
    typedef typename M::raw raw;
    static constexpr bool kSwap = M::kSplit;
    static constexpr int kPitch = DIM + (kSwap ? 0 : 4);
    static constexpr int kSpan = DIM < 128 ? DIM : 128;  // columns that the exchange covers
    static constexpr int kRows = kSwap ? kSpan / 32 : 1;
    uint32_t r[kRows], c[kRows];  // bytes

    // A number of the row: its upper bits differ among four rows, its lower two among every fourth, in an order that
    // keeps the 16 lanes which a 16-byte read serves at a time apart (0-3, 12-15 and 20-27 of 32, so rows of two lane groups).
    static __device__ __forceinline__ int swap(int row) {
        const int x = (row >> 2) & 3, low = (((x ^ (x >> 1)) & 1) << 1) + (x >> 1);
        return kSpan == 32 ? low : 4 * (kSpan == 64 ? (row >> 1) & 1 : row & 3) + low;
    }
    // Element offset of four elements (col a multiple of 4).
    static __device__ __forceinline__ int quad(int row, int col) {
        if constexpr (kSwap) {
            const int piece = (col >> 5) * 4 + ((col >> 2) & 3);
            return row * kPitch + (piece ^ swap(row)) * 8 + ((col >> 4) & 1) * 4;
        }
        return row * kPitch + col;
    }
    // A 16-byte vector of a row in memory.
    static __device__ __forceinline__ void put(raw* m, int row, int col, const u32x4& v) {
        if constexpr (kSwap) {
            // the rows that share banks start with different halves
            const bool odd = kSpan == 32 ? row & 4 : kSpan == 64 ? row & 2 : row & 1;
            const u32x2 a{v[0], v[1]}, b{v[2], v[3]};
            *reinterpret_cast<u32x2*>(m + quad(row, col + (odd ? 4 : 0))) = odd ? b : a;
            *reinterpret_cast<u32x2*>(m + quad(row, col + (odd ? 0 : 4))) = odd ? a : b;
        } else {
            *reinterpret_cast<u32x4*>(m + quad(row, col)) = v;
        }
    }
    // Steps and tiles count from column `first` on, a multiple of 32 (of kSpan where that is less than what is used;
    // of 16 for the tile that starts there).
    __device__ __forceinline__ explicit LdsTile(int first = 0) {
        const int l16 = lane16(), g = group4();
        if constexpr (kSwap) {
#pragma unroll
            for (int n = 0; n < kRows; ++n) r[n] = quad(l16, (first + 32 * n) % DIM + 4 * g) * sizeof(raw);
#pragma unroll
            for (int n = 0; n < kRows; ++n) c[n] = quad(4 * g + (l16 >> 2), (first + 32 * n) % DIM + 4 * (l16 & 3)) * sizeof(raw);
        } else {
            r[0] = (l16 * kPitch + first + 4 * g) * sizeof(raw);
            c[0] = (4 * g * kPitch + first + l16) * sizeof(raw);
        }
    }
    // Operand of 16 rows from 16 t on, depths 32 s.. of them.
    __device__ __forceinline__ typename M::frag rows(const raw* m, int t, int s) const {
        const char* p = reinterpret_cast<const char*>(m + 16 * t * kPitch);
        if constexpr (kSwap) {
            p += 32 * s / kSpan * kSpan * sizeof(raw);
            return *reinterpret_cast<const u32x4*>(p + r[s % kRows]);
        } else {
            p += r[0] + 32 * s * sizeof(raw);
            return typename M::frag{*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 16 * sizeof(raw))};
        }
    }
    // Operand of 16 columns from 16 t on, depths the rows 32 s..
    __device__ __forceinline__ typename M::frag cols(const raw* m, int s, int t) const {
        const char* p = reinterpret_cast<const char*>(m + 32 * s * kPitch);
        if constexpr (kSwap) {
            typedef __attribute__((address_space(3))) s16x4* lp;
            p += 16 * t / kSpan * kSpan * sizeof(raw) + c[t / 2 % kRows] + t % 2 * 4 * sizeof(raw);
            const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(p)));
            const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(p + 16 * kPitch * sizeof(raw))));
            return u32x4{a[0], a[1], b[0], b[1]};
        } else {
            const raw* at = reinterpret_cast<const raw*>(p + c[0]) + 16 * t;
            typename M::frag f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f.a[k] = as_float(at[k * kPitch]);
                f.b[k] = as_float(at[(16 + k) * kPitch]);
            }
            return f;
        }
    }
};

// Workgroup barrier for LDS traffic only: the wave's LDS operations are complete, then all waves meet.  Loads and
// stores of memory stay in flight across it.
__device__ __forceinline__ void lds_meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Nothing is scheduled across it.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// At the end of a loop that carries results of matrix products: they are all written before it goes on or ends.  The
// compiler (AMD clang 22.0.0git of ROCm 7.2.0) left out the wait states on a loop's way out: copies of a result
// (v_mov_b64) stood there two instructions behind its product, which needs 8 (16-bit) or 10 (fp32) between them.
// Within a block, and on the way back to a loop's start, it has them.
__device__ __forceinline__ void settle() {
    fence();
    asm volatile("s_nop 15");
    fence();
}

// ---------------------------------------------------------------------------
// matrices in memory: buffers of up to 2^31 bytes from a row on, where what lies outside reads as zeros and is not
// written.  Strides are bounded by kDeltaMaxToken, so that the rows of a chunk lie within.
// ---------------------------------------------------------------------------
constexpr uint32_t kOutside = 0x80000000u;
constexpr int kStream = 2;  // of a load or store: not to be kept in the caches (nt)
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer(const void* p, int64_t bytes = kOutside) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes < int64_t(kOutside) ? int(bytes) : int(kOutside),
                                             0x00020000);
}

// A tile of ROWS tokens of a matrix with whole 16-byte vectors in its rows, padded to DIM columns, held by THREADS
// threads between memory and LDS.
template <typename E, int ROWS, int DIM, int THREADS>
struct TileRegs {
    typedef typename E::raw raw;
    static constexpr int VE = 16 / int(sizeof(raw)), PER_ROW = DIM / VE, STEP = THREADS / PER_ROW, N = ROWS / STEP;
    static_assert(THREADS % PER_ROW == 0 && ROWS % STEP == 0, "");
    u32x4 r[N];

    // The offset of a thread's first vector, for rows `pitch` elements apart of `dim` columns.
    static __device__ __forceinline__ uint32_t offset(int64_t pitch, int dim, int tid) {
        const int row = tid / PER_ROW, col = tid % PER_ROW * VE;
        return col < dim ? uint32_t((row * pitch + col) * sizeof(raw)) : kOutside;
    }
    __device__ __forceinline__ void load(Buffer b, uint32_t offset, int64_t pitch) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            r[n] = __builtin_amdgcn_raw_buffer_load_b128(b, int(offset + uint32_t(n * STEP * pitch * sizeof(raw))), 0, 0);
    }
    template <typename T>
    __device__ __forceinline__ void store(raw* lds, int tid) const {
        const int row = tid / PER_ROW, col = tid % PER_ROW * VE;
#pragma unroll
        for (int n = 0; n < N; ++n) T::put(lds, row + n * STEP, col, r[n]);
    }
};

// One element of a result tile's place.
template <typename E>
__device__ __forceinline__ typename E::raw load_one(Buffer b, uint32_t offset) {
    if constexpr (sizeof(typename E::raw) == 4) return __builtin_amdgcn_raw_buffer_load_b32(b, int(offset), 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b16(b, int(offset), 0, 0);
}
template <typename E>
__device__ __forceinline__ void store_one(Buffer b, uint32_t offset, float v) {
    if constexpr (sizeof(typename E::raw) == 4) __builtin_amdgcn_raw_buffer_store_b32(as_uint(v), b, int(offset), 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b16(E::put(v), b, int(offset), 0, 0);
}

// The lane's part of an operand of rows in memory: depths col.. of `dim`, of the row at byte offset `row`.
template <typename E>
__device__ __forceinline__ typename Mat<E>::frag load_frag(Buffer b, uint32_t row, int col, int dim) {
    constexpr int SZ = sizeof(typename E::raw);
    const int d = col + 4 * group4();
    const int lo = int(d < dim ? row + d * SZ : kOutside), hi = int(d + 16 < dim ? row + (d + 16) * SZ : kOutside);
    if constexpr (SZ == 4) {
        return {__builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lo, 0, 0)),
                __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, hi, 0, 0))};
    } else {
        const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(b, lo, 0, 0), y = __builtin_amdgcn_raw_buffer_load_b64(b, hi, 0, 0);
        return u32x4{x[0], x[1], y[0], y[1]};
    }
}

// Four adjacent elements.
template <typename E>
__device__ __forceinline__ f32x4 load4(const typename E::raw* p) {
    if constexpr (sizeof(typename E::raw) == 4) {
        return *reinterpret_cast<const f32x4*>(p);
    } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t x = w[e >> 1];
            v[e] = Mat<E>::part(x, e & 1);
        }
        return v;
    }
}

// Four adjacent computed values as an operand's parts, `lo` elements after the first for the small ones.
template <typename E>
__device__ __forceinline__ void put4(typename E::raw* p, int lo, const f32x4& v) {
    const Two<E> t = two<E>(v, v);
    if constexpr (Mat<E>::kSplit) {
        *reinterpret_cast<u32x2*>(p) = u32x2{t.hi[0], t.hi[1]};
        if (lo) *reinterpret_cast<u32x2*>(p + lo) = u32x2{t.lo[0], t.lo[1]};
    } else {
        *reinterpret_cast<f32x4*>(p) = t.hi.a;
    }
}

// Sums over 16 adjacent lanes (a row of the data-parallel primitives): inclusive from the row's start, and of those
// behind a lane.
template <int CTRL>
__device__ __forceinline__ float row_move(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_prefix(float v) {
    v += row_move<0x111>(v);
    v += row_move<0x112>(v);
    v += row_move<0x114>(v);
    return v + row_move<0x118>(v);
}
__device__ __forceinline__ float row_behind(float v) {
    v = row_move<0x101>(v);
    v += row_move<0x101>(v);
    v += row_move<0x102>(v);
    v += row_move<0x104>(v);
    return v + row_move<0x108>(v);
}
// The sum of the row, in all of its lanes.
__device__ __forceinline__ float row_total(float v) {
    v += row_move<0x121>(v);
    v += row_move<0x122>(v);
    v += row_move<0x124>(v);
    return v + row_move<0x128>(v);
}

// Decays between the tokens of a chunk, all exponentials of sums of g between the two tokens, never of differences
// of running sums: terms of one sign, so nothing cancels, and g = -infinity gives exactly 0.  In LDS: g, and of each
// token the sum of its tile of 16 up to it, that of its tile behind it, and the tiles' sums.
template <int C>
struct Decays {
    static constexpr int NT = C / 16, kFloats = 3 * C + 16;
    // By the first C threads.
    static __device__ __forceinline__ void put(float* s, float g) {
        const int i = threadIdx.x;
        const float to = row_prefix(g);
        s[i] = g;
        s[C + i] = to;
        s[2 * C + i] = row_behind(g);
        if ((i & 15) == 15) s[3 * C + (i >> 4)] = to;
    }
    // Calls f(t, d) for the tiles t = w..0, where d[r] = e^(g_{j+1} + .. + g_i) for the lane's token i = 16 w + l%16 and
    // j = 16 t + 4 (l/16) + r (of t = w only where j <= i is d of use).
    template <typename F>
    static __device__ __forceinline__ void each(const float* s, int w, F&& f) {
        const int l16 = lane16(), g4 = group4();
        const float pre = s[C + 16 * w + l16];
        {
            f32x4 g[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) g[q] = *reinterpret_cast<const f32x4*>(s + 16 * w + 4 * q);
            float base = 0.0f;  // of the tokens behind the lane's four
            f32x4 own = g[0];
#pragma unroll
            for (int q = 1; q < 4; ++q) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    base += q > g4 && 4 * q + r <= l16 ? g[q][r] : 0.0f;
                    own[r] = q == g4 ? g[q][r] : own[r];
                }
            }
            f32x4 x;
            x[3] = base;
#pragma unroll
            for (int r = 2; r >= 0; --r) x[r] = x[r + 1] + (4 * g4 + r + 1 <= l16 ? own[r + 1] : 0.0f);
            f32x4 d;
#pragma unroll
            for (int r = 0; r < 4; ++r) d[r] = fexp(x[r]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (t == w) f(t, d);
        }
        float mid = pre;  // and of the tiles between
#pragma unroll
        for (int t = NT - 2; t >= 0; --t) {
            if (t >= w) continue;
            const f32x4 behind = *reinterpret_cast<const f32x4*>(s + 2 * C + 16 * t + 4 * g4);
            f32x4 d;
#pragma unroll
            for (int r = 0; r < 4; ++r) d[r] = fexp(behind[r] + mid);
            f(t, d);
            mid += s[3 * C + t];
        }
    }
    // e^ of the sum up to the lane's token, and of that behind it.
    static __device__ __forceinline__ float start(const float* s, int w) {
        float v = s[C + 16 * w + lane16()];
        for (int t = 0; t < w; ++t) v += s[3 * C + t];
        return fexp(v);
    }
    static __device__ __forceinline__ float behind(const float* s, int w) {
        float v = s[2 * C + 16 * w + lane16()];
        for (int t = w + 1; t < NT; ++t) v += s[3 * C + t];
        return fexp(v);
    }
};

// A workgroup's unit (of n) and its place in it (of `per`): workgroups go to the eight dies in turn, so those of a
// unit, which read the same rows, are eight apart and share a die's L2.
struct UnitPart { int unit, part; };
__device__ __forceinline__ UnitPart unit_part(int n, int per) {
    const int group = blockIdx.x / (8 * per), r = blockIdx.x % (8 * per);
    const int units = n - 8 * group < 8 ? n - 8 * group : 8;
    return {8 * group + r % units, r / units};
}

// Calls f with the element type and the padded size of a key (its place in LDS and registers).
template <typename F>
int by_type(int dtype, int dk, F&& f) {
    const auto sized = [&](auto e) {
        if (dk <= 64) return f(e, std::integral_constant<int, 64>());
        if (dk <= 128) return f(e, std::integral_constant<int, 128>());
        return f(e, std::integral_constant<int, 256>());
    };
    if (dtype == SSD_F32) return sized(ElemF32());
    return dtype == SSD_BF16 ? sized(ElemBF16()) : sized(ElemF16());
}

}  // namespace cls
