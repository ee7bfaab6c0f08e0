// Device helpers of the gated delta rule's kernels: operands of the matrix
// instructions for three element types, and the launch parameters.
//
// Every product is made of 16x16 tiles with a depth of 32.  Lane l holds of the
// left operand the row l%16 and of the right operand the column l%16, and of
// both the depths 16 (j/4) + 4 (l/16) + j%4, j = 0..7: the order in which two
// result tiles, one below the other, lie in the lanes (rows 4 (l/16) + r of
// column l%16).  So a result goes on as the right operand of the next product
// without leaving its lanes: the states, the corrections and the gradients of a
// chunk never pass through LDS.
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
    static constexpr int kPad = 8;        // elements behind each row in LDS

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
    // Four elements of a row from k on, and the four 16 further on.
    static __device__ __forceinline__ frag rows(const raw* p) {
        const u32x2 a = *reinterpret_cast<const u32x2*>(p + 4 * group4());
        const u32x2 b = *reinterpret_cast<const u32x2*>(p + 16 + 4 * group4());
        return frag{a[0], a[1], b[0], b[1]};
    }
    // The same of a column: depths run over the rows of a matrix in LDS from p on; p at the first of 16 columns.
    static __device__ __forceinline__ frag cols(const raw* p, int pitch) {
        typedef __attribute__((address_space(3))) s16x4* lp;
        const raw* at = p + (4 * group4() + (lane16() >> 2)) * pitch + 4 * (lane16() & 3);
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at)));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at + 16 * pitch)));
        return frag{a[0], a[1], b[0], b[1]};
    }
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
    static constexpr int kPad = 4;
    static __device__ __forceinline__ frag cvt(const f32x4& a, const f32x4& b) { return frag{a, b}; }
    static __device__ __forceinline__ frag rows(const raw* p) {
        return frag{*reinterpret_cast<const f32x4*>(p + 4 * group4()),
                    *reinterpret_cast<const f32x4*>(p + 16 + 4 * group4())};
    }
    static __device__ __forceinline__ frag cols(const raw* p, int pitch) {
        const raw* at = p + 4 * group4() * pitch + lane16();
        frag f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            f.a[r] = as_float(at[r * pitch]);
            f.b[r] = as_float(at[(16 + r) * pitch]);
        }
        return f;
    }
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
// computed x computed: the product of the two small parts, at most 2^-16 of the whole (bf16), is left out
template <typename E>
__device__ __forceinline__ f32x4 mma3(const Two<E>& a, const Two<E>& b, f32x4 c) {
    if constexpr (Mat<E>::kSplit) {
        c = Mat<E>::mma(a.lo, b.hi, c);
        c = Mat<E>::mma(a.hi, b.lo, c);
    }
    return Mat<E>::mma(a.hi, b.hi, c);
}

// ---------------------------------------------------------------------------
// launch parameters and tiles
// ---------------------------------------------------------------------------
struct Strided3 { int64_t batch, token, head; };

struct DeltaParams {
    const void *q, *k, *v, *dy;
    const float *g, *beta, *h0, *dh_last;
    const int32_t* seqlens;
    void *y, *dq, *dk_, *dv_;
    float *h_last, *dg, *dbeta, *dh0;
    float* states;   // [batch, chunks, heads, dk, dv]: the state before each chunk (NULL = not kept)
    float* fixes;    // [batch, L, heads, dv]: N, the corrections (NULL = not kept)
    void* mats;      // per (batch, chunk, head): (I + A)^-1 - I and D QK^T, in one part or two
    float* vecs;     // per (batch, chunk, head): e^gamma, e^(gamma_C - gamma), beta
    float* dstates;  // as states: the gradient of the state behind each chunk
    float* z;        // as fixes: (I + A)^-T dN
    float *part_q, *part_k;  // [batch, L, heads, dk], where key heads are shared
    Strided3 sq, sk, sv, sdy;
    int64_t g_batch, g_token, b_batch, b_token;
    int batch, L, Hk, H, dk, dv, nchunk;
    float scale;
    uint8_t vec_q, vec_k, vec_v, vec_dy;  // rows of whole 16-byte vectors
    uint8_t vec_out;                      // dq and dk start on 16 bytes
};

// Matrices of a chunk in `mats`: T hi, T lo, P hi, P lo (16-bit), T, P (fp32).
template <typename E>
struct ChunkMats {
    typedef Mat<E> M;
    static constexpr int kSize = M::kChunk * M::kChunk;
    static constexpr int kParts = M::kSplit ? 2 : 1;
    static constexpr int kAll = 2 * kParts;
    static constexpr int kPitch = M::kChunk + M::kPad;
};

// A 16-byte vector of a row: elements col.. of `dim` (zeros past it).
template <typename E>
__device__ __forceinline__ u32x4 load_vec(const typename E::raw* row, int col, int dim, bool vec) {
    constexpr int VE = 16 / sizeof(typename E::raw);
    if (vec) return col < dim ? ldg_b128(row + col) : u32x4{0, 0, 0, 0};
    u32x4 v{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        if (col + e >= dim) continue;
        const uint32_t w = row[col + e];
        if constexpr (VE == 4) v[e] = w;
        else v[e >> 1] |= w << (16 * (e & 1));
    }
    return v;
}

// A tile of ROWS tokens of a [.., dim] matrix, padded to DIM columns, held by the threads of a workgroup between
// memory and LDS.
template <typename E, int ROWS, int DIM, int THREADS>
struct TileRegs {
    static constexpr int VE = 16 / sizeof(typename E::raw);
    static constexpr int PER_ROW = DIM / VE;
    static constexpr int N = ROWS * PER_ROW / THREADS;
    static_assert(ROWS * PER_ROW % THREADS == 0, "");
    u32x4 r[N];

    __device__ __forceinline__ void load(const typename E::raw* base, int64_t token, int t0, int end, int dim, bool vec) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = threadIdx.x + n * THREADS, row = at / PER_ROW, col = at % PER_ROW * VE;
            r[n] = t0 + row < end ? load_vec<E>(base + (t0 + row) * token, col, dim, vec) : u32x4{0, 0, 0, 0};
        }
    }
    __device__ __forceinline__ void store(typename E::raw* lds, int pitch) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = threadIdx.x + n * THREADS, row = at / PER_ROW, col = at % PER_ROW * VE;
            *reinterpret_cast<u32x4*>(lds + row * pitch + col) = r[n];
        }
    }
};

// Four values of a row: elements col.. of `dim` (zeros past it).
template <typename E>
__device__ __forceinline__ f32x4 load4(const typename E::raw* row, int col, int dim, bool vec) {
    f32x4 v{0, 0, 0, 0};
    if (vec) {
        if (col >= dim) return v;
        if constexpr (sizeof(typename E::raw) == 4) {
            return *reinterpret_cast<const f32x4*>(row + col);
        } else {
            const u32x2 w = *reinterpret_cast<const u32x2*>(row + col);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t x = w[e >> 1];
                v[e] = Mat<E>::part(x, e & 1);
            }
            return v;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < dim) v[e] = E::get(row[col + e]);
    return v;
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

// Decays between the tokens of a chunk, from its logarithms g (in LDS): calls f(t, d) for the tiles t = w..0 of
// 16 tokens, where d[r] = e^(g_{j+1} + .. + g_i) for the lane's token i = 16 w + l%16 and j = 16 t + 4 (l/16) + r
// (of t = w only where j <= i is d of use).  All are exponentials of sums of g between the two tokens, never of
// differences of running sums: terms of one sign, so nothing cancels, and g = -infinity gives exactly 0.
// Returns the sum of g up to i.
template <int NT, typename F>
__device__ __forceinline__ float for_decays(const float* sG, int w, F&& f) {
    const int l16 = lane16(), g4 = group4();
    float pre = 0.0f, mid = 0.0f;  // of i's own tile up to i; of the tiles between j's and i's
#pragma unroll
    for (int l = 0; l < 16; ++l) pre += l <= l16 ? sG[16 * w + l] : 0.0f;
#pragma unroll
    for (int t = NT - 1; t >= 0; --t) {
        if (t > w) continue;
        f32x4 s{0, 0, 0, 0};
        float whole = 0.0f;
#pragma unroll
        for (int l = 0; l < 16; ++l) {
            const float gl = sG[16 * t + l];
            whole += gl;
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] += l > 4 * g4 + r && (t < w || l <= l16) ? gl : 0.0f;
        }
        f32x4 d;
#pragma unroll
        for (int r = 0; r < 4; ++r) d[r] = fexp(t < w ? s[r] + mid + pre : s[r]);
        f(t, d);
        if (t < w) mid += whole;
    }
    return mid + pre;
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
