// Device helpers of the selective scan, the short convolution and the state
// cache: activation elements of three types, and the scalar functions that
// their formulas share.
#pragma once

#include "common.hpp"

namespace cls {

// Activation elements: raw bits in memory, fp32 in registers.
struct ElemF32 {
    typedef uint32_t raw;
    static __device__ __forceinline__ float get(raw v) { return as_float(v); }
    static __device__ __forceinline__ raw put(float v) { return as_uint(v); }
};
struct ElemBF16 {
    typedef uint16_t raw;
    static __device__ __forceinline__ float get(raw v) { return as_float(uint32_t(v) << 16); }
    static __device__ __forceinline__ raw put(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
struct ElemF16 {
    typedef uint16_t raw;
    static __device__ __forceinline__ float get(raw v) { return float(__builtin_bit_cast(_Float16, v)); }
    static __device__ __forceinline__ raw put(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float fexp(float x) { return fexp2(x * kLog2e); }

// 1 / (1 + exp(-x)): exp overflows to infinity for very negative x, whose
// reciprocal is the right 0.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + fexp(-x)); }

// log(1 + exp(x)) = max(x, 0) + log(1 + t) with t = exp(-|x|) <= 1.  What the
// rounding of w = 1 + t lost, t - (w - 1), is exact and comes back to first
// order, over w.  Tiny steps keep what t has: x log2(e) rounded leaves it about
// 1.5 |x| 2^-24 off, as rounding dt + dt_bias to fp32 does, too (5e-7 of the step
// at x = -5, 2e-6 at -20).  s: sigmoid(x), the derivative, from the same t and 1 / w.
__device__ __forceinline__ float softplus(float x, float* s = nullptr) {
    const float t = fexp(-fabsf(x));
    const float w = 1.0f + t;
    const float rw = __builtin_amdgcn_rcpf(w);
    if (s) *s = x < 0.0f ? t * rw : rw;
    return fmaxf(x, 0.0f) + fmaf(__builtin_amdgcn_logf(w), kLn2, (t - (w - 1.0f)) * rw);
}

// d silu(x) / dx with s = sigmoid(x)
__device__ __forceinline__ float dsilu(float x, float s) { return s * (1.0f + x * (1.0f - s)); }

// The tokens of sequence b that count.
__device__ __forceinline__ int seq_end(const int32_t* seqlens, int64_t b, int L) {
    if (!seqlens) return L;
    const int e = seqlens[b];
    return e < 0 ? 0 : (e > L ? L : e);
}

}  // namespace cls
