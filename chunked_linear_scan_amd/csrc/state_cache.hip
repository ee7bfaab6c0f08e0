// States in 8 bits with a scale per row, written to and read from slots of a
// cache, on gfx950.
//
// Moves 5 bytes a value each way and is bound by memory: 32 states of 5120 rows
// of 128 written and read back in 41.5 us (210 MB: 40.6 us at copy rate).  A row
// is held by up to 64 lanes as float4s; its largest magnitude is found by lane
// permutes.  The division that gives a row's scale and inverse is one per row;
// values are multiplied by the inverse, so every rounding is one that a plain
// evaluation makes, too, and the bytes agree bit for bit.
#include "selective.hpp"

#include "launch_selective.hpp"

namespace cls {
namespace {

struct CacheParams {
    float* h;              // read by the write, written by the read
    const int32_t* slots;
    uint8_t* cache;
    float* scales;
    int64_t rows, nslots, blocks;  // blocks: workgroups per state
    int batch, S;
};

constexpr float kCacheSmallest = 0x1p-100f;

// four scaled values as bytes
template <bool FP8>
__device__ __forceinline__ uint32_t pack4(f32x4 q) {
    if constexpr (FP8) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(q.x, q.y, 0, false);
        return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(q.z, q.w, v, true));
    } else {
        uint32_t v = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f = __builtin_amdgcn_fmed3f(rintf(q[e]), -127.0f, 127.0f);  // a NaN becomes a number
            v |= (uint32_t(int(f)) & 0xffu) << (8 * e);
        }
        return v;
    }
}

template <bool FP8>
__device__ __forceinline__ f32x4 unpack4(uint32_t v) {
    f32x4 f;
    if constexpr (FP8) {
        f.x = __builtin_amdgcn_cvt_f32_fp8(v, 0);
        f.y = __builtin_amdgcn_cvt_f32_fp8(v, 1);
        f.z = __builtin_amdgcn_cvt_f32_fp8(v, 2);
        f.w = __builtin_amdgcn_cvt_f32_fp8(v, 3);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = float(int8_t(v >> (8 * e)));
    }
    return f;
}

// The lane's four values of a row; WIDE: whole aligned vectors, past the caches (a state is written to the cache once:
// write and read of 32 states of 5120 rows of 128 in 41.5 us for 49.4).
template <bool WIDE>
__device__ __forceinline__ f32x4 load4(const float* row, int s, int S) {
    if constexpr (WIDE) {
        return s < S ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(row + s)) : f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = s + e < S ? row[s + e] : 0.0f;
        return v;
    }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, true));
    return o > v ? o : v;
}

// The largest of LS adjacent lanes, in all of them: within rows of 16 lanes, then across rows.
template <int LS>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
    if constexpr (LS > 1) v = dpp_max<0xb1>(v);
    if constexpr (LS > 2) v = dpp_max<0x4e>(v);
    if constexpr (LS > 4) v = dpp_max<0x141>(v);
    if constexpr (LS > 8) v = dpp_max<0x128>(v);
    if constexpr (LS > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = r[0] > r[1] ? r[0] : r[1];
    }
    if constexpr (LS > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = r[0] > r[1] ? r[0] : r[1];
    }
    return v;
}

// A thread has a part of U rows, 256 / LS apart, whose loads are in flight together.
template <bool FP8, bool WIDE, int LS, int U>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheParams p) {
    const int64_t b = blockIdx.x / uint32_t(p.blocks), blk = blockIdx.x % uint32_t(p.blocks);
    const int l = threadIdx.x % LS;
    const int64_t r0 = blk * (U * 256 / LS) + threadIdx.x / LS;
    f32x4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t r = r0 + i * (256 / LS);
        v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (r < p.rows) v[i] = load4<WIDE>(p.h + (b * p.rows + r) * p.S, 4 * l, p.S);
    }
    const int slot = p.slots[b];
    if (slot < 0 || slot >= p.nslots) return;
    // a later state that names the slot is the one to keep
    bool later = false;
    for (int i = int(b) + 1 + int(threadIdx.x); i < p.batch; i += 256) later |= p.slots[i] == slot;
    if (__syncthreads_or(later)) return;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t r = r0 + i * (256 / LS);
        // the largest magnitude by its bits: NaN is above infinity
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f = v[i][e];
            const uint32_t a = as_uint(f) & 0x7fffffffu;
            m = a > m ? a : m;
        }
        m = max_lanes<LS>(m);
        const float top = FP8 ? 448.0f : 127.0f, big = as_float(m);
        const bool held = !(big < kCacheSmallest);
        const float scale = m >= 0x7f800000u ? as_float(0x7fc00000u) : held ? big / top : 0.0f;  // not finite: NaN
        const float inv = held ? top / big : 0.0f;
        if (r >= p.rows) continue;
        const int64_t at = int64_t(slot) * p.rows + r;
        if (l == 0) p.scales[at] = scale;
        f32x4 q;
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = v[i][e] * inv;
        const uint32_t bits = pack4<FP8>(q);
        uint8_t* out = p.cache + at * p.S + 4 * l;
        if constexpr (WIDE) {
            if (4 * l < p.S) *reinterpret_cast<uint32_t*>(out) = bits;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * l + e < p.S) out[e] = uint8_t(bits >> (8 * e));
        }
    }
}

template <bool FP8, bool WIDE, int LS>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheParams p) {
    const int64_t b = blockIdx.x / uint32_t(p.blocks), blk = blockIdx.x % uint32_t(p.blocks);
    const int slot = p.slots[b];
    const bool held = slot >= 0 && slot < p.nslots;
    const int l = threadIdx.x % LS;
    const int64_t r = (blk * 256 + threadIdx.x) / LS;
    if (r >= p.rows) return;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (held) {
        const int64_t at = int64_t(slot) * p.rows + r;
        const uint8_t* in = p.cache + at * p.S + 4 * l;
        uint32_t bits = 0;
        if constexpr (WIDE) {
            if (4 * l < p.S) bits = *reinterpret_cast<const uint32_t*>(in);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * l + e < p.S) bits |= uint32_t(in[e]) << (8 * e);
        }
        const float scale = p.scales[at];
        v = unpack4<FP8>(bits);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= scale;
    }
    float* out = p.h + (b * p.rows + r) * p.S + 4 * l;
    if constexpr (WIDE) {
        if (4 * l < p.S) *reinterpret_cast<f32x4*>(out) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (4 * l + e < p.S) out[e] = v[e];
    }
}

template <bool READ, bool FP8, bool WIDE, int LS>
int launch(CacheParams p, hipStream_t s) {
    const auto blocks = [&](int64_t u) { return (p.rows + u * (256 / LS) - 1) / (u * (256 / LS)); };
    p.blocks = blocks(1);
    if constexpr (READ) {
        hipLaunchKernelGGL((cache_read_kernel<FP8, WIDE, LS>), dim3(uint32_t(p.blocks * p.batch)), dim3(256), 0, s, p);
    } else if (blocks(4) * p.batch >= 1024) {
        // four rows to a thread where that leaves every CU a few workgroups: 32 states of 5120 rows of 128 in 25.4 us
        // for 28.6 us with one, 4 states of 1536 rows of 16 in 4.0 for 2.9
        p.blocks = blocks(4);
        hipLaunchKernelGGL((cache_write_kernel<FP8, WIDE, LS, 4>), dim3(uint32_t(p.blocks * p.batch)), dim3(256), 0, s, p);
    } else {
        hipLaunchKernelGGL((cache_write_kernel<FP8, WIDE, LS, 1>), dim3(uint32_t(p.blocks * p.batch)), dim3(256), 0, s, p);
    }
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

template <bool READ, bool FP8, bool WIDE>
int launch_lanes(const CacheParams& p, hipStream_t s) {
    const int lanes = (p.S + 3) / 4;
    return lanes <= 1    ? launch<READ, FP8, WIDE, 1>(p, s)
           : lanes <= 2  ? launch<READ, FP8, WIDE, 2>(p, s)
           : lanes <= 4  ? launch<READ, FP8, WIDE, 4>(p, s)
           : lanes <= 8  ? launch<READ, FP8, WIDE, 8>(p, s)
           : lanes <= 16 ? launch<READ, FP8, WIDE, 16>(p, s)
           : lanes <= 32 ? launch<READ, FP8, WIDE, 32>(p, s)
                         : launch<READ, FP8, WIDE, 64>(p, s);
}

template <bool READ>
int launch_any(const CacheParams& p, int format, hipStream_t s) {
    const bool wide = p.S % 4 == 0 && reinterpret_cast<uintptr_t>(p.h) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(p.cache) % 4 == 0;
    if (format == SSD_E4M3) return wide ? launch_lanes<READ, true, true>(p, s) : launch_lanes<READ, true, false>(p, s);
    return wide ? launch_lanes<READ, false, true>(p, s) : launch_lanes<READ, false, false>(p, s);
}

}  // namespace
}  // namespace cls

int cls_state_cache_write_launch(const float* h, const int32_t* slots, int64_t batch, int64_t rows, int64_t S,
                                 int64_t nslots, int format, void* cache, float* scales, hipStream_t stream) {
    const cls::CacheParams p{const_cast<float*>(h), slots, static_cast<uint8_t*>(cache), scales, rows, nslots, 0,
                             int(batch), int(S)};
    return cls::launch_any<false>(p, format, stream);
}

int cls_state_cache_read_launch(const void* cache, const float* scales, const int32_t* slots, int64_t batch,
                                int64_t rows, int64_t S, int64_t nslots, int format, float* h, hipStream_t stream) {
    const cls::CacheParams p{h, slots, static_cast<uint8_t*>(const_cast<void*>(cache)), const_cast<float*>(scales),
                             rows, nslots, 0, int(batch), int(S)};
    return cls::launch_any<true>(p, format, stream);
}
