// The norms around a block: gated_norm behind a recurrence and residual_norm in
// front of the next block, with their gradients:
//     y = unit(x) w silu(z)  or  unit(x silu(z)) w;   r = residual + s x, y = unit(r) w,
//     unit(u) = u / sqrt(mean(u^2) + eps),  du = rstd (a - unit mean(a unit)), a the gradient of unit.
// All are bound by memory: a row is read once, kept in registers between its sum
// and its output, and written once.  8 adjacent values (one or two 16-byte vectors)
// to a lane at a time; a row has 8, 16, 64 or more lanes, up to 1024: one run of
// them for the gradients of up to 8192 values, which keep several arrays of a row
// (5461 x 6144 in 256 lanes of three runs: 174 us, in 1024 of one: 98), and up to
// three otherwise, where barriers and the lanes behind a row's end cost more (1021
// x 5120 in 1024 lanes of one run: 17 us, in 256 of three: 10).  Rows of 129 to 256
// values leave half of their lanes or more without any (bf16 65536 x 256: 34 us,
// 2.9 TB/s; gradients and their sums 60), and rows off 8 values go one element at a
// time (16384 x 4095: 352 us, 4096: 103).  Workgroups walk over rows, so that w and
// s are read once (16384 x 4096: 102 us, 5.3 TB/s; one row to a workgroup: 165).
// The gradients of w and s are summed over the rows that a workgroup walks in its
// lanes, then over the workgroups by a second launch in a fixed order.
//
//     bf16             forward          gradients           their sums over workgroups
//     131072 x 128     19.4 us  5.2 TB/s  30.7 us  5.5 TB/s   4.7 us    gated_norm
//     8192 x 2048      34.1 us  5.9 TB/s  58.2 us  5.2 TB/s   7.0 us    residual_norm, the stream in fp32
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/gated_delta.h"
#include "launch_delta.hpp"
#include "selective.hpp"

namespace cls {
namespace {

// A workgroup has as many rows as fit 256 lanes, or one.
constexpr int threads_of(int lanes) { return lanes > 256 ? lanes : 256; }

template <typename E>
__device__ __forceinline__ void load8(const void* base, int64_t at, int left, bool vec, float (&v)[8]) {
    const typename E::raw* p = static_cast<const typename E::raw*>(base) + at;
    if (vec && left >= 8) {
        if constexpr (sizeof(typename E::raw) == 4) {
            const u32x4 a = ldg_b128(p), b = ldg_b128(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = as_float(a[e]);
                v[4 + e] = as_float(b[e]);
            }
        } else {
            const u32x4 a = ldg_b128(p);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t w = a[e >> 1];
                v[e] = E::get(typename E::raw(e & 1 ? w >> 16 : w));
            }
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? E::get(p[e]) : 0.0f;
}

template <typename E>
__device__ __forceinline__ void store8(void* base, int64_t at, int left, bool vec, const float (&v)[8]) {
    typedef typename E::raw raw;
    raw* p = static_cast<raw*>(base) + at;
    if (vec && left >= 8) {
        if constexpr (sizeof(raw) == 4) {
            *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = uint32_t(E::put(v[2 * e])) | (uint32_t(E::put(v[2 * e + 1])) << 16);
            *reinterpret_cast<u32x4*>(p) = w;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left) p[e] = E::put(v[e]);
}

// Where a lane has two runs of a row (more than 8192 values) its gradients do not keep both: they are read one at a
// time, and again, from the cache, when the row's sum is there (gated_norm of 2048 x 16384 in bf16: 146 us; all kept: 286).
// The factors and their gradients' sums stay in registers from row to row and do not fit the 128 that 1024 lanes have
// each: up to 36 are spilled, of residual_norm's up to 192 (bf16 230 us, 1.8 TB/s; with the stream in fp32 269; fp32 259).
template <int NV>
__device__ __forceinline__ void again() {
    if constexpr (NV > 1) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
}

// A lane's part of a row's factors, `fill` where there are none.
template <int LANES, int NV>
__device__ __forceinline__ void load_row(const float* p, int dim, bool vec, float fill, float (&v)[NV][8]) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int col = (n * LANES + threadIdx.x % LANES) * 8;
        if (p) {
            load8<ElemF32>(p, col, dim - col, vec, v[n]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[n][e] = fill;
        }
    }
}

// Sum over the LANES lanes of a row.  Where those are of more than one wave all of a workgroup's waves meet, once: calls
// use the two halves of scratch (kSums floats) in turn.
template <int LANES>
constexpr int kSums = LANES > 64 ? 2 * threads_of(LANES) / 64 : 1;
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* scratch, int& turn) {
#pragma unroll
    for (int d = (LANES < 64 ? LANES : 64) / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    if constexpr (LANES > 64) {
        constexpr int W = LANES / 64;
        float* s = scratch + (turn ^= threads_of(LANES) / 64);
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) s[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) v += s[wave / W * W + k];
    }
    return v;
}

// Column sums of a workgroup's rows: one row of `parts`.
template <int LANES, int NV>
__device__ __forceinline__ void put_parts(const float (&sum)[NV][8], float* parts, int dim, float* scratch) {
    constexpr int THREADS = threads_of(LANES), ROWS = THREADS / LANES;
    const int lane = threadIdx.x % LANES;
    if constexpr (ROWS == 1) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int col = (n * LANES + lane) * 8 + e;
                if (col < dim) parts[int64_t(blockIdx.x) * dim + col] = sum[n][e];
            }
    } else {  // scratch: [THREADS][8]
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) scratch[threadIdx.x * 8 + e] = sum[n][e];
            __syncthreads();
            for (int col = threadIdx.x; col < LANES * 8; col += THREADS) {
                float v = 0.0f;
                for (int r = 0; r < ROWS; ++r) v += scratch[r * LANES * 8 + col];
                const int at = n * LANES * 8 + col;
                if (at < dim) parts[int64_t(blockIdx.x) * dim + at] = v;
            }
        }
    }
}

struct GatedParams {
    const void *x, *z, *dy;
    const float* weight;
    float* rstd;
    void *y, *dx, *dz;
    float* parts;
    int64_t x_row, x_head, z_row, z_head, dy_row, dy_head;
    int64_t total;  // rows * heads
    int heads, dim, gate_first;
    float eps;
    uint8_t vec_x, vec_z, vec_dy, vec_out, vec_w;
};

template <typename E, int LANES, int NV, bool BWD>
__global__ __launch_bounds__(threads_of(LANES)) void gated_norm_kernel(GatedParams p) {
    constexpr int THREADS = threads_of(LANES), ROWS = THREADS / LANES;
    __shared__ float scratch[BWD && ROWS > 1 ? THREADS * 8 : kSums<LANES>];
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const float inv = 1.0f / float(p.dim);
    int turn = 0;
    float w[NV][8], dw[NV][8] = {};
    load_row<LANES, NV>(p.weight, p.dim, p.vec_w, 1.0f, w);
    // rows are counted with their heads: one division, then steps
    const int64_t step = int64_t(gridDim.x) * ROWS;
    int64_t at = int64_t(blockIdx.x) * ROWS + sub, row = at / p.heads, head = at % p.heads;
    const int64_t rows = step / p.heads, heads = step % p.heads;
    // all of a workgroup's lanes take the same number of turns: sums may meet at a barrier
    for (; at - sub < p.total; at += step, row += rows, head += heads) {
        if (head >= p.heads) {
            head -= p.heads;
            ++row;
        }
        const bool on = at < p.total;
        float x[NV][8], z[NV][8], dy[NV][8], u[NV][8], gate[NV][8], sig[NV][8];
        const auto read = [&](int n) {
            const int col = (n * LANES + lane) * 8, left = on ? p.dim - col : 0;
            load8<E>(p.x, row * p.x_row + head * p.x_head + col, left, p.vec_x, x[n]);
            load8<E>(p.z ? p.z : p.x, row * p.z_row + head * p.z_head + col, p.z ? left : 0, p.vec_z, z[n]);
            if (BWD) load8<E>(p.dy, row * p.dy_row + head * p.dy_head + col, left, p.vec_dy, dy[n]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sig[n][e] = p.z ? sigmoid(z[n][e]) : 1.0f;
                gate[n][e] = p.z ? z[n][e] * sig[n][e] : 1.0f;
                u[n][e] = p.gate_first ? x[n][e] * gate[n][e] : x[n][e];
            }
        };
        float rstd = 0.0f, ss = 0.0f;
        if (BWD) {
            rstd = on ? p.rstd[at] : 0.0f;
        } else {
#pragma unroll
            for (int n = 0; n < NV; ++n) read(n);
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(u[n][e], u[n][e], ss);
            rstd = 1.0f / sqrtf(fmaf(row_sum<LANES>(ss, scratch, turn), inv, p.eps));
            if (p.rstd && on && lane == 0) p.rstd[at] = rstd;
        }
        const int64_t out = at * p.dim;
        if (!BWD) {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int col = (n * LANES + lane) * 8, left = on ? p.dim - col : 0;
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = u[n][e] * rstd * w[n][e];
                    if (!p.gate_first) y[e] *= gate[n][e];
                }
                store8<E>(p.y, out + col, left, p.vec_out, y);
            }
            continue;
        }
        // the gradient of u: rstd (a - unit mean(a unit)), a that of unit = u rstd
        float mean = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            read(n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dn = p.gate_first ? dy[n][e] : dy[n][e] * gate[n][e];
                const float unit = u[n][e] * rstd;
                dw[n][e] = fmaf(dn, unit, dw[n][e]);
                mean = fmaf(dn * w[n][e], unit, mean);
            }
            again<NV>();
        }
        mean = row_sum<LANES>(mean, scratch, turn) * inv;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (n * LANES + lane) * 8, left = on ? p.dim - col : 0;
            float dx[8], dz[8];
            if (NV > 1) read(n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float unit = u[n][e] * rstd, a = dy[n][e] * w[n][e];
                const float slope = dsilu(z[n][e], sig[n][e]);
                const float du = rstd * fmaf(-unit, mean, p.gate_first ? a : a * gate[n][e]);
                dx[e] = p.gate_first ? du * gate[n][e] : du;
                dz[e] = (p.gate_first ? du * x[n][e] : a * unit) * slope;
            }
            store8<E>(p.dx, out + col, left, p.vec_out, dx);
            if (p.z) store8<E>(p.dz, out + col, left, p.vec_out, dz);
            again<NV>();
        }
    }
    if (BWD && p.parts) put_parts<LANES, NV>(dw, p.parts, p.dim, scratch);
}

struct ResidualParams {
    const void *x, *residual, *dy, *dr, *r_in;
    const float *scale, *weight;
    float* rstd;
    void *y, *r, *dresidual, *dx;
    float *parts_w, *parts_s;
    int64_t x_row, residual_row, dy_row, dr_row, r_row, rows;
    int dim;
    float eps;
    uint8_t vec_x, vec_res, vec_dy, vec_dr, vec_r, vec_out, vec_w;  // vec_w: scale and weight
};

template <typename E, typename S, int LANES, int NV>
__global__ __launch_bounds__(threads_of(LANES)) void residual_norm_kernel(ResidualParams p) {
    constexpr int THREADS = threads_of(LANES), ROWS = THREADS / LANES;
    __shared__ float scratch[kSums<LANES>];
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const float inv = 1.0f / float(p.dim);
    int turn = 0;
    float w[NV][8], s[NV][8];
    load_row<LANES, NV>(p.weight, p.dim, p.vec_w, 1.0f, w);
    load_row<LANES, NV>(p.scale, p.dim, p.vec_w, 1.0f, s);
    for (int64_t first = int64_t(blockIdx.x) * ROWS; first < p.rows; first += int64_t(gridDim.x) * ROWS) {
        const int64_t row = first + sub;
        const bool on = row < p.rows;
        float r[NV][8], x[NV][8];
        float ss = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (n * LANES + lane) * 8, left = on ? p.dim - col : 0;
            load8<E>(p.x, row * p.x_row + col, left, p.vec_x, x[n]);
            if (p.residual) load8<S>(p.residual, row * p.residual_row + col, left, p.vec_res, r[n]);
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (n * LANES + lane) * 8, left = on ? p.dim - col : 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = p.residual ? fmaf(s[n][e], x[n][e], r[n][e]) : s[n][e] * x[n][e];
                r[n][e] = S::get(S::put(v));  // the norm is that of the stream as it is kept
                ss = fmaf(r[n][e], r[n][e], ss);
            }
            store8<S>(p.r, row * p.dim + col, left, p.vec_out, r[n]);
        }
        const float rstd = 1.0f / sqrtf(fmaf(row_sum<LANES>(ss, scratch, turn), inv, p.eps));
        if (p.rstd && on && lane == 0) p.rstd[row] = rstd;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (n * LANES + lane) * 8, left = on ? p.dim - col : 0;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = r[n][e] * rstd * w[n][e];
            store8<E>(p.y, row * p.dim + col, left, p.vec_out, y);
        }
    }
}

template <typename E, typename S, int LANES, int NV>
__global__ __launch_bounds__(threads_of(LANES)) void residual_norm_bwd_kernel(ResidualParams p) {
    constexpr int THREADS = threads_of(LANES), ROWS = THREADS / LANES;
    __shared__ float scratch[ROWS > 1 ? THREADS * 8 : kSums<LANES>];
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const float inv = 1.0f / float(p.dim);
    int turn = 0;
    float w[NV][8], s[NV][8], dw[NV][8] = {}, ds[NV][8] = {};
    load_row<LANES, NV>(p.weight, p.dim, p.vec_w, 1.0f, w);
    load_row<LANES, NV>(p.scale, p.dim, p.vec_w, 1.0f, s);
    for (int64_t first = int64_t(blockIdx.x) * ROWS; first < p.rows; first += int64_t(gridDim.x) * ROWS) {
        const int64_t row = first + sub;
        const bool on = row < p.rows;
        const float rstd = on ? p.rstd[row] : 0.0f;
        float dy[NV][8], unit[NV][8], dr[NV][8], x[NV][8];
        float mean = 0.0f;
        const auto read = [&](int n, bool all) {
            const int col = (n * LANES + lane) * 8, left = on ? p.dim - col : 0;
            load8<E>(p.dy, row * p.dy_row + col, left, p.vec_dy, dy[n]);
            load8<S>(p.r_in, row * p.r_row + col, left, p.vec_r, unit[n]);
            if (all) {
                load8<S>(p.dr ? p.dr : p.r_in, row * p.dr_row + col, p.dr ? left : 0, p.vec_dr, dr[n]);
                load8<E>(p.parts_s ? p.x : p.dy, row * p.x_row + col, p.parts_s ? left : 0, p.vec_x, x[n]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) unit[n][e] *= rstd;
        };
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            read(n, NV == 1);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[n][e] = fmaf(dy[n][e], unit[n][e], dw[n][e]);
                mean = fmaf(dy[n][e] * w[n][e], unit[n][e], mean);
            }
            again<NV>();
        }
        mean = row_sum<LANES>(mean, scratch, turn) * inv;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (n * LANES + lane) * 8, left = on ? p.dim - col : 0;
            float du[8], dx[8];
            if (NV > 1) read(n, true);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                du[e] = rstd * fmaf(-unit[n][e], mean, dy[n][e] * w[n][e]);
                du[e] += dr[n][e];
                dx[e] = du[e] * s[n][e];
                ds[n][e] = fmaf(du[e], x[n][e], ds[n][e]);
            }
            store8<S>(p.dresidual, row * p.dim + col, left, p.vec_out, du);
            if (p.dx) store8<E>(p.dx, row * p.dim + col, left, p.vec_out, dx);
            again<NV>();
        }
    }
    if (p.parts_w) put_parts<LANES, NV>(dw, p.parts_w, p.dim, scratch);
    if (p.parts_s) put_parts<LANES, NV>(ds, p.parts_s, p.dim, scratch);
}

// out[col] = sum of parts[0..n)[col], for one or two: 16 columns by 64 threads each, in a fixed order.
struct SumsParams {
    const float* parts[2];
    float* out[2];
    int n, dim;
};
__global__ __launch_bounds__(1024) void norm_sums_kernel(SumsParams p) {
    __shared__ float s[64][17];
    const int col = blockIdx.x * 16 + (threadIdx.x & 15), at = threadIdx.x >> 4;
    const float* parts = blockIdx.y ? p.parts[1] : p.parts[0];
    float v = 0.0f;
    if (col < p.dim) {
        constexpr int U = 8;  // loads in flight
        for (int k = at; k < p.n; k += 64 * U) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = k + 64 * u < p.n ? parts[int64_t(k + 64 * u) * p.dim + col] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) v += x[u];
        }
    }
    s[at][threadIdx.x & 15] = v;
    __syncthreads();
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        if (at < d) s[at][threadIdx.x & 15] += s[at + d][threadIdx.x & 15];
        __syncthreads();
    }
    if (at == 0 && col < p.dim) (blockIdx.y ? p.out[1] : p.out[0])[col] = s[0][threadIdx.x & 15];
}

int sums(const SumsParams& p, hipStream_t stream) {
    norm_sums_kernel<<<dim3((p.dim + 15) / 16, p.out[1] ? 2 : 1), 1024, 0, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

// Calls f with the lanes of a row and the runs of 8 values that each has.  The gradients keep several arrays of a row, so
// theirs are of one run.
template <bool BWD, typename F>
auto by_dim(int dim, F&& f) {
    const auto of = [&](auto lanes, auto nv) { return f(lanes, nv); };
    using std::integral_constant;
    if (dim <= 64) return of(integral_constant<int, 8>(), integral_constant<int, 1>());
    if (dim <= 128) return of(integral_constant<int, 16>(), integral_constant<int, 1>());
    if (dim <= 512) return of(integral_constant<int, 64>(), integral_constant<int, 1>());
    if constexpr (BWD) {
        if (dim <= 1024) return of(integral_constant<int, 128>(), integral_constant<int, 1>());
        if (dim <= 2048) return of(integral_constant<int, 256>(), integral_constant<int, 1>());
        if (dim <= 4096) return of(integral_constant<int, 512>(), integral_constant<int, 1>());
        if (dim <= 8192) return of(integral_constant<int, 1024>(), integral_constant<int, 1>());
    } else {
        if (dim <= 1024) return of(integral_constant<int, 64>(), integral_constant<int, 2>());
        if (dim <= 2048) return of(integral_constant<int, 256>(), integral_constant<int, 1>());
        if (dim <= 4096) return of(integral_constant<int, 256>(), integral_constant<int, 2>());
        if (dim <= 6144) return of(integral_constant<int, 256>(), integral_constant<int, 3>());
        if (dim <= 8192) return of(integral_constant<int, 512>(), integral_constant<int, 2>());
    }
    return of(integral_constant<int, 1024>(), integral_constant<int, 2>());
}

template <typename F>
int by_element(int dtype, F&& f) {
    if (dtype == SSD_F32) return f(ElemF32());
    return dtype == SSD_BF16 ? f(ElemBF16()) : f(ElemF16());
}

bool whole(const void* p, int64_t dim, int dtype, int64_t a, int64_t b) {
    const int64_t ve = dtype == SSD_F32 ? 4 : 8;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && dim % 8 == 0 && a % ve == 0 && b % ve == 0;
}

// Workgroups of a launch: as many rows as a compute unit's lanes have, or half of them for the gradients, whose partial sums
// are one to a workgroup.
template <bool BWD>
unsigned groups(int64_t rows, int64_t dim) {
    return by_dim<BWD>(int(dim), [&](auto lanes, auto) {
        constexpr int THREADS = threads_of(decltype(lanes)::value);
        const int64_t per = THREADS / lanes, n = (rows + per - 1) / per, most = 256 * (BWD ? 1024 : 2048) / THREADS;
        return unsigned(n < most ? n : most);
    });
}

}  // namespace
}  // namespace cls

// Workgroups of the gradients' launch, each with a partial sum of the parameters' gradients.
int64_t cls_norm_parts(int64_t rows, int64_t dim) { return cls::groups<true>(rows, dim); }

int cls_gated_norm_launch(const gated_norm_inputs& in, const void* dy, int64_t dy_row, int64_t dy_head, float* rstd,
                          void* y, void* dx, void* dz, float* dweight, float* parts, hipStream_t stream) {
    using namespace cls;
    GatedParams p{};
    p.x = in.x; p.z = in.z; p.dy = dy; p.weight = in.weight; p.rstd = rstd;
    p.y = y; p.dx = dx; p.dz = dz; p.parts = dweight ? parts : nullptr;
    p.x_row = in.x_row; p.x_head = in.x_head; p.z_row = in.z_row; p.z_head = in.z_head;
    p.dy_row = dy_row; p.dy_head = dy_head;
    p.total = in.rows * in.heads;
    p.heads = int(in.heads); p.dim = int(in.dim); p.gate_first = in.gate_first; p.eps = in.eps;
    p.vec_x = whole(in.x, in.dim, in.dtype, in.x_row, in.x_head);
    p.vec_w = whole(in.weight, in.dim, SSD_F32, 0, 0);
    p.vec_z = whole(in.z, in.dim, in.dtype, in.z_row, in.z_head);
    p.vec_dy = whole(dy, in.dim, in.dtype, dy_row, dy_head);
    p.vec_out = whole(dy ? dx : y, in.dim, in.dtype, 0, 0) && whole(dy ? dz : nullptr, in.dim, in.dtype, 0, 0);
    const unsigned n = dy ? groups<true>(p.total, in.dim) : groups<false>(p.total, in.dim);
    const int st = by_element(in.dtype, [&](auto e) {
        const auto launch = [&](auto bwd) {
            return by_dim<decltype(bwd)::value>(p.dim, [&](auto lanes, auto nv) {
                constexpr int LANES = decltype(lanes)::value;
                gated_norm_kernel<decltype(e), LANES, decltype(nv)::value, decltype(bwd)::value>
                    <<<n, threads_of(LANES), 0, stream>>>(p);
                return hipGetLastError() == hipSuccess ? 0 : -7;
            });
        };
        return dy ? launch(std::true_type()) : launch(std::false_type());
    });
    return st == 0 && p.parts ? sums({{parts, nullptr}, {dweight, nullptr}, int(n), p.dim}, stream) : st;
}

int cls_residual_norm_fwd_launch(const residual_norm_inputs& in, void* y, void* r, float* rstd, hipStream_t stream) {
    using namespace cls;
    ResidualParams p{};
    p.x = in.x; p.residual = in.residual; p.scale = in.scale; p.weight = in.weight; p.rstd = rstd; p.y = y; p.r = r;
    p.x_row = in.x_row; p.residual_row = in.residual_row; p.rows = in.rows; p.dim = int(in.dim); p.eps = in.eps;
    p.vec_x = whole(in.x, in.dim, in.dtype, in.x_row, 0);
    p.vec_w = whole(in.weight, in.dim, SSD_F32, 0, 0) && whole(in.scale, in.dim, SSD_F32, 0, 0);
    p.vec_res = whole(in.residual, in.dim, in.stream_dtype, in.residual_row, 0);
    p.vec_out = whole(y, in.dim, in.dtype, 0, 0) && whole(r, in.dim, in.stream_dtype, 0, 0);
    const unsigned n = groups<false>(in.rows, in.dim);
    return by_element(in.dtype, [&](auto e) {
        return by_dim<false>(p.dim, [&](auto lanes, auto nv) {
            typedef decltype(e) E;
            constexpr int LANES = decltype(lanes)::value, NV = decltype(nv)::value;
            if (in.stream_dtype == SSD_F32) residual_norm_kernel<E, ElemF32, LANES, NV><<<n, threads_of(LANES), 0, stream>>>(p);
            else residual_norm_kernel<E, E, LANES, NV><<<n, threads_of(LANES), 0, stream>>>(p);
            return hipGetLastError() == hipSuccess ? 0 : -7;
        });
    });
}

int cls_residual_norm_bwd_launch(const residual_norm_inputs& in, const residual_norm_grads& g, float* parts,
                                 hipStream_t stream) {
    using namespace cls;
    ResidualParams p{};
    p.x = in.x; p.scale = in.scale; p.weight = in.weight; p.x_row = in.x_row; p.rows = in.rows; p.dim = int(in.dim);
    p.dy = g.dy; p.dr = g.dr; p.r_in = g.r; p.rstd = const_cast<float*>(g.rstd);
    p.dy_row = g.dy_row; p.dr_row = g.dr_row; p.r_row = g.r_row;
    p.dresidual = g.dresidual; p.dx = g.dx;
    const int64_t n = cls_norm_parts(in.rows, in.dim);
    p.parts_w = g.dweight ? parts : nullptr;
    p.parts_s = g.dscale ? parts + n * in.dim : nullptr;
    p.vec_x = whole(in.x, in.dim, in.dtype, in.x_row, 0);
    p.vec_w = whole(in.weight, in.dim, SSD_F32, 0, 0) && whole(in.scale, in.dim, SSD_F32, 0, 0);
    p.vec_dy = whole(g.dy, in.dim, in.dtype, g.dy_row, 0);
    p.vec_dr = whole(g.dr, in.dim, in.stream_dtype, g.dr_row, 0);
    p.vec_r = whole(g.r, in.dim, in.stream_dtype, g.r_row, 0);
    p.vec_out = whole(g.dresidual, in.dim, in.stream_dtype, 0, 0) && whole(g.dx, in.dim, in.dtype, 0, 0);
    const int st = by_element(in.dtype, [&](auto e) {
        return by_dim<true>(p.dim, [&](auto lanes, auto nv) {
            typedef decltype(e) E;
            constexpr int LANES = decltype(lanes)::value, NV = decltype(nv)::value;
            if (in.stream_dtype == SSD_F32)
                residual_norm_bwd_kernel<E, ElemF32, LANES, NV><<<unsigned(n), threads_of(LANES), 0, stream>>>(p);
            else residual_norm_bwd_kernel<E, E, LANES, NV><<<unsigned(n), threads_of(LANES), 0, stream>>>(p);
            return hipGetLastError() == hipSuccess ? 0 : -7;
        });
    });
    if (st != 0 || (!g.dweight && !g.dscale)) return st;
    if (!g.dweight) return sums({{p.parts_s, nullptr}, {g.dscale, nullptr}, int(n), p.dim}, stream);
    return sums({{p.parts_w, p.parts_s}, {g.dweight, g.dscale}, int(n), p.dim}, stream);
}
