// Gated delta rule, one token: every state is read and written once, which
// bounds it.  With a = S k and b = S q of the state as it came,
//     delta = beta (v - e^g a),  S' = e^g S + delta k^T,  y = scale (e^g b + delta k.q)
// so both sums over a row are taken in one pass and the new state is not read again.
#include <hip/hip_runtime.h>

#include "delta.hpp"
#include "launch_delta.hpp"

namespace cls {
namespace {

struct StepParams {
    const void *q, *k, *v;
    const float *g, *beta;
    float* h;
    void* y;
    int64_t q_batch, q_head, k_batch, k_head, v_batch, v_head, g_batch, b_batch;
    int batch, Hk, H, dk, dv;
    float scale;
};

template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// LANES lanes, four states each, to a row of the state; ROWS rows to a thread, all loads of them in flight together.
// WHOLE: dk is 4 LANES exactly or a multiple of 4, and rows start on 16 bytes.
template <typename E, int LANES, int ROWS, bool WHOLE>
__global__ __launch_bounds__(256) void delta_step_kernel(StepParams p) {
    typedef typename E::raw raw;
    constexpr int PASS = 256 / LANES;  // rows of a workgroup at a time
    const int nblk = (p.dv + PASS * ROWS - 1) / (PASS * ROWS);
    const int blk = blockIdx.x % nblk, h = blockIdx.x / nblk % p.H, b = blockIdx.x / nblk / p.H;
    const int kh = h / (p.H / p.Hk), lane = threadIdx.x % LANES, d0 = 4 * lane;
    const int row0 = blk * PASS * ROWS + threadIdx.x / LANES;
    float* S = p.h + (int64_t(b) * p.H + h) * p.dv * p.dk;

    f32x4 s[ROWS];
#pragma unroll
    for (int n = 0; n < ROWS; ++n) {
        const int row = row0 + n * PASS;
        s[n] = f32x4{0, 0, 0, 0};
        if (row >= p.dv) continue;
        const float* at = S + int64_t(row) * p.dk + d0;
        if (WHOLE) {
            if (d0 < p.dk) s[n] = *reinterpret_cast<const f32x4*>(at);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d0 + e < p.dk) s[n][e] = at[e];
        }
    }
    const raw* K = static_cast<const raw*>(p.k) + b * p.k_batch + kh * p.k_head + d0;
    const raw* Q = static_cast<const raw*>(p.q) + b * p.q_batch + kh * p.q_head + d0;
    f32x4 k{0, 0, 0, 0}, q{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (d0 + e < p.dk) {
            k[e] = E::get(K[e]);
            q[e] = E::get(Q[e]);
        }
    const raw* V = static_cast<const raw*>(p.v) + b * p.v_batch + h * p.v_head;
    raw* Y = static_cast<raw*>(p.y) + (int64_t(b) * p.H + h) * p.dv;
    float v[ROWS];
#pragma unroll
    for (int n = 0; n < ROWS; ++n) v[n] = row0 + n * PASS < p.dv ? E::get(V[row0 + n * PASS]) : 0.0f;
    const float fade = fexp(p.g[b * p.g_batch + h]), beta = p.beta[b * p.b_batch + h];
    const float kq = sum_lanes<LANES>(fmaf(k[0], q[0], k[1] * q[1]) + fmaf(k[2], q[2], k[3] * q[3]));
#pragma unroll
    for (int n = 0; n < ROWS; ++n) {
        const int row = row0 + n * PASS;
        const float a = sum_lanes<LANES>(fmaf(k[0], s[n][0], k[1] * s[n][1]) + fmaf(k[2], s[n][2], k[3] * s[n][3]));
        const float c = sum_lanes<LANES>(fmaf(q[0], s[n][0], q[1] * s[n][1]) + fmaf(q[2], s[n][2], q[3] * s[n][3]));
        if (row >= p.dv) continue;
        const float delta = beta * fmaf(-fade, a, v[n]);
        f32x4 t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = fmaf(delta, k[e], fade * s[n][e]);
        float* at = S + int64_t(row) * p.dk + d0;
        if (WHOLE) {
            if (d0 < p.dk) *reinterpret_cast<f32x4*>(at) = t;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d0 + e < p.dk) at[e] = t[e];
        }
        if (lane == 0) Y[row] = E::put(p.scale * fmaf(fade, c, delta * kq));
    }
}

int lanes_of(int64_t dk) { return dk <= 32 ? 8 : dk <= 64 ? 16 : dk <= 128 ? 32 : 64; }

// Rows of a state to a workgroup: four to a thread once that still leaves eight workgroups to a compute unit.
int rows_of(int64_t heads, int64_t dk, int64_t dv) {
    const int pass = 256 / lanes_of(dk);
    return heads * ((dv + 4 * pass - 1) / (4 * pass)) >= 2048 ? 4 * pass : pass;
}
int64_t groups_of(int64_t heads, int64_t dk, int64_t dv) {
    const int rows = rows_of(heads, dk, dv);
    return heads * ((dv + rows - 1) / rows);
}

template <typename E, int LANES>
int launch(const StepParams& p, hipStream_t stream) {
    const int64_t heads = int64_t(p.batch) * p.H;
    const bool whole = p.dk % 4 == 0, four = rows_of(heads, p.dk, p.dv) > 256 / LANES;
    const unsigned wgs = unsigned(groups_of(heads, p.dk, p.dv));
    if (four && whole) delta_step_kernel<E, LANES, 4, true><<<wgs, 256, 0, stream>>>(p);
    else if (four) delta_step_kernel<E, LANES, 4, false><<<wgs, 256, 0, stream>>>(p);
    else if (whole) delta_step_kernel<E, LANES, 1, true><<<wgs, 256, 0, stream>>>(p);
    else delta_step_kernel<E, LANES, 1, false><<<wgs, 256, 0, stream>>>(p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

template <typename E>
int launch(const StepParams& p, hipStream_t stream) {
    switch (lanes_of(p.dk)) {
        case 8: return launch<E, 8>(p, stream);
        case 16: return launch<E, 16>(p, stream);
        case 32: return launch<E, 32>(p, stream);
        default: return launch<E, 64>(p, stream);
    }
}

}  // namespace
}  // namespace cls

int64_t cls_delta_step_groups(int64_t heads, int64_t dk, int64_t dv) { return cls::groups_of(heads, dk, dv); }

int cls_delta_step_launch(const gated_delta_inputs& in, float* h, void* y, hipStream_t stream) {
    cls::StepParams p{};
    p.q = in.q; p.k = in.k; p.v = in.v; p.g = in.g; p.beta = in.beta; p.h = h; p.y = y;
    p.q_batch = in.q_batch; p.q_head = in.q_head; p.k_batch = in.k_batch; p.k_head = in.k_head;
    p.v_batch = in.v_batch; p.v_head = in.v_head; p.g_batch = in.g_batch; p.b_batch = in.beta_batch;
    p.batch = int(in.batch); p.Hk = int(in.kheads); p.H = int(in.heads); p.dk = int(in.dk); p.dv = int(in.dv);
    p.scale = in.scale;
    if (in.dtype == SSD_F32) return cls::launch<cls::ElemF32>(p, stream);
    return in.dtype == SSD_BF16 ? cls::launch<cls::ElemBF16>(p, stream) : cls::launch<cls::ElemF16>(p, stream);
}
