// Short causal convolution of each channel over the tokens, forward, backward
// and for one token, on gfx950.
//
// A few operations per element read and written, so bound by memory: a thread
// walks adjacent tokens of 4 or 8 channels with the last `width` inputs in
// registers, reading each row once but for the width - 1 before its run.
// 8 x 2048 x 1536 bf16: forward 22.3 us (101 MB: 19.5 us at copy rate), backward
// 39 us (151 MB: 29 us; its recomputed convolution, silu' and four products each
// for dx and the weights are some 22 us of vector instructions, which the one
// round of workgroups does not overlap with the loads wholly) and 4.7 us for the
// weights' sums.  3 x 1021 x 1536: 7.0 us; one token of 64 x 5120: 3.6 us.
#include "selective.hpp"

#include "launch_selective.hpp"

namespace cls {
namespace {

// V adjacent channels of one token.
template <typename E, int V>
struct Vec {
    typedef typename E::raw raw;
    typedef raw vec __attribute__((ext_vector_type(V)));
    static __device__ __forceinline__ vec load_raw(const raw* p) { return *reinterpret_cast<const vec*>(p); }
    static __device__ __forceinline__ void widen(vec v, float (&f)[V]) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const raw x = v[e];
            f[e] = E::get(x);
        }
    }
    static __device__ __forceinline__ void load(const raw* p, float (&f)[V]) {
        widen(load_raw(p), f);
    }
    static __device__ __forceinline__ void store(raw* p, const float (&f)[V]) {
        vec v;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = E::put(f[e]);
        *reinterpret_cast<vec*>(p) = v;
    }
    static __device__ __forceinline__ void zero(float (&f)[V]) {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = 0.0f;
    }
};

struct ConvParams {
    const void* x;
    int64_t x_b, x_t;
    const float *w, *bias;
    const void* init;
    const int32_t* seqlens;
    void* y;
    void* fin;
    const void* dy;
    int64_t dy_b, dy_t;
    const void* dfin;
    void* dx;
    float* parts;  // [parts][ch][W + 1]
    void* dinit;
    float *dw, *dbias;
    int batch, L, ch, nvec, silu;
    int run, chunks;  // tokens of a thread, and how many such runs a sequence has
    int lanes;        // backward: threads of a workgroup side by side in the channels, a power of two
    int64_t nparts;
};

constexpr int kConvGroup = 4;    // tokens that the backward pass loads together

// The input at token t of sequence b (t >= 1 - W), zeros before a sequence without a start.
template <typename E, int V, int W>
__device__ __forceinline__ void conv_input(const ConvParams& p, int64_t b, int64_t t, int c, float (&f)[V]) {
    typedef typename E::raw raw;
    if (t >= 0) Vec<E, V>::load(static_cast<const raw*>(p.x) + b * p.x_b + t * p.x_t + c, f);
    else if (p.init) Vec<E, V>::load(static_cast<const raw*>(p.init) + (b * (W - 1) + t + W - 1) * p.ch + c, f);
    else Vec<E, V>::zero(f);
}

// V channels' weights and biases are adjacent: whole vectors where V allows.
template <int V, int W>
__device__ __forceinline__ void conv_weights(const ConvParams& p, int c, float (&w)[W][V], float (&bias)[V]) {
    if constexpr (V % 4 == 0) {
        float flat[V * W];
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(p.w + int64_t(c) * W + 4 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) flat[4 * i + e] = v[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][e] = flat[e * W + k];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const f32x4 v = p.bias ? *reinterpret_cast<const f32x4*>(p.bias + c + 4 * i) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 4; ++e) bias[4 * i + e] = v[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][e] = p.w[int64_t(c + e) * W + k];
            bias[e] = p.bias ? p.bias[c + e] : 0.0f;
        }
    }
}

// A thread: V channels, RUN tokens, all of whose rows are loaded before the
// first is used.  The chunk after the last (of each sequence) writes the final
// state.
template <typename E, int V, int W, int RUN>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvParams p) {
    typedef typename E::raw raw;
    typedef Vec<E, V> vec;
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    const uint32_t per = uint32_t(p.chunks) + (p.fin ? 1u : 0u);
    const uint32_t j = id / uint32_t(p.nvec);
    const int c = int(id % uint32_t(p.nvec)) * V;
    const int chunk = int(j % per);
    const int64_t b = j / per;
    if (b >= p.batch) return;
    const int end = seq_end(p.seqlens, b, p.L);
    if (chunk == p.chunks) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float f[V];
            conv_input<E, V, W>(p, b, int64_t(end) - (W - 1) + k, c, f);
            vec::store(static_cast<raw*>(p.fin) + (b * (W - 1) + k) * p.ch + c, f);
        }
        return;
    }
    const int t0 = chunk * RUN;
    const raw* x = static_cast<const raw*>(p.x) + b * p.x_b + t0 * p.x_t + c;
    raw* y = static_cast<raw*>(p.y) + (b * p.L + t0) * p.ch + c;
    typename vec::vec rx[RUN];
    float w[W][V], bias[V], win[W][V];  // win: the last W inputs, the newest last
#pragma unroll
    for (int i = 0; i < RUN; ++i)
        if (t0 + i < end) rx[i] = vec::load_raw(x + i * p.x_t);
#pragma unroll
    for (int k = 1; k < W; ++k) conv_input<E, V, W>(p, b, t0 - W + k, c, win[k]);
    conv_weights<V, W>(p, c, w, bias);
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        if (t0 + i >= p.L) break;
#pragma unroll
        for (int k = 0; k + 1 < W; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) win[k][e] = win[k + 1][e];
        float out[V];
        vec::zero(out);
        if (t0 + i < end) {
            vec::widen(rx[i], win[W - 1]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float s = bias[e];
#pragma unroll
                for (int k = 0; k < W; ++k) s = fmaf(w[k][e], win[k][e], s);
                out[e] = p.silu ? s * sigmoid(s) : s;
            }
        }
        vec::store(y + i * int64_t(p.ch), out);
    }
}

// A thread: V channels and a run of tokens, of which it owns the weight
// gradients and the input gradients W - 1 tokens earlier; it walks the W - 1
// tokens behind its run for their dp, too.  Tokens come kConvGroup at a time,
// loaded while the group before them is computed.  The weight gradients of a
// workgroup's runs are added in LDS.
template <typename E, int V, int W>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvParams p) {
    typedef typename E::raw raw;
    typedef Vec<E, V> vec;
    constexpr int U = kConvGroup, Q = V * (W + 1);
    __shared__ float s_part[256 * (Q + 1)];
    const int runs = 256 / p.lanes;  // of a workgroup
    const int blocks = (p.nvec + p.lanes - 1) / p.lanes;
    const int v = int(blockIdx.x % uint32_t(blocks)) * p.lanes + int(threadIdx.x) % p.lanes;
    const int64_t group = blockIdx.x / uint32_t(blocks);
    const int64_t part = group * runs + int(threadIdx.x) / p.lanes;
    const bool on = v < p.nvec && part < int64_t(p.batch) * p.chunks;
    const int c = (v < p.nvec ? v : 0) * V;
    const int chunk = on ? int(part % p.chunks) : 0;
    const int64_t b = on ? part / p.chunks : 0;
    float dw[W][V], db[V];
#pragma unroll
    for (int k = 0; k < W; ++k) vec::zero(dw[k]);
    vec::zero(db);
    if (on) {
        const int end = seq_end(p.seqlens, b, p.L);
        const int t0 = chunk * p.run;
        float w[W][V], bias[V], x[W][V], dp[W][V];  // x, dp: of the last W tokens, the newest last
        conv_weights<V, W>(p, c, w, bias);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            vec::zero(x[k]);
            vec::zero(dp[k]);
        }
        if (t0 < end) {
#pragma unroll
            for (int k = 1; k < W; ++k) conv_input<E, V, W>(p, b, t0 - W + k, c, x[k]);
        }
        const raw* px = static_cast<const raw*>(p.x) + b * p.x_b + c;
        const raw* pg = static_cast<const raw*>(p.dy) + b * p.dy_b + c;
        typename vec::vec rx[U], rg[U];
        auto load = [&](int s) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (s + i < end) {
                    rx[i] = vec::load_raw(px + (s + i) * p.x_t);
                    rg[i] = vec::load_raw(pg + (s + i) * p.dy_t);
                }
        };
        load(t0);
        for (int i0 = 0; i0 < p.run + W - 1; i0 += U) {
            typename vec::vec cx[U], cg[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                cx[i] = rx[i];
                cg[i] = rg[i];
            }
            if (i0 + U < p.run + W - 1) load(t0 + i0 + U);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int i = i0 + j, s = t0 + i;
                if (i >= p.run + W - 1) break;
#pragma unroll
                for (int k = 0; k + 1 < W; ++k)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        x[k][e] = x[k + 1][e];
                        dp[k][e] = dp[k + 1][e];
                    }
                vec::zero(dp[W - 1]);
                if (s < end) {
                    float g[V];
                    vec::widen(cx[j], x[W - 1]);
                    vec::widen(cg[j], g);
                    const bool own = i < p.run;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float q = bias[e];
#pragma unroll
                        for (int k = 0; k < W; ++k) q = fmaf(w[k][e], x[k][e], q);
                        const float d = p.silu ? g[e] * dsilu(q, sigmoid(q)) : g[e];
                        dp[W - 1][e] = d;
                    }
                    if (own) {
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            db[e] += dp[W - 1][e];
#pragma unroll
                            for (int k = 0; k < W; ++k) dw[k][e] = fmaf(dp[W - 1][e], x[k][e], dw[k][e]);
                        }
                    }
                }
                // the input that token s is the last to see
                const int t = s - (W - 1);
                if ((i < W - 1 && chunk > 0) || t >= p.L) continue;
                float dx[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float a = 0.0f;
#pragma unroll
                    for (int k = 0; k < W; ++k) a = fmaf(w[W - 1 - k][e], dp[k][e], a);
                    dx[e] = a;
                }
                const int kept = t - (end - (W - 1));  // its place in the final state
                if (p.dfin && kept >= 0 && t < end) {
                    float f[V];
                    vec::load(static_cast<const raw*>(p.dfin) + (b * (W - 1) + kept) * p.ch + c, f);
#pragma unroll
                    for (int e = 0; e < V; ++e) dx[e] += f[e];
                }
                if (t >= 0) vec::store(static_cast<raw*>(p.dx) + (b * p.L + t) * p.ch + c, dx);
                else if (p.dinit) vec::store(static_cast<raw*>(p.dinit) + (b * (W - 1) + t + W - 1) * p.ch + c, dx);
            }
        }
    }
    float* mine = s_part + threadIdx.x * (Q + 1);  // an odd stride: lanes on different banks
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) mine[e * (W + 1) + k] = dw[k][e];
        mine[e * (W + 1) + W] = db[e];
    }
    __syncthreads();
    const int first = int(blockIdx.x % uint32_t(blocks)) * p.lanes;
    for (int i = threadIdx.x; i < p.lanes * Q; i += 256) {
        if (first + i / Q >= p.nvec) continue;
        float s = 0.0f;
        for (int r = 0; r < runs; ++r) s += s_part[(r * p.lanes + i / Q) * (Q + 1) + i % Q];
        p.parts[(group * p.ch + first * V) * (W + 1) + i] = s;
    }
}

// A workgroup: 64 adjacent values, its four waves a quarter of the parts each.
template <int W>
__global__ __launch_bounds__(256) void conv_bwd_sum_kernel(ConvParams p) {
    __shared__ float s_sum[4][64];
    const int64_t per = int64_t(p.ch) * (W + 1);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i = int64_t(blockIdx.x) * 64 + lane;
    float s = 0.0f;
    if (i < per) {
#pragma unroll 8
        for (int64_t q = wave; q < p.nparts; q += 4) s += p.parts[q * per + i];
    }
    s_sum[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || i >= per) return;
    s = (s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]);
    const int64_t ch = i / (W + 1);
    const int k = int(i % (W + 1));
    if (k < W) { if (p.dw) p.dw[ch * W + k] = s; }
    else if (p.dbias) p.dbias[ch] = s;
}

template <typename E, int V, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvParams p) {
    typedef typename E::raw raw;
    const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (id >= int64_t(p.batch) * p.nvec) return;
    const int c = int(id % p.nvec) * V;
    const int64_t b = id / p.nvec;
    float w[W][V], bias[V], x[W][V], y[V];
    raw* st = static_cast<raw*>(p.fin) + b * (W - 1) * p.ch + c;
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) Vec<E, V>::load(st + int64_t(k) * p.ch, x[k]);
    Vec<E, V>::load(static_cast<const raw*>(p.x) + b * p.x_b + c, x[W - 1]);
    conv_weights<V, W>(p, c, w, bias);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float s = bias[e];
#pragma unroll
        for (int k = 0; k < W; ++k) s = fmaf(w[k][e], x[k][e], s);
        y[e] = p.silu ? s * sigmoid(s) : s;
    }
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) Vec<E, V>::store(st + int64_t(k) * p.ch, x[k + 1]);
    Vec<E, V>::store(static_cast<raw*>(p.y) + b * p.ch + c, y);
}

int launched() { return hipGetLastError() == hipSuccess ? 0 : -7; }

dim3 blocks_for(int64_t threads) { return dim3(uint32_t((threads + 255) / 256)); }

int conv_bwd_run(int64_t batch, int64_t L, int64_t ch) {
    // One round of three workgroups, what the registers leave room for, on each of 256 CUs, with 4 channels to a
    // thread: 8 x 2048 x 1536 bf16 in runs of 32 (one round) took 39.5 us, of 16 (1.9 rounds) 45, of 48 (0.7) 49.6.
    const int64_t threads = int64_t(3) * 256 * 256;
    const int64_t run = (batch * L * ((ch + 3) / 4) + 8 * threads - 1) / (8 * threads) * 8;
    return int(run < 16 ? 16 : run > 512 ? 512 : run);
}

enum { kFwd, kBwd, kStep };

template <int WHAT, typename E, int V, int W>
int launch(ConvParams p, hipStream_t s) {
    p.nvec = p.ch / V;
    const int64_t row = int64_t(p.batch) * p.nvec;
    if constexpr (WHAT == kFwd) {
        // Longer runs read fewer rows twice, shorter ones give the device more threads.  bf16, 16, 8 and 4 tokens:
        // 8 x 2048 x 1536 23.5, 26, - us; 4 x 1000 x 2560 15.8, 12.3, 13.7; 3 x 1021 x 1536 -, 7.8, 7.3.
        const auto threads = [&](int run) { return row * ((p.L + run - 1) / run); };
        p.run = V > 4 || threads(16) >= (int64_t(1) << 18) ? 16 : threads(8) >= (int64_t(1) << 18) ? 8 : 4;
        p.chunks = (p.L + p.run - 1) / p.run;
        const dim3 grid = blocks_for(row * (p.chunks + (p.fin ? 1 : 0)));
        if (p.run == 16) hipLaunchKernelGGL((conv_fwd_kernel<E, V, W, 16>), grid, dim3(256), 0, s, p);
        if constexpr (V <= 4) {
            if (p.run == 8) hipLaunchKernelGGL((conv_fwd_kernel<E, V, W, 8>), grid, dim3(256), 0, s, p);
            if (p.run == 4) hipLaunchKernelGGL((conv_fwd_kernel<E, V, W, 4>), grid, dim3(256), 0, s, p);
        }
        return launched();
    } else if constexpr (WHAT == kStep) {
        hipLaunchKernelGGL((conv_step_kernel<E, V, W>), blocks_for(row), dim3(256), 0, s, p);
        return launched();
    } else {
        p.lanes = 64;
        while (p.lanes > 1 && p.lanes / 2 >= p.nvec) p.lanes /= 2;
        const int64_t runs = 256 / p.lanes;
        p.nparts = (int64_t(p.batch) * p.chunks + runs - 1) / runs;
        const int64_t blocks = (p.nvec + p.lanes - 1) / p.lanes;
        hipLaunchKernelGGL((conv_bwd_kernel<E, V, W>), dim3(uint32_t(blocks * p.nparts)), dim3(256), 0, s, p);
        if (launched() != 0) return -7;
        hipLaunchKernelGGL((conv_bwd_sum_kernel<W>), dim3(uint32_t((int64_t(p.ch) * (W + 1) + 63) / 64)), dim3(256), 0, s,
                           p);
        return launched();
    }
}

template <int WHAT, typename E, int V>
int launch_width(int64_t W, const ConvParams& p, hipStream_t s) {
    return W == 2   ? launch<WHAT, E, V, 2>(p, s)
           : W == 3 ? launch<WHAT, E, V, 3>(p, s)
                    : launch<WHAT, E, V, 4>(p, s);
}

// Whole vectors of 4 channels where every row of every tensor starts on one,
// and of 8 for the largest forward calls of 16-bit elements (4 x 8192 x 5120
// bf16: 144 us for 157; 8 x 2048 x 1536: 26.5 for 23.5).
template <int WHAT, typename E>
int launch_type(int64_t W, const ConvParams& p, hipStream_t s) {
    constexpr int size = int(sizeof(typename E::raw));
    uint64_t at = 0, params = 0;
    for (const void* q : {p.x, p.init, p.dy, p.dfin, static_cast<const void*>(p.y), static_cast<const void*>(p.fin),
                          static_cast<const void*>(p.dx), static_cast<const void*>(p.dinit)})
        at |= reinterpret_cast<uintptr_t>(q);
    for (const void* q : {static_cast<const void*>(p.w), static_cast<const void*>(p.bias)})
        params |= reinterpret_cast<uintptr_t>(q);
    at |= uint64_t(p.ch | p.x_b | p.x_t | p.dy_b | p.dy_t) * size;
    if (params % 16 != 0 || at % (4 * size) != 0) return launch_width<WHAT, E, 1>(W, p, s);
    if constexpr (WHAT == kFwd && size == 2) {
        if (at % 16 == 0 && int64_t(p.batch) * (p.ch / 8) * ((p.L + 15) / 16) >= (int64_t(1) << 19))
            return launch_width<WHAT, E, 8>(W, p, s);
    }
    return launch_width<WHAT, E, 4>(W, p, s);
}

template <int WHAT>
int launch_any(const short_conv_inputs& in, const ConvParams& p, hipStream_t s) {
    return in.dtype == 0   ? launch_type<WHAT, ElemF32>(in.width, p, s)
           : in.dtype == 1 ? launch_type<WHAT, ElemBF16>(in.width, p, s)
                           : launch_type<WHAT, ElemF16>(in.width, p, s);
}

ConvParams params(const short_conv_inputs& in) {
    ConvParams p{};
    p.x = in.x; p.x_b = in.x_batch; p.x_t = in.x_token;
    p.w = in.weight; p.bias = in.bias; p.init = in.initial_state; p.seqlens = in.seqlens;
    p.batch = int(in.batch); p.L = int(in.seqlen); p.ch = int(in.channels); p.silu = in.silu;
    return p;
}

}  // namespace
}  // namespace cls

int64_t cls_short_conv_bwd_parts(int64_t batch, int64_t seqlen, int64_t channels) {
    const int64_t run = cls::conv_bwd_run(batch, seqlen, channels);
    return (batch * ((seqlen + run - 1) / run) + 3) / 4;  // a workgroup adds four runs at least
}

int cls_short_conv_fwd_launch(const short_conv_inputs& in, void* y, void* final_state, hipStream_t stream) {
    cls::ConvParams p = cls::params(in);
    p.y = y; p.fin = final_state;
    return cls::launch_any<cls::kFwd>(in, p, stream);
}

int cls_short_conv_bwd_launch(const short_conv_inputs& in, const void* dy, int64_t dy_batch, int64_t dy_token,
                              const void* dfinal, void* dx, float* dweight, float* dbias, void* dinitial, float* parts,
                              hipStream_t stream) {
    cls::ConvParams p = cls::params(in);
    p.dy = dy; p.dy_b = dy_batch; p.dy_t = dy_token; p.dfin = dfinal;
    p.dx = dx; p.dw = dweight; p.dbias = dbias; p.dinit = dinitial; p.parts = parts;
    p.run = cls::conv_bwd_run(in.batch, in.seqlen, in.channels);
    p.chunks = (p.L + p.run - 1) / p.run;
    return cls::launch_any<cls::kBwd>(in, p, stream);
}

int cls_short_conv_step_launch(const short_conv_inputs& in, void* state, void* y, hipStream_t stream) {
    cls::ConvParams p = cls::params(in);
    p.init = nullptr; p.x_t = 0;
    p.fin = state; p.y = y;
    return cls::launch_any<cls::kStep>(in, p, stream);
}
