// Short causal convolution of each channel over the tokens, forward, backward
// and for one token, on gfx950.
#include "selective.hpp"

#include "launch_selective.hpp"

namespace cls {
namespace {

// V adjacent channels of one token.
template <typename E, int V>
struct Vec {
    typedef typename E::raw raw;
    typedef raw vec __attribute__((ext_vector_type(V)));
    static __device__ __forceinline__ void load(const raw* p, float (&f)[V]) {
        if constexpr (V == 1) {
            f[0] = E::get(*p);
        } else {
            const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const raw x = v[e];
                f[e] = E::get(x);
            }
        }
    }
    static __device__ __forceinline__ void store(raw* p, const float (&f)[V]) {
        if constexpr (V == 1) {
            *p = E::put(f[0]);
        } else {
            vec v;
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = E::put(f[e]);
            *reinterpret_cast<vec*>(p) = v;
        }
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
    int batch, L, ch, nvec, chunks, silu;
    int64_t nparts;
};

constexpr int kConvRun = 8;      // tokens of a thread, forward
constexpr int kConvBwdRun = 32;  // and backward

// The input at token t of sequence b (t >= 1 - W), zeros before a sequence without a start.
template <typename E, int V, int W>
__device__ __forceinline__ void conv_input(const ConvParams& p, int64_t b, int64_t t, int c, float (&f)[V]) {
    typedef typename E::raw raw;
    if (t >= 0) Vec<E, V>::load(static_cast<const raw*>(p.x) + b * p.x_b + t * p.x_t + c, f);
    else if (p.init) Vec<E, V>::load(static_cast<const raw*>(p.init) + (b * (W - 1) + t + W - 1) * p.ch + c, f);
    else Vec<E, V>::zero(f);
}

template <int V, int W>
__device__ __forceinline__ void conv_weights(const ConvParams& p, int c, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][e] = p.w[int64_t(c + e) * W + k];
        bias[e] = p.bias ? p.bias[c + e] : 0.0f;
    }
}

// A thread: V channels, kConvRun tokens.  The chunk after the last (of each
// sequence) writes the final state.
template <typename E, int V, int W>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvParams p) {
    typedef typename E::raw raw;
    const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int per = p.chunks + (p.fin ? 1 : 0);
    if (id >= int64_t(p.batch) * per * p.nvec) return;
    const int c = int(id % p.nvec) * V;
    const int64_t j = id / p.nvec;
    const int chunk = int(j % per);
    const int64_t b = j / per;
    const int end = seq_end(p.seqlens, b, p.L);
    if (chunk == p.chunks) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float f[V];
            conv_input<E, V, W>(p, b, int64_t(end) - (W - 1) + k, c, f);
            Vec<E, V>::store(static_cast<raw*>(p.fin) + (b * (W - 1) + k) * p.ch + c, f);
        }
        return;
    }
    float w[W][V], bias[V], x[kConvRun + W - 1][V];
    conv_weights<V, W>(p, c, w, bias);
    const int t0 = chunk * kConvRun;
#pragma unroll
    for (int i = 0; i < kConvRun + W - 1; ++i) {
        const int t = t0 + i - (W - 1);
        if (t < end) conv_input<E, V, W>(p, b, t, c, x[i]);
        else Vec<E, V>::zero(x[i]);
    }
#pragma unroll
    for (int i = 0; i < kConvRun; ++i) {
        const int t = t0 + i;
        if (t >= p.L) break;
        float y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float s = bias[e];
#pragma unroll
            for (int k = 0; k < W; ++k) s = fmaf(w[k][e], x[i + k][e], s);
            if (p.silu) s *= sigmoid(s);
            y[e] = t < end ? s : 0.0f;
        }
        Vec<E, V>::store(static_cast<raw*>(p.y) + (b * p.L + t) * p.ch + c, y);
    }
}

// A thread: V channels, kConvBwdRun tokens of which it owns the weight
// gradients and the input gradients W - 1 tokens earlier; it walks the W - 1
// tokens behind its run for their dp, too.
template <typename E, int V, int W>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvParams p) {
    typedef typename E::raw raw;
    const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (id >= int64_t(p.batch) * p.chunks * p.nvec) return;
    const int c = int(id % p.nvec) * V;
    const int64_t part = id / p.nvec;
    const int chunk = int(part % p.chunks);
    const int64_t b = part / p.chunks;
    const int end = seq_end(p.seqlens, b, p.L);
    const int t0 = chunk * kConvBwdRun;
    float w[W][V], bias[V], dw[W][V], db[V], x[W][V], dp[W][V];  // x, dp: of the last W tokens, the newest last
    conv_weights<V, W>(p, c, w, bias);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        Vec<E, V>::zero(dw[k]);
        Vec<E, V>::zero(x[k]);
        Vec<E, V>::zero(dp[k]);
    }
    Vec<E, V>::zero(db);
    if (t0 < end) {
#pragma unroll
        for (int k = 1; k < W; ++k) conv_input<E, V, W>(p, b, t0 - W + k, c, x[k]);
    }
    for (int i = 0; i < kConvBwdRun + W - 1; ++i) {
        const int s = t0 + i;
#pragma unroll
        for (int k = 0; k + 1 < W; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                x[k][e] = x[k + 1][e];
                dp[k][e] = dp[k + 1][e];
            }
        Vec<E, V>::zero(dp[W - 1]);
        if (s < end) {
            float g[V];
            conv_input<E, V, W>(p, b, s, c, x[W - 1]);
            Vec<E, V>::load(static_cast<const raw*>(p.dy) + b * p.dy_b + s * p.dy_t + c, g);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float q = bias[e];
#pragma unroll
                for (int k = 0; k < W; ++k) q = fmaf(w[k][e], x[k][e], q);
                const float d = p.silu ? g[e] * dsilu(q, sigmoid(q)) : g[e];
                dp[W - 1][e] = d;
                if (i < kConvBwdRun) {
                    db[e] += d;
#pragma unroll
                    for (int k = 0; k < W; ++k) dw[k][e] = fmaf(d, x[k][e], dw[k][e]);
                }
            }
        }
        // the input that token s is the last to see
        const int t = s - (W - 1);
        if ((i < W - 1 && chunk > 0) || t >= p.L) continue;
        float dx[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) v = fmaf(w[W - 1 - k][e], dp[k][e], v);
            dx[e] = v;
        }
        const int kept = t - (end - (W - 1));  // its place in the final state
        if (p.dfin && kept >= 0 && t < end) {
            float f[V];
            Vec<E, V>::load(static_cast<const raw*>(p.dfin) + (b * (W - 1) + kept) * p.ch + c, f);
#pragma unroll
            for (int e = 0; e < V; ++e) dx[e] += f[e];
        }
        if (t >= 0) Vec<E, V>::store(static_cast<raw*>(p.dx) + (b * p.L + t) * p.ch + c, dx);
        else if (p.dinit) Vec<E, V>::store(static_cast<raw*>(p.dinit) + (b * (W - 1) + t + W - 1) * p.ch + c, dx);
    }
    float* out = p.parts + (part * p.ch + c) * (W + 1);
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) out[e * (W + 1) + k] = dw[k][e];
        out[e * (W + 1) + W] = db[e];
    }
}

template <int W>
__global__ __launch_bounds__(256) void conv_bwd_sum_kernel(ConvParams p) {
    const int64_t per = int64_t(p.ch) * (W + 1);
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= per) return;
    float s = 0.0f;
    for (int64_t q = 0; q < p.nparts; ++q) s += p.parts[q * per + i];
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

template <typename E, int V, int W>
int launch(int what, ConvParams p, hipStream_t s) {
    p.nvec = p.ch / V;
    const int64_t row = int64_t(p.batch) * p.nvec;
    if (what == 0) {
        hipLaunchKernelGGL((conv_fwd_kernel<E, V, W>), blocks_for(row * (p.chunks + (p.fin ? 1 : 0))), dim3(256), 0, s, p);
        return launched();
    }
    if (what == 2) {
        hipLaunchKernelGGL((conv_step_kernel<E, V, W>), blocks_for(row), dim3(256), 0, s, p);
        return launched();
    }
    hipLaunchKernelGGL((conv_bwd_kernel<E, V, W>), blocks_for(row * p.chunks), dim3(256), 0, s, p);
    if (launched() != 0) return -7;
    hipLaunchKernelGGL((conv_bwd_sum_kernel<W>), blocks_for(int64_t(p.ch) * (W + 1)), dim3(256), 0, s, p);
    return launched();
}

template <typename E, int V>
int launch_width(int what, int64_t W, const ConvParams& p, hipStream_t s) {
    return W == 2 ? launch<E, V, 2>(what, p, s) : W == 3 ? launch<E, V, 3>(what, p, s) : launch<E, V, 4>(what, p, s);
}

// Whole 16-byte vectors where every row of every tensor starts on one.
template <typename E>
int launch_type(int what, int64_t W, const ConvParams& p, hipStream_t s) {
    constexpr int V = 16 / int(sizeof(typename E::raw));
    uintptr_t at = 0;
    for (const void* q : {p.x, p.init, p.dy, p.dfin, static_cast<const void*>(p.y), static_cast<const void*>(p.fin),
                          static_cast<const void*>(p.dx), static_cast<const void*>(p.dinit)})
        at |= reinterpret_cast<uintptr_t>(q);
    const bool whole = at % 16 == 0 && p.ch % V == 0 && p.x_b % V == 0 && p.x_t % V == 0 && p.dy_b % V == 0 &&
                       p.dy_t % V == 0;
    return whole ? launch_width<E, V>(what, W, p, s) : launch_width<E, 1>(what, W, p, s);
}

int launch_any(int what, const short_conv_inputs& in, const ConvParams& p, hipStream_t s) {
    return in.dtype == 0 ? launch_type<ElemF32>(what, in.width, p, s)
         : in.dtype == 1 ? launch_type<ElemBF16>(what, in.width, p, s)
                         : launch_type<ElemF16>(what, in.width, p, s);
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

int64_t cls_short_conv_bwd_parts(int64_t batch, int64_t seqlen) {
    return batch * ((seqlen + cls::kConvBwdRun - 1) / cls::kConvBwdRun);
}

int cls_short_conv_fwd_launch(const short_conv_inputs& in, void* y, void* final_state, hipStream_t stream) {
    cls::ConvParams p = cls::params(in);
    p.y = y; p.fin = final_state;
    p.chunks = (p.L + cls::kConvRun - 1) / cls::kConvRun;
    return cls::launch_any(0, in, p, stream);
}

int cls_short_conv_bwd_launch(const short_conv_inputs& in, const void* dy, int64_t dy_batch, int64_t dy_token,
                              const void* dfinal, void* dx, float* dweight, float* dbias, void* dinitial, float* parts,
                              hipStream_t stream) {
    cls::ConvParams p = cls::params(in);
    p.dy = dy; p.dy_b = dy_batch; p.dy_t = dy_token; p.dfin = dfinal;
    p.dx = dx; p.dw = dweight; p.dbias = dbias; p.dinit = dinitial; p.parts = parts;
    p.chunks = (p.L + cls::kConvBwdRun - 1) / cls::kConvBwdRun;
    p.nparts = cls_short_conv_bwd_parts(in.batch, in.seqlen);
    return cls::launch_any(1, in, p, stream);
}

int cls_short_conv_step_launch(const short_conv_inputs& in, void* state, void* y, hipStream_t stream) {
    cls::ConvParams p = cls::params(in);
    p.init = nullptr; p.x_t = 0;
    p.fin = state; p.y = y;
    return cls::launch_any(2, in, p, stream);
}
