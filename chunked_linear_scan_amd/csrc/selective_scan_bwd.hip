// Selective scan, backward, on gfx950.
//
// With q = dL/dh of a token after it has used its own output,
//     q_t = dy_t C_t + a_{t+1} q_{t+1},   r_t = a_t q_t (handed to token t - 1)
// the gradients of a token are sums of products with h_{t-1}, h_t and r_t:
//     dC = sum_d dy h_t     dB = sum_d q (dt' u)        (over the lanes)
//     du = dt' s + D dy     ddt' = u s + sum_n r h_{t-1} A,  s = sum_n q B
//     dA = sum_t r h_{t-1} dt'    dz = dout y silu'(z)
// A tile of 8 tokens is taken from its checkpoint: its states and decays are
// computed forward into registers (64 of them), then the tokens are walked
// back.  dy C + r is a matrix instruction with r as its addend, s and y are sums
// by DPP operands as in the forward pass.  dB and dC need sums over the 64 lanes
// of 8 values per token and wave: permlane swaps of half waves and of rows add
// two values at once, so 8 values cost 15 instructions down to one register of
// eight lanes each, and eight tokens' registers then share 21 more.  The sums
// over channel blocks, segments and sequences are left to a second kernel,
// through partial results in the workspace: no atomics, the same bits every run.
//
// Bound by vector instructions: 16 per value (exp2 counting twice 17) and some
// 170 per tile and wave for staging and finishing; busy 84 % of the time.  Its
// waits are not hidden well: the state of a tile's checkpoint is loaded in the
// tile that uses it, and its wait covers the next tile's loads, too.
// 4 x 2048 x 1536 x 16 bf16: 188 us (185 at the fastest), after 50 us for the
// segments' own carries; then the sums, 8 us.  Its data at copy rate: 39 us.
// 16 tokens to a tile measured 305 us where 8 took 252 (registers; LDS for the
// partial sums).  Above 32 states a workgroup's 16 waves leave 128 registers to
// each, and 112 to 196 bytes a lane go to scratch memory in the loop:
// 2 x 1024 x 1536 bf16 takes 527 us at 64 states and 156 at 24.
#include "selective_scan.hpp"

#include "launch_selective.hpp"

namespace cls {
namespace {

// Waves per SIMD that the backward kernel's registers are kept to: 3 (168
// registers) measured 186 us where 2 took 198 and 4, with spills, 475.  With one
// or two waves to a workgroup each stages more rows and needs more registers.
constexpr int scan_bwd_waves(int NW, bool agg) { return NW > 8 || agg ? 4 : NW > 2 ? 3 : 2; }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Each halving step adds two lanes' values of two sums at once: a lane keeps
// the one that `bit` names and hands the other over.
__device__ __forceinline__ float swap_add32(float lo, float hi) {
    const auto r = __builtin_amdgcn_permlane32_swap(as_uint(lo), as_uint(hi), false, false);
    return as_float(r[0]) + as_float(r[1]);
}
__device__ __forceinline__ float swap_add16(float lo, float hi) {
    const auto r = __builtin_amdgcn_permlane16_swap(as_uint(lo), as_uint(hi), false, false);
    return as_float(r[0]) + as_float(r[1]);
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(bool bit, float lo, float hi) {
    return (bit ? hi : lo) + dpp<CTRL>(bit ? lo : hi);
}

// Z: with a gate.  AGG: what a segment alone hands back to the tokens before it (and its summed
// steps), from no gradient behind it.
template <typename E, int NW, bool AGG, bool Z>
__global__ __launch_bounds__(NW * 64, scan_bwd_waves(NW, AGG)) void scan_bwd_kernel(ScanParams p) {
    constexpr int K = kScanK;
    constexpr int TT = kScanTile;
    constexpr int R = TT >= NW ? TT / NW : 1;
    typedef typename E::raw raw;
    __shared__ float2 s_d[TT][kScanCh];   // dt', dt' u
    __shared__ float s_dy[TT][kScanCh];   // the gradient of y before the gate
    __shared__ float s_p[NW][Z ? 3 : 2][AGG ? 1 : TT][kScanCh];  // each wave's share of the sums over the states

    const ScanPlace at = scan_place(p, AGG ? 1 : 0);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t b = at.b;
    const bool on = at.on;
    const uint32_t ch = uint32_t(at.ch), lane_off = ch * uint32_t(sizeof(raw));
    const int seg = at.seg;
    const int64_t first = at.first, last = at.last;
    const float bias = p.dt_bias ? p.dt_bias[ch] : 0.0f;
    const float Dc = p.D ? p.D[ch] : 0.0f;

    const int n0 = wave * K;
    float A2[K], dA[K];
    f32x4 carry;  // the gradient that reaches the state from later tokens
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int n = n0 + k;
        A2[k] = n < p.N ? p.A[int64_t(ch) * p.N + n] * kLog2e : 0.0f;
        carry[k] = dA[k] = 0.0f;
    }
    if constexpr (!AGG) {
        if (p.dh_last) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (n0 + k < p.N) carry[k] = p.dh_last[(b * p.ch + ch) * p.N + n0 + k];
        }
        scan_fold(p, p.nseg - 1, -1, p.nseg - 1 - seg, b, at.ch, n0, A2, carry);
    }
    float sum_dt = 0.0f, dD = 0.0f, dbias = 0.0f;

    // the tiles from the last one back, from wave-uniform pointers that step with them
    const int64_t tiles = last > first ? (last - first + TT - 1) / TT : 0;
    const int64_t top = first + (tiles - 1) * TT;
    const raw* u = static_cast<const raw*>(p.u) + b * p.su.b + top * p.su.t;
    const raw* dt = static_cast<const raw*>(p.dt) + b * p.sdt.b + top * p.sdt.t;
    const raw* z = static_cast<const raw*>(p.z) + (Z ? b * p.sz.b + top * p.sz.t : 0);
    const raw* dy = static_cast<const raw*>(p.dy) + b * p.sdy.b + top * p.sdy.t;
    ScanRows<E> B(p.B, p.sB, b, at.g, top, n0, p.N, lane), C(p.C, p.sC, b, at.g, top, n0, p.N, lane);
    const int u_t = int(p.su.t), dt_t = int(p.sdt.t), z_t = int(p.sz.t), dy_t = int(p.sdy.t);
    raw ru[R], rdt[R], rz[R], rdy[R];
    // Loads the tile at t0 and steps back; before the segment there is none.
    auto load = [&](int64_t t0) {
        if (t0 < first) return;
        const int rem = int(last - 1 - t0 < TT ? last - 1 - t0 : TT);
        C.load(rem);
        if (!AGG) B.load(rem);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = wave + r * NW < rem ? wave + r * NW : rem;
            ru[r] = at_bytes(u + row * u_t, lane_off);
            rdt[r] = at_bytes(dt + row * dt_t, lane_off);
            rdy[r] = at_bytes(dy + row * dy_t, lane_off);
            rz[r] = 0;
            if (Z) rz[r] = at_bytes(z + row * z_t, lane_off);
        }
        u -= TT * int64_t(u_t);
        dt -= TT * int64_t(dt_t);
        dy -= TT * int64_t(dy_t);
        if (Z) z -= TT * int64_t(z_t);
        if (!AGG) B.step(-1);
        C.step(-1);
    };
    const int64_t out0 = (b * p.L + top) * p.ch;
    raw* du = static_cast<raw*>(p.du) + out0;
    raw* ddt = static_cast<raw*>(p.ddt) + out0;
    raw* dz = static_cast<raw*>(p.dz) + out0;
    const float* ckpt = p.ckpt + ((b * ((p.L + TT - 1) / TT) + top / TT) * p.N + n0) * p.ch;
    // the sums over the lanes of dB and dC end up in the lane (B or C, state, token of eight)
    const int sum_n = n0 + ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1), sum_t = lane & 7;
    float* part = p.part_bc + ((((int64_t(blockIdx.x) % p.bpg * p.batch + b) * p.L + top + sum_t) * p.G + at.g) * 2 +
                               (lane >> 5)) * p.N + sum_n;
    const int64_t part_t = int64_t(p.G) * 2 * p.N;
    if (tiles > 0) load(top);
    for (int64_t t0 = top; t0 >= first; t0 -= TT) {
        const int nt = int(last - t0 < TT ? last - t0 : TT);
        float hin[K];
        if constexpr (!AGG) {
#pragma unroll
            for (int k = 0; k < K; ++k) hin[k] = n0 + k < p.N ? at_bytes(ckpt + k * p.ch, ch * 4) : 0.0f;
        }
        float uc[R], zc[R], sz[R], sx[R], dc[R], oc[R], gc[R];  // sz, sx: the sigmoids of z and of dt + bias
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = wave + r * NW;
            uc[r] = E::get(ru[r]);
            zc[r] = E::get(rz[r]);
            oc[r] = E::get(rdy[r]);
            dc[r] = E::get(rdt[r]) + bias;
            sx[r] = 1.0f;
            if (p.softplus) dc[r] = softplus(dc[r], &sx[r]);
            sz[r] = Z ? sigmoid(zc[r]) : 1.0f;
            gc[r] = Z ? oc[r] * zc[r] * sz[r] : oc[r];
            float d = dc[r], s = dc[r] * uc[r], gy = gc[r];
            if (row >= nt) d = 0.0f;
            if (row >= nt || !on) s = gy = 0.0f;  // nothing of a lane without a channel in the sums over the lanes
            if (AGG && row < TT) sum_dt += d;
            if (row < TT) {
                s_d[row][lane] = make_float2(d, s);
                s_dy[row][lane] = gy;
            }
        }
        const float fC = C.get(), fB = AGG ? 0.0f : B.get();
        float qB[2], qC[2];
        if (!AGG) {
            row_quads(fB, qB);
            if (Z) row_quads(fC, qC);
        }
        load(t0 - TT);
        __syncthreads();
        if constexpr (AGG) {
            [&]<int... T>(std::integer_sequence<int, T...>) {
                (
                    [&] {
                        constexpr int t = TT - 1 - T;
                        const float d = s_d[t][lane].x;
                        const f32x4 q = outer<t>(fC, s_dy[t][lane], carry);
#pragma unroll
                        for (int k = 0; k < K; ++k) carry[k] = fexp2(d * A2[k]) * q[k];
                    }(),
                    ...);
            }(std::make_integer_sequence<int, TT>{});
            __syncthreads();
        } else {
            float a[TT][K], hs[TT][K];
            [&]<int... T>(std::integer_sequence<int, T...>) {
                (
                    [&] {
                        const float2 d = s_d[T][lane];
                        const f32x4 b4 = outer<T>(fB, d.y);
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            a[T][k] = fexp2(d.x * A2[k]);
                            hs[T][k] = fmaf(a[T][k], T ? hs[T ? T - 1 : 0][k] : hin[k], b4[k]);
                        }
                        if constexpr (Z) s_p[wave][2][T][lane] = dot<T>(qC, hs[T]);
                    }(),
                    ...);
            }(std::make_integer_sequence<int, TT>{});
            const bool bit3 = lane & 8, bit2 = lane & 4, bit1 = lane & 2, bit0 = lane & 1;
            float r8[8];
            [&]<int... I>(std::integer_sequence<int, I...>) {
                (
                    [&] {
                        constexpr int t = TT - 1 - I, i = t & 7;
                        const float2 d = s_d[t][lane];
                        const float gy = s_dy[t][lane];
                        const f32x4 q4 = outer<t>(fC, gy, carry);
                        float q[K], vB[K], vC[K], to_dt = 0.0f;
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            q[k] = q4[k];
                            const float qa = q[k] * a[t][k];
                            carry[k] = qa;
                            const float qah = qa * (t ? hs[t ? t - 1 : 0][k] : hin[k]);
                            dA[k] = fmaf(qah, d.x, dA[k]);
                            to_dt = fmaf(qah, A2[k], to_dt);
                            vB[k] = q[k] * d.y;
                            vC[k] = gy * hs[t][k];
                        }
                        s_p[wave][0][t][lane] = dot<t, true>(qB, q);
                        s_p[wave][1][t][lane] = to_dt;
                        const float w0 = swap_add32(vB[0], vC[0]), w1 = swap_add32(vB[1], vC[1]);
                        const float w2 = swap_add32(vB[2], vC[2]), w3 = swap_add32(vB[3], vC[3]);
                        r8[i] = dpp_add<0x128>(bit3, swap_add16(w0, w2), swap_add16(w1, w3));
                        if constexpr (i == 0) {
                            // eight tokens' sums over the last three lane bits: half-row mirror, then within four lanes
                            const float x0 = dpp_add<0x141>(bit2, r8[0], r8[4]), x1 = dpp_add<0x141>(bit2, r8[1], r8[5]);
                            const float x2 = dpp_add<0x141>(bit2, r8[2], r8[6]), x3 = dpp_add<0x141>(bit2, r8[3], r8[7]);
                            const float y0 = dpp_add<0x4e>(bit1, x0, x2), y1 = dpp_add<0x4e>(bit1, x1, x3);
                            const float sum = dpp_add<0xb1>(bit0, y0, y1);
                            if (t + sum_t < nt && sum_n < p.N) part[t * part_t] = sum;
                        }
                    }(),
                    ...);
            }(std::make_integer_sequence<int, TT>{});
            part -= TT * part_t;
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = wave + r * NW;
                if (row >= nt) continue;
                float to_sig = 0.0f, to_dt = 0.0f, y = Dc * uc[r];
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    to_sig += s_p[w][0][row][lane];
                    to_dt += s_p[w][1][row][lane];
                    if constexpr (Z) y += s_p[w][2][row][lane];
                }
                const float d = fmaf(uc[r], to_sig, to_dt * kLn2) * sx[r];  // A2 is A log2(e)
                dbias += d;
                dD = fmaf(gc[r], uc[r], dD);
                if (!on) continue;
                const int64_t o = int64_t(row) * p.ch;
                at_bytes(du + o, lane_off) = E::put(fmaf(Dc, gc[r], dc[r] * to_sig));
                at_bytes(ddt + o, lane_off) = E::put(d);
                if (Z) at_bytes(dz + o, lane_off) = E::put(oc[r] * y * dsilu(zc[r], sz[r]));
            }
            du -= int64_t(TT) * p.ch;
            ddt -= int64_t(TT) * p.ch;
            dz -= int64_t(TT) * p.ch;
            ckpt -= int64_t(p.N) * p.ch;
        }
    }
    __syncthreads();
    s_p[wave][0][0][lane] = AGG ? sum_dt : dD;
    s_p[wave][1][0][lane] = dbias;
    __syncthreads();
    if (!on) return;
    float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        sum0 += s_p[w][0][0][lane];
        sum1 += s_p[w][1][0][lane];
    }
    if constexpr (AGG) {
        const int64_t sb = int64_t(seg) * p.batch + b;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (n0 + k < p.N) p.seg_h[(sb * p.N + n0 + k) * p.ch + ch] = carry[k];
        if (wave == 0) p.seg_dt[sb * p.ch + ch] = sum0;
    } else {
        float* pa = p.part_a + (b * p.nseg + seg) * int64_t(p.N + 2) * p.ch + ch;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (n0 + k < p.N) pa[int64_t(n0 + k) * p.ch] = dA[k];
        if (wave == 0) {
            pa[int64_t(p.N) * p.ch] = sum0;
            pa[int64_t(p.N + 1) * p.ch] = sum1;
        }
        if (p.dh0 && seg == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (n0 + k < p.N) p.dh0[(b * p.ch + ch) * p.N + n0 + k] = carry[k];
        }
        const int64_t row0 = b * p.L * p.ch + ch;
        for (int64_t t = (last > first ? last : first) + wave; t < at.stop; t += NW) {
            static_cast<raw*>(p.du)[row0 + t * p.ch] = static_cast<raw*>(p.ddt)[row0 + t * p.ch] = E::put(0.0f);
            if (Z) static_cast<raw*>(p.dz)[row0 + t * p.ch] = E::put(0.0f);
        }
    }
}

// The sums that are left.  The first `blocks_a` workgroups: dA, dD and
// ddt_bias over sequences and segments, 64 adjacent values each, a quarter of
// the summands to a wave.  The others: dB and dC over the group's channel
// blocks, a thread to a value.
template <typename E>
__global__ __launch_bounds__(256) void scan_bwd_sums_kernel(ScanParams p, uint32_t blocks_a) {
    typedef typename E::raw raw;
    if (blockIdx.x < blocks_a) {
        __shared__ float s_sum[4][64];
        const int64_t per = int64_t(p.N + 2) * p.ch;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int64_t i = int64_t(blockIdx.x) * 64 + lane;
        const int rows = p.batch * p.nseg;
        float s = 0.0f;
        if (i < per) {
#pragma unroll 8
            for (int q = wave; q < rows; q += 4) s += p.part_a[q * per + i];
        }
        s_sum[wave][lane] = s;
        __syncthreads();
        if (wave != 0 || i >= per) return;
        s = (s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]);
        const int ch = int(i % p.ch), r = int(i / p.ch);
        if (r < p.N) p.dA[int64_t(ch) * p.N + r] = s;
        else if (r == p.N) { if (p.dD) p.dD[ch] = s; }
        else if (p.dbias) p.dbias[ch] = s;
        return;
    }
    const int64_t per = int64_t(p.batch) * p.L * p.G * 2 * p.N;
    const int64_t step = int64_t(gridDim.x - blocks_a) * 256;
    for (int64_t base = int64_t(blockIdx.x - blocks_a) * 256; base < per; base += step) {
        const int64_t i = base + threadIdx.x;
        if (i >= per) return;
        // the row (b, t, g) of the workgroup's first value, and from there in 32 bits
        const uint32_t j = uint32_t(base % (2 * p.N)) + threadIdx.x;
        const int64_t row = base / (2 * p.N) + j / uint32_t(2 * p.N);
        const uint32_t at = j % uint32_t(2 * p.N), n = at % uint32_t(p.N);
        bool counts = true;
        if (p.seqlens) {
            const int64_t bt = row / p.G;
            counts = bt % p.L < seq_end(p.seqlens, bt / p.L, p.L);
        }
        float s = 0.0f;
        if (counts) {
#pragma unroll 8
            for (int c = 0; c < p.bpg; ++c) s += p.part_bc[int64_t(c) * per + i];
        }
        static_cast<raw*>(at < uint32_t(p.N) ? p.dB : p.dC)[row * p.N + n] = E::put(s);
    }
}

template <typename E, int NW, bool Z>
int launch_bwd(const ScanParams& p, hipStream_t stream) {
    const uint32_t per_seg = uint32_t(p.bpg) * uint32_t(p.G) * uint32_t(p.batch);
    const dim3 block{NW * 64u, 1u, 1u};
    if (p.nseg > 1) {
        hipLaunchKernelGGL((scan_bwd_kernel<E, NW, true, Z>), dim3(per_seg * uint32_t(p.nseg - 1)), block, 0, stream, p);
        if (hipGetLastError() != hipSuccess) return -7;
    }
    hipLaunchKernelGGL((scan_bwd_kernel<E, NW, false, Z>), dim3(per_seg * uint32_t(p.nseg)), block, 0, stream, p);
    if (hipGetLastError() != hipSuccess) return -7;
    const int64_t blocks_bc = (int64_t(p.batch) * p.L * p.G * 2 * p.N + 255) / 256;
    const uint32_t blocks_a = uint32_t((int64_t(p.N + 2) * p.ch + 63) / 64);
    hipLaunchKernelGGL((scan_bwd_sums_kernel<E>), dim3(blocks_a + uint32_t(blocks_bc < 65536 ? blocks_bc : 65536)),
                       dim3(256), 0, stream, p, blocks_a);
    return hipGetLastError() == hipSuccess ? 0 : -7;
}

template <typename E, bool Z>
int launch_waves(const ScanParams& p, hipStream_t stream) {
    switch (scan_waves(p.N)) {
        case 1: return launch_bwd<E, 1, Z>(p, stream);
        case 2: return launch_bwd<E, 2, Z>(p, stream);
        case 4: return launch_bwd<E, 4, Z>(p, stream);
        case 8: return launch_bwd<E, 8, Z>(p, stream);
        default: return launch_bwd<E, 16, Z>(p, stream);
    }
}

template <typename E>
int launch_type(const ScanParams& p, hipStream_t stream) {
    return p.z ? launch_waves<E, true>(p, stream) : launch_waves<E, false>(p, stream);
}

}  // namespace
}  // namespace cls

int cls_selective_scan_bwd_launch(const cls::ScanParams& p, int dtype, hipStream_t stream) {
    return dtype == 0 ? cls::launch_type<cls::ElemF32>(p, stream)
         : dtype == 1 ? cls::launch_type<cls::ElemBF16>(p, stream)
                      : cls::launch_type<cls::ElemF16>(p, stream);
}
