// C ABI of the selective scan, the short convolution and the state cache:
// host-side checks, workspace sizes and the cut of the work.  Every argument
// is checked before anything is launched.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <cmath>

#include "../../include/selective_scan.h"
#include "launch_selective.hpp"
#include "selective_scan.hpp"

namespace {

using cls::ScanCut;
using cls::ScanParams;

constexpr int64_t kMaxThreads = int64_t(1) << 32;  // of a launch
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxStride = int64_t(1) << 40;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline uintptr_t elem_size(int dtype) { return dtype == SSD_F32 ? 4 : 2; }

bool dtype_ok(int d) { return d == SSD_F32 || d == SSD_BF16 || d == SSD_F16; }

bool strides_ok(const int64_t* s, int n) {
    for (int i = 0; i < n; ++i)
        if (s[i] < 0 || s[i] > kMaxStride) return false;
    return true;
}

// Where the channels and states alone give the device too few waves (below one
// per SIMD), each sequence is cut into segments, to 8 waves per SIMD where its
// length allows.  Output pass of 1 x 32768 x 4096 x 16 bf16 at 2048, 4096 and
// 8192 waves: 818, 632 and 570 us.  What bounds their number is that each starts
// by folding all before it, and that a second launch and pass are paid for: with
// the device nearly empty a call takes about 5 + 1.2 tiles us in one piece and
// 12.5 + 2.2 tiles / segments + 0.3 segments in several, so nothing is cut below
// 16 tiles and the best number is 2.7 roots of the tiles; with some waves on
// every SIMD fewer are better (2 x 1000 x 1536 x 16 fp32 in 11, 16, 21 and 32
// segments: 23.4, 22, 21.5 and 26 us).  The border of one wave per SIMD is not
// the best one: 8 x 2048 tokens of 1984 channels (cut) and of 2048 (whole) take
// 254 and 318 us forward and 523 and 851 us for the gradients, of 4096 (whole,
// two waves) 404 and 1048 us.  Nor is the most of 64 segments for long sequences
// of few channels: 1 x 65536 x 64 x 16 takes 272 us, where more would be faster
// by the formula above.
ScanCut scan_cut(int64_t batch, int64_t L, int64_t ch, int64_t N, int64_t G) {
    const int64_t tiles = ceil_div(L, cls::kScanTile);
    const int64_t waves = batch * G * ceil_div(ch / G, cls::kScanCh) * cls::scan_waves(N);
    int64_t nseg = 1;
    if (waves < 1024 && tiles >= 16) {
        const double root = std::sqrt(double(tiles));
        const int64_t three = 3 * 1024 / waves;  // segments that give each SIMD three waves
        const int64_t empty = int64_t(2.7 * root) < three ? int64_t(2.7 * root) : three;
        const int64_t full = int64_t(1.75 * root);
        nseg = ceil_div(8192, waves);
        for (int64_t most : {int64_t(cls::kScanMaxSegs), empty > full ? empty : full}) nseg = nseg < most ? nseg : most;
    }
    const int64_t len = ceil_div(tiles, nseg) * cls::kScanTile;
    return ScanCut{ceil_div(L, len), len};
}

// SSD_OK or the status of sizes that the scan, whole or one token, refuses.
int scan_dims(int64_t batch, int64_t L, int64_t ch, int64_t N, int64_t G) {
    if (batch <= 0 || L <= 0 || ch <= 0 || N <= 0 || G <= 0 || ch % G != 0) return SSD_ERR_SHAPE;
    if (batch > kMaxDim || L > kMaxTokens || ch > kMaxDim) return SSD_ERR_SHAPE;
    return N > cls::kScanMaxStates ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

// Of whole sequences: indexes are 64 bits wide, but for a launch's threads.
int scan_sizes(int64_t batch, int64_t L, int64_t ch, int64_t N, int64_t G) {
    const int st = scan_dims(batch, L, ch, N, G);
    if (st != SSD_OK) return st;
    if (batch * L > (int64_t(1) << 40) / ch) return SSD_ERR_SHAPE;
    const int64_t wgs = batch * G * ceil_div(ch / G, cls::kScanCh) * scan_cut(batch, L, ch, N, G).nseg;
    if (wgs * cls::scan_waves(N) * 64 >= kMaxThreads) return SSD_ERR_SHAPE;
    // the last sums of the gradients: four threads to a value of dA, dD and ddt_bias, and 65536 workgroups
    if (ch * (N + 2) > kMaxThreads / 4 - 65536 * 64 - 64) return SSD_ERR_SHAPE;
    return SSD_OK;
}

struct ScanSpace { size_t seg_h, seg_dt, fwd, part_bc, part_a, bwd; };  // offsets, and the totals

ScanSpace scan_space(int64_t batch, int64_t L, int64_t ch, int64_t N, int64_t G) {
    const ScanCut cut = scan_cut(batch, L, ch, N, G);
    ScanSpace s{};
    s.seg_dt = cut.nseg > 1 ? round_up(size_t(cut.nseg * batch * N * ch) * 4, 256) : 0;
    s.fwd = cut.nseg > 1 ? round_up(s.seg_dt + size_t(cut.nseg * batch * ch) * 4, 256) : 0;
    s.part_bc = s.fwd;
    const int64_t bpg = ceil_div(ch / G, cls::kScanCh);
    s.part_a = s.part_bc + round_up(size_t(bpg * batch * L * G * 2 * N) * 4, 256);
    s.bwd = s.part_a + round_up(size_t(batch * cut.nseg * (N + 2) * ch) * 4, 256);
    return s;
}

// The checks of what the forward and the backward pass, or one token (step), read.
int scan_check(const selective_scan_inputs* in, bool step = false) {
    if (!in || !in->u || !in->dt || !in->B || !in->C || !in->A) return SSD_ERR_NULL;
    if (!dtype_ok(in->dtype)) return SSD_ERR_DTYPE;
    const int st = (step ? scan_dims : scan_sizes)(in->batch, in->seqlen, in->channels, in->dstate, in->ngroups);
    if (st != SSD_OK) return st;
    if (step && cls_selective_scan_step_groups(*in) * 256 >= kMaxThreads) return SSD_ERR_SHAPE;
    const int64_t strides[] = {in->u_batch, in->u_token, in->dt_batch, in->dt_token, in->z_batch, in->z_token,
                               in->B_batch, in->B_token, in->B_group, in->C_batch, in->C_token, in->C_group};
    if (!strides_ok(strides, 12)) return SSD_ERR_SHAPE;
    for (int64_t s : {in->u_token, in->dt_token, in->z_token, in->B_token, in->C_token})
        if (s > cls::kScanMaxTokenStride) return SSD_ERR_SHAPE;
    for (const void* p : {in->u, in->dt, in->z, in->B, in->C})
        if (!aligned(p, elem_size(in->dtype))) return SSD_ERR_ALIGN;
    for (const float* p : {in->A, in->D, in->dt_bias, in->h0})
        if (!aligned(p, 4)) return SSD_ERR_ALIGN;
    return aligned(in->seqlens, 4) ? SSD_OK : SSD_ERR_ALIGN;
}

ScanParams scan_params(const selective_scan_inputs& in) {
    ScanParams p{};
    p.u = in.u; p.dt = in.dt; p.z = in.z; p.B = in.B; p.C = in.C;
    p.A = in.A; p.D = in.D; p.dt_bias = in.dt_bias; p.h0 = in.h0; p.seqlens = in.seqlens;
    p.su = {in.u_batch, in.u_token, 0};
    p.sdt = {in.dt_batch, in.dt_token, 0};
    p.sz = {in.z_batch, in.z_token, 0};
    p.sB = {in.B_batch, in.B_token, in.B_group};
    p.sC = {in.C_batch, in.C_token, in.C_group};
    p.batch = int(in.batch); p.L = int(in.seqlen); p.ch = int(in.channels);
    p.N = int(in.dstate); p.G = int(in.ngroups);
    p.cpg = p.ch / p.G;
    p.bpg = int(ceil_div(p.cpg, cls::kScanCh));
    const ScanCut cut = scan_cut(in.batch, in.seqlen, in.channels, in.dstate, in.ngroups);
    p.nseg = int(cut.nseg);
    p.seg_len = int(cut.seg_len);
    p.softplus = in.softplus;
    return p;
}

// SSD_OK or the status of sizes that the convolution refuses.
int conv_sizes(int64_t batch, int64_t L, int64_t ch, int64_t W) {
    if (batch <= 0 || L <= 0 || ch <= 0 || W <= 0) return SSD_ERR_SHAPE;
    if (batch > kMaxDim || L > kMaxTokens || ch > kMaxDim) return SSD_ERR_SHAPE;
    if (W < 2 || W > 4) return SSD_ERR_UNSUPPORTED;
    // a thread per channel and four tokens, and for the final state; workgroups of 256
    if (batch * (ceil_div(L, 4) + 1) >= (kMaxThreads - 256) / (ch + 64)) return SSD_ERR_SHAPE;
    return SSD_OK;
}

int conv_check(const short_conv_inputs* in) {
    if (!in || !in->x || !in->weight) return SSD_ERR_NULL;
    if (!dtype_ok(in->dtype)) return SSD_ERR_DTYPE;
    const int st = conv_sizes(in->batch, in->seqlen, in->channels, in->width);
    if (st != SSD_OK) return st;
    const int64_t strides[] = {in->x_batch, in->x_token};
    if (!strides_ok(strides, 2)) return SSD_ERR_SHAPE;
    if (!aligned(in->x, elem_size(in->dtype)) || !aligned(in->initial_state, elem_size(in->dtype))) return SSD_ERR_ALIGN;
    if (!aligned(in->weight, 4) || !aligned(in->bias, 4) || !aligned(in->seqlens, 4)) return SSD_ERR_ALIGN;
    return SSD_OK;
}

size_t conv_space(int64_t batch, int64_t L, int64_t ch, int64_t W) {
    return size_t(cls_short_conv_bwd_parts(batch, L, ch)) * size_t(ch) * size_t(W + 1) * 4;
}

int cache_check(const void* h, const int32_t* slots, int64_t batch, int64_t rows, int64_t S, int64_t nslots, int format,
                const void* cache, const float* scales) {
    if (!h || !slots || !cache || !scales) return SSD_ERR_NULL;
    if (format != SSD_I8 && format != SSD_E4M3) return SSD_ERR_DTYPE;
    if (batch <= 0 || rows <= 0 || S <= 0 || nslots <= 0) return SSD_ERR_SHAPE;
    if (batch > kMaxDim || rows > kMaxThreads || nslots > (int64_t(1) << 31) - 1) return SSD_ERR_SHAPE;
    if (S > 256) return SSD_ERR_UNSUPPORTED;
    if (batch * (rows + 256) >= kMaxThreads / 64 || nslots > (int64_t(1) << 46) / (rows * S)) return SSD_ERR_SHAPE;
    if (!aligned(h, 4) || !aligned(slots, 4) || !aligned(scales, 4)) return SSD_ERR_ALIGN;
    return SSD_OK;
}

int launched(int st) { return st == 0 ? SSD_OK : SSD_ERR_HIP; }

}  // namespace

extern "C" {

size_t selective_scan_workspace_size(int64_t batch, int64_t seqlen, int64_t channels, int64_t dstate, int64_t ngroups) {
    if (scan_sizes(batch, seqlen, channels, dstate, ngroups) != SSD_OK) return 0;
    return scan_space(batch, seqlen, channels, dstate, ngroups).fwd;
}

size_t selective_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t channels, int64_t dstate,
                                         int64_t ngroups) {
    if (scan_sizes(batch, seqlen, channels, dstate, ngroups) != SSD_OK) return 0;
    return scan_space(batch, seqlen, channels, dstate, ngroups).bwd;
}

size_t selective_scan_checkpoint_size(int64_t batch, int64_t seqlen, int64_t channels, int64_t dstate) {
    if (scan_sizes(batch, seqlen, channels, dstate, 1) != SSD_OK) return 0;
    return size_t(batch * ceil_div(seqlen, cls::kScanTile)) * size_t(dstate * channels) * 4;
}

int selective_scan_fwd(const selective_scan_inputs* in, void* y, float* h_final, void* checkpoints, void* workspace,
                       size_t workspace_bytes, void* stream) {
    if (!y) return SSD_ERR_NULL;
    const int st = scan_check(in);
    if (st != SSD_OK) return st;
    if (!aligned(y, elem_size(in->dtype)) || !aligned(h_final, 4) || !aligned(checkpoints, 16) || !aligned(workspace, 16))
        return SSD_ERR_ALIGN;
    const ScanSpace s = scan_space(in->batch, in->seqlen, in->channels, in->dstate, in->ngroups);
    if (s.fwd > 0 && (!workspace || workspace_bytes < s.fwd)) return SSD_ERR_WORKSPACE;
    ScanParams p = scan_params(*in);
    p.y = y;
    p.h_last = h_final;
    p.ckpt = static_cast<float*>(checkpoints);
    char* ws = static_cast<char*>(workspace);
    p.seg_h = reinterpret_cast<float*>(ws + s.seg_h);
    p.seg_dt = reinterpret_cast<float*>(ws + s.seg_dt);
    return launched(cls_selective_scan_fwd_launch(p, in->dtype, static_cast<hipStream_t>(stream)));
}

int selective_scan_bwd(const selective_scan_inputs* in, const selective_scan_grads* g, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const int st = scan_check(in);
    if (st != SSD_OK) return st;
    if (!g || !g->dy || !g->checkpoints || !g->du || !g->ddt || !g->dB || !g->dC || !g->dA || !workspace ||
        (in->z && !g->dz))
        return SSD_ERR_NULL;
    const int64_t strides[] = {g->dy_batch, g->dy_token};
    if (!strides_ok(strides, 2) || g->dy_token > cls::kScanMaxTokenStride) return SSD_ERR_SHAPE;
    for (const void* p : {g->dy, static_cast<const void*>(g->du), static_cast<const void*>(g->ddt),
                          static_cast<const void*>(g->dz), static_cast<const void*>(g->dB), static_cast<const void*>(g->dC)})
        if (!aligned(p, elem_size(in->dtype))) return SSD_ERR_ALIGN;
    for (const float* p : {g->dh_final, static_cast<const float*>(g->dA), static_cast<const float*>(g->dD),
                           static_cast<const float*>(g->ddt_bias), static_cast<const float*>(g->dh0)})
        if (!aligned(p, 4)) return SSD_ERR_ALIGN;
    if (!aligned(g->checkpoints, 16) || !aligned(workspace, 16)) return SSD_ERR_ALIGN;
    const ScanSpace s = scan_space(in->batch, in->seqlen, in->channels, in->dstate, in->ngroups);
    if (workspace_bytes < s.bwd) return SSD_ERR_WORKSPACE;
    ScanParams p = scan_params(*in);
    p.dy = g->dy;
    p.sdy = {g->dy_batch, g->dy_token, 0};
    p.dh_last = g->dh_final;
    p.ckpt = static_cast<float*>(const_cast<void*>(g->checkpoints));
    p.du = g->du; p.ddt = g->ddt; p.dz = g->dz; p.dB = g->dB; p.dC = g->dC;
    p.dA = g->dA; p.dD = g->dD; p.dbias = g->ddt_bias; p.dh0 = g->dh0;
    char* ws = static_cast<char*>(workspace);
    p.seg_h = reinterpret_cast<float*>(ws + s.seg_h);
    p.seg_dt = reinterpret_cast<float*>(ws + s.seg_dt);
    p.part_bc = reinterpret_cast<float*>(ws + s.part_bc);
    p.part_a = reinterpret_cast<float*>(ws + s.part_a);
    return launched(cls_selective_scan_bwd_launch(p, in->dtype, static_cast<hipStream_t>(stream)));
}

int selective_scan_step(const selective_scan_inputs* in, float* h, void* y, void* stream) {
    if (!in || !h || !y) return SSD_ERR_NULL;
    selective_scan_inputs one = *in;
    one.seqlen = 1;
    one.u_token = one.dt_token = one.z_token = one.B_token = one.C_token = 0;
    one.h0 = nullptr;
    one.seqlens = nullptr;
    const int st = scan_check(&one, true);
    if (st != SSD_OK) return st;
    // whole vectors of states only where every row starts on one
    if (!aligned(h, one.dstate % 4 == 0 ? 16 : 4) || !aligned(y, elem_size(one.dtype))) return SSD_ERR_ALIGN;
    return launched(cls_selective_scan_step_launch(one, h, y, static_cast<hipStream_t>(stream)));
}

int short_conv_fwd(const short_conv_inputs* in, void* y, void* final_state, void* stream) {
    if (!y) return SSD_ERR_NULL;
    const int st = conv_check(in);
    if (st != SSD_OK) return st;
    if (!aligned(y, elem_size(in->dtype)) || !aligned(final_state, elem_size(in->dtype))) return SSD_ERR_ALIGN;
    return launched(cls_short_conv_fwd_launch(*in, y, final_state, static_cast<hipStream_t>(stream)));
}

size_t short_conv_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t channels, int64_t width) {
    if (conv_sizes(batch, seqlen, channels, width) != SSD_OK) return 0;
    return conv_space(batch, seqlen, channels, width);
}

int short_conv_bwd(const short_conv_inputs* in, const void* dy, int64_t dy_batch, int64_t dy_token, const void* dfinal,
                   void* dx, float* dweight, float* dbias, void* dinitial, void* workspace, size_t workspace_bytes,
                   void* stream) {
    if (!dy || !dx || !workspace) return SSD_ERR_NULL;
    const int st = conv_check(in);
    if (st != SSD_OK) return st;
    const int64_t strides[] = {dy_batch, dy_token};
    if (!strides_ok(strides, 2)) return SSD_ERR_SHAPE;
    const void* elems[] = {dy, dfinal, dx, dinitial};
    for (const void* p : elems)
        if (!aligned(p, elem_size(in->dtype))) return SSD_ERR_ALIGN;
    if (!aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(workspace, 16)) return SSD_ERR_ALIGN;
    if (workspace_bytes < conv_space(in->batch, in->seqlen, in->channels, in->width)) return SSD_ERR_WORKSPACE;
    return launched(cls_short_conv_bwd_launch(*in, dy, dy_batch, dy_token, dfinal, dx, dweight, dbias, dinitial,
                                              static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

int short_conv_step(const short_conv_inputs* in, void* state, void* y, void* stream) {
    if (!in || !state || !y) return SSD_ERR_NULL;
    short_conv_inputs one = *in;
    one.seqlen = 1;
    one.x_token = 0;
    one.initial_state = nullptr;
    one.seqlens = nullptr;
    const int st = conv_check(&one);
    if (st != SSD_OK) return st;
    if (!aligned(state, elem_size(one.dtype)) || !aligned(y, elem_size(one.dtype))) return SSD_ERR_ALIGN;
    return launched(cls_short_conv_step_launch(one, state, y, static_cast<hipStream_t>(stream)));
}

int state_cache_write(const float* h, const int32_t* slots, int64_t batch, int64_t rows, int64_t dstate, int64_t nslots,
                      int format, void* cache, float* scales, void* stream) {
    const int st = cache_check(h, slots, batch, rows, dstate, nslots, format, cache, scales);
    if (st != SSD_OK) return st;
    return launched(cls_state_cache_write_launch(h, slots, batch, rows, dstate, nslots, format, cache, scales,
                                                 static_cast<hipStream_t>(stream)));
}

int state_cache_read(const void* cache, const float* scales, const int32_t* slots, int64_t batch, int64_t rows,
                     int64_t dstate, int64_t nslots, int format, float* h, void* stream) {
    const int st = cache_check(h, slots, batch, rows, dstate, nslots, format, cache, scales);
    if (st != SSD_OK) return st;
    return launched(cls_state_cache_read_launch(cache, scales, slots, batch, rows, dstate, nslots, format, h,
                                                static_cast<hipStream_t>(stream)));
}

}  // extern "C"
