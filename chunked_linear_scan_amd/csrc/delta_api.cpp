// C ABI of the gated delta rule and of the norms around its block: host-side
// checks, workspace sizes and launches.  Every argument is checked before
// anything is launched.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <initializer_list>

#include "../../include/gated_delta.h"
#include "delta.hpp"
#include "launch_delta.hpp"

namespace {

using cls::DeltaParams;

constexpr int64_t kMaxThreads = int64_t(1) << 32;  // of a launch
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxBatch = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 40;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline uintptr_t elem_size(int dtype) { return dtype == SSD_F32 ? 4 : 2; }
inline int64_t chunk_of(int dtype) { return dtype == SSD_F32 ? 32 : 64; }
bool dtype_ok(int d) { return d == SSD_F32 || d == SSD_BF16 || d == SSD_F16; }

bool strides_ok(std::initializer_list<int64_t> strides) {
    for (int64_t s : strides)
        if (s < 0 || s > kMaxStride) return false;
    return true;
}

// Rows of a strided activation start on 16-byte vectors and hold whole ones.
template <typename... S>
uint8_t whole_vectors(const void* p, int64_t dim, int dtype, S... strides) {
    const int64_t ve = 16 / int64_t(elem_size(dtype));
    return aligned(p, 16) && dim % ve == 0 && ((strides % ve == 0) && ...);
}

// A copied row's length.
int64_t padded(int64_t dim, int dtype) {
    const int64_t ve = 16 / int64_t(elem_size(dtype));
    return ceil_div(dim, ve) * ve;
}

// SSD_OK or the status of sizes that are refused.
int delta_dims(const gated_delta_inputs& s) {
    if (!dtype_ok(s.dtype)) return SSD_ERR_DTYPE;
    if (s.batch <= 0 || s.seqlen <= 0 || s.kheads <= 0 || s.heads <= 0 || s.dk <= 0 || s.dv <= 0) return SSD_ERR_SHAPE;
    if (s.heads % s.kheads != 0 || s.batch > kMaxBatch || s.heads > kMaxBatch || s.seqlen > kMaxTokens) return SSD_ERR_SHAPE;
    return s.dk > 256 || s.dv > 65536 ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

int delta_sizes(const gated_delta_inputs& s) {
    const int st = delta_dims(s);
    if (st != SSD_OK) return st;
    if (s.heads * padded(s.dv, s.dtype) > cls::kDeltaMaxToken || s.kheads * 256 > cls::kDeltaMaxToken) return SSD_ERR_SHAPE;
    const int64_t heads = s.batch * s.heads;
    if (heads * ceil_div(s.dv, 32) >= kMaxThreads / 512) return SSD_ERR_SHAPE;
    if (heads >= ceil_div(kMaxThreads / 256, ceil_div(s.seqlen, chunk_of(s.dtype)))) return SSD_ERR_SHAPE;
    return SSD_OK;
}

// What is read of the inputs, by a pass over sequences or by one token (step).
int delta_check(const gated_delta_inputs* in, bool step) {
    if (!in || !in->q || !in->k || !in->v || !in->g || !in->beta) return SSD_ERR_NULL;
    const int st = (step ? delta_dims : delta_sizes)(*in);
    if (st != SSD_OK) return st;
    if (step && cls_delta_step_groups(in->batch * in->heads, in->dk, in->dv) >= kMaxThreads / 256) return SSD_ERR_SHAPE;
    if (!strides_ok({in->q_batch, in->q_token, in->q_head, in->k_batch, in->k_token, in->k_head, in->v_batch, in->v_token,
                     in->v_head, in->g_batch, in->g_token, in->beta_batch, in->beta_token}))
        return SSD_ERR_SHAPE;
    for (const void* p : {in->q, in->k, in->v})
        if (!aligned(p, elem_size(in->dtype))) return SSD_ERR_ALIGN;
    for (const float* p : {in->g, in->beta, in->h0})
        if (!aligned(p, 4)) return SSD_ERR_ALIGN;
    return aligned(in->seqlens, 4) ? SSD_OK : SSD_ERR_ALIGN;
}

// Whether the kernels read an activation's rows where they are: tokens apart by a row or more and no further than
// their offsets reach, in whole 16-byte vectors.  Others are copied into the workspace.
bool in_place(const void* p, int64_t L, int64_t dim, int dtype, int64_t batch, int64_t token, int64_t head) {
    if (L > 1 && (token < dim || token > cls::kDeltaMaxToken)) return false;
    return whole_vectors(p, dim, dtype, batch, L > 1 ? token : 0, head);
}

// Offsets in the workspaces and checkpoints, and their sizes.
struct DeltaSpace {
    bool pack_q, pack_k, pack_v;
    size_t mats, vecs, q, k, v, fwd;             // both passes: matrices and factors of the chunks, copies
    size_t fixes, ckpt;                          // checkpoints: states, then corrections
    size_t dstates, z, part_q, part_k, dy, sizes, bwd;  // backward
};

DeltaSpace delta_space(const gated_delta_inputs& s) {
    const int64_t C = chunk_of(s.dtype), n = s.batch * s.heads * ceil_div(s.seqlen, C), rows = s.batch * s.seqlen;
    const size_t mat = size_t(C * C) * elem_size(s.dtype) * (s.dtype == SSD_F32 ? 2 : 4);
    const size_t keys = round_up(size_t(rows * s.kheads * padded(s.dk, s.dtype)) * elem_size(s.dtype), 256);
    const size_t values = round_up(size_t(rows * s.heads * padded(s.dv, s.dtype)) * elem_size(s.dtype), 256);
    DeltaSpace d{};
    d.pack_q = !in_place(s.q, s.seqlen, s.dk, s.dtype, s.q_batch, s.q_token, s.q_head);
    d.pack_k = !in_place(s.k, s.seqlen, s.dk, s.dtype, s.k_batch, s.k_token, s.k_head);
    d.pack_v = !in_place(s.v, s.seqlen, s.dv, s.dtype, s.v_batch, s.v_token, s.v_head);
    d.vecs = round_up(size_t(n) * mat, 256);
    d.q = d.vecs + round_up(size_t(n) * cls::kVecs * C * 4, 256);
    d.k = d.q + (d.pack_q ? keys : 0);
    d.v = d.k + (d.pack_k ? keys : 0);
    d.fwd = d.v + (d.pack_v ? values : 0);
    const size_t states = round_up(size_t(n) * round_up(size_t(s.dk), 4) * s.dv * 4, 256);
    const size_t tokens = round_up(size_t(n) * s.dv * C * 4, 256);
    const size_t parts = s.heads > s.kheads ? round_up(size_t(rows * s.heads) * s.dk * 4, 256) : 0;
    d.fixes = states;
    d.ckpt = states + tokens;
    d.dstates = d.fwd;
    d.z = d.dstates + states;
    d.part_q = d.z + tokens;
    d.part_k = d.part_q + parts;
    d.dy = d.part_k + parts;
    d.sizes = d.dy + values;
    d.bwd = d.sizes + (s.dtype == SSD_F16 ? size_t(s.batch * s.heads) * 2 * cls::kSizes * 4 : 0);
    return d;
}

DeltaParams delta_params(const gated_delta_inputs& in, void* workspace, void* checkpoints, const DeltaSpace& s) {
    DeltaParams p{};
    p.g = in.g; p.beta = in.beta; p.h0 = in.h0; p.seqlens = in.seqlens;
    p.g_batch = in.g_batch; p.g_token = in.g_token; p.b_batch = in.beta_batch; p.b_token = in.beta_token;
    p.batch = int(in.batch); p.L = int(in.seqlen); p.Hk = int(in.kheads); p.H = int(in.heads);
    p.dk = int(in.dk); p.dv = int(in.dv); p.kpitch = (p.dk + 3) / 4 * 4;
    p.nchunk = int(ceil_div(in.seqlen, chunk_of(in.dtype)));
    p.scale = in.scale;
    char* ws = static_cast<char*>(workspace);
    const auto place = [&](const void* given, bool copied, size_t at, int64_t heads, int64_t dim, cls::Strided3 given_strides,
                           const void*& to, cls::Strided3& strides) {
        to = copied ? ws + at : given;
        if (copied) strides = {in.seqlen * heads * dim, heads * dim, dim};
        else strides = {given_strides.batch, in.seqlen > 1 ? given_strides.token : heads * dim, given_strides.head};
    };
    place(in.q, s.pack_q, s.q, in.kheads, padded(in.dk, in.dtype), {in.q_batch, in.q_token, in.q_head}, p.q, p.sq);
    place(in.k, s.pack_k, s.k, in.kheads, padded(in.dk, in.dtype), {in.k_batch, in.k_token, in.k_head}, p.k, p.sk);
    place(in.v, s.pack_v, s.v, in.heads, padded(in.dv, in.dtype), {in.v_batch, in.v_token, in.v_head}, p.v, p.sv);
    p.mats = ws + s.mats;
    p.vecs = reinterpret_cast<float*>(ws + s.vecs);
    if (checkpoints) {
        p.states = static_cast<float*>(checkpoints);
        p.fixes = reinterpret_cast<float*>(static_cast<char*>(checkpoints) + s.fixes);
    }
    return p;
}

// The copies, where there are any.
int delta_pack(const gated_delta_inputs& in, void* workspace, const DeltaSpace& s, hipStream_t stream) {
    char* ws = static_cast<char*>(workspace);
    const int64_t size = int64_t(elem_size(in.dtype)), dk = padded(in.dk, in.dtype);
    int st = 0;
    if (s.pack_q)
        st = cls_delta_pack_launch(in.q, ws + s.q, size, in.batch, in.seqlen, in.kheads, in.dk, dk, in.q_batch, in.q_token,
                                   in.q_head, stream);
    if (st == 0 && s.pack_k)
        st = cls_delta_pack_launch(in.k, ws + s.k, size, in.batch, in.seqlen, in.kheads, in.dk, dk, in.k_batch, in.k_token,
                                   in.k_head, stream);
    if (st == 0 && s.pack_v)
        st = cls_delta_pack_launch(in.v, ws + s.v, size, in.batch, in.seqlen, in.heads, in.dv, padded(in.dv, in.dtype), in.v_batch, in.v_token,
                                   in.v_head, stream);
    return st;
}

constexpr int64_t kMaxNormDim = 16384;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

int norm_sizes(int64_t rows, int64_t heads, int64_t dim) {
    if (rows <= 0 || heads <= 0 || dim <= 0 || rows > kMaxRows || heads > kMaxRows / rows) return SSD_ERR_SHAPE;
    return dim > kMaxNormDim ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

int gated_check(const gated_norm_inputs* in) {
    if (!in || !in->x) return SSD_ERR_NULL;
    if (!dtype_ok(in->dtype)) return SSD_ERR_DTYPE;
    const int st = norm_sizes(in->rows, in->heads, in->dim);
    if (st != SSD_OK) return st;
    if (!strides_ok({in->x_row, in->x_head, in->z_row, in->z_head})) return SSD_ERR_SHAPE;
    if (!aligned(in->x, elem_size(in->dtype)) || !aligned(in->z, elem_size(in->dtype)) || !aligned(in->weight, 4))
        return SSD_ERR_ALIGN;
    return SSD_OK;
}

int residual_check(const residual_norm_inputs* in) {
    if (!in) return SSD_ERR_NULL;
    if (!dtype_ok(in->dtype) || (in->stream_dtype != SSD_F32 && in->stream_dtype != in->dtype)) return SSD_ERR_DTYPE;
    const int st = norm_sizes(in->rows, 1, in->dim);
    if (st != SSD_OK) return st;
    if (!strides_ok({in->x_row, in->residual_row})) return SSD_ERR_SHAPE;
    if (!aligned(in->x, elem_size(in->dtype)) || !aligned(in->residual, elem_size(in->stream_dtype)) ||
        !aligned(in->scale, 4) || !aligned(in->weight, 4))
        return SSD_ERR_ALIGN;
    return SSD_OK;
}

int launched(int st) { return st == 0 ? SSD_OK : SSD_ERR_HIP; }

}  // namespace

extern "C" {

int64_t gated_delta_chunk(int dtype) { return dtype_ok(dtype) ? chunk_of(dtype) : 0; }

size_t gated_delta_workspace_size(const gated_delta_inputs* in) {
    return in && delta_sizes(*in) == SSD_OK ? delta_space(*in).fwd : 0;
}

size_t gated_delta_bwd_workspace_size(const gated_delta_inputs* in) {
    return in && delta_sizes(*in) == SSD_OK ? delta_space(*in).bwd : 0;
}

size_t gated_delta_checkpoint_size(const gated_delta_inputs* in) {
    return in && delta_sizes(*in) == SSD_OK ? delta_space(*in).ckpt : 0;
}

int gated_delta_fwd(const gated_delta_inputs* in, void* y, float* h_final, void* checkpoints, void* workspace,
                    size_t workspace_bytes, void* stream) {
    if (!y) return SSD_ERR_NULL;
    const int st = delta_check(in, false);
    if (st != SSD_OK) return st;
    if (!aligned(y, elem_size(in->dtype)) || !aligned(h_final, 4) || !aligned(checkpoints, 16) || !aligned(workspace, 16))
        return SSD_ERR_ALIGN;
    const DeltaSpace s = delta_space(*in);
    if (!workspace || workspace_bytes < s.fwd) return SSD_ERR_WORKSPACE;
    DeltaParams p = delta_params(*in, workspace, checkpoints, s);
    p.y = y;
    p.vec_out = whole_vectors(y, in->dv, in->dtype);
    p.h_last = h_final;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    int rc = delta_pack(*in, workspace, s, hs);
    if (rc == 0) rc = cls_delta_prep_launch(p, in->dtype, hs);
    if (rc == 0) rc = cls_delta_fwd_launch(p, in->dtype, hs);
    return launched(rc);
}

int gated_delta_bwd(const gated_delta_inputs* in, const gated_delta_grads* g, void* workspace, size_t workspace_bytes,
                    void* stream) {
    const int st = delta_check(in, false);
    if (st != SSD_OK) return st;
    if (!g || !g->dy || !g->checkpoints || !g->dq || !g->dk || !g->dv || !g->dg || !g->dbeta) return SSD_ERR_NULL;
    if (!strides_ok({g->dy_batch, g->dy_token, g->dy_head})) return SSD_ERR_SHAPE;
    if (in->heads > in->kheads && in->batch * in->seqlen >= kMaxThreads / (in->kheads * in->dk)) return SSD_ERR_SHAPE;
    for (const void* p : {g->dy, static_cast<const void*>(g->dq), static_cast<const void*>(g->dk),
                          static_cast<const void*>(g->dv)})
        if (!aligned(p, elem_size(in->dtype))) return SSD_ERR_ALIGN;
    for (const float* p : {g->dh_final, static_cast<const float*>(g->dg), static_cast<const float*>(g->dbeta),
                           static_cast<const float*>(g->dh0)})
        if (!aligned(p, 4)) return SSD_ERR_ALIGN;
    if (!aligned(g->checkpoints, 16) || !aligned(workspace, 16)) return SSD_ERR_ALIGN;
    const DeltaSpace s = delta_space(*in);
    if (!workspace || workspace_bytes < s.bwd) return SSD_ERR_WORKSPACE;
    DeltaParams p = delta_params(*in, workspace, const_cast<void*>(g->checkpoints), s);
    char* ws = static_cast<char*>(workspace);
    const bool pack_dy = !in_place(g->dy, in->seqlen, in->dv, in->dtype, g->dy_batch, g->dy_token, g->dy_head);
    const int64_t dv = padded(in->dv, in->dtype), row = in->heads * dv;
    p.dy = pack_dy ? ws + s.dy : g->dy;
    if (pack_dy) p.sdy = {in->seqlen * row, row, dv};
    else p.sdy = {g->dy_batch, in->seqlen > 1 ? g->dy_token : row, g->dy_head};
    p.vec_out = whole_vectors(g->dv, in->dv, in->dtype);
    p.vec_dqk = aligned(g->dq, 16) && aligned(g->dk, 16);
    p.dh_last = g->dh_final;
    p.dq = g->dq; p.dk_ = g->dk; p.dv_ = g->dv; p.dg = g->dg; p.dbeta = g->dbeta; p.dh0 = g->dh0;
    p.dstates = reinterpret_cast<float*>(ws + s.dstates);
    p.z = reinterpret_cast<float*>(ws + s.z);
    p.part_q = reinterpret_cast<float*>(ws + s.part_q);
    p.part_k = reinterpret_cast<float*>(ws + s.part_k);
    p.sizes = reinterpret_cast<float*>(ws + s.sizes);
    // parts of a head, so that a few heads have workgroups for the whole device, too
    const int64_t heads = in->batch * in->heads, parts = 2048 / heads;
    p.nsize = int(parts < 1 ? 1 : parts < cls::kSizes ? parts : cls::kSizes);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    int rc = delta_pack(*in, workspace, s, hs);
    if (rc == 0 && pack_dy)
        rc = cls_delta_pack_launch(g->dy, ws + s.dy, int64_t(elem_size(in->dtype)), in->batch, in->seqlen, in->heads, in->dv,
                                   dv, g->dy_batch, g->dy_token, g->dy_head, hs);
    if (rc == 0) rc = cls_delta_prep_launch(p, in->dtype, hs);
    if (rc == 0 && in->dtype == SSD_F16) rc = cls_delta_size_launch(p, hs);
    if (rc == 0) rc = cls_delta_bwd_launch(p, in->dtype, hs);
    if (rc == 0) rc = cls_delta_grad_launch(p, in->dtype, hs);
    return launched(rc);
}

int gated_delta_step(const gated_delta_inputs* in, float* h, void* y, void* stream) {
    if (!in || !h || !y) return SSD_ERR_NULL;
    gated_delta_inputs one = *in;
    one.seqlen = 1;
    one.q_token = one.k_token = one.v_token = one.g_token = one.beta_token = 0;
    one.h0 = nullptr;
    one.seqlens = nullptr;
    const int st = delta_check(&one, true);
    if (st != SSD_OK) return st;
    if (!aligned(h, one.dk % 4 == 0 ? 16 : 4) || !aligned(y, elem_size(one.dtype))) return SSD_ERR_ALIGN;
    return launched(cls_delta_step_launch(one, h, y, static_cast<hipStream_t>(stream)));
}

int gated_norm_fwd(const gated_norm_inputs* in, void* y, float* rstd, void* stream) {
    if (!y) return SSD_ERR_NULL;
    const int st = gated_check(in);
    if (st != SSD_OK) return st;
    if (!aligned(y, elem_size(in->dtype)) || !aligned(rstd, 4)) return SSD_ERR_ALIGN;
    return launched(cls_gated_norm_launch(*in, nullptr, 0, 0, rstd, y, nullptr, nullptr, nullptr, nullptr,
                                          static_cast<hipStream_t>(stream)));
}

size_t gated_norm_bwd_workspace_size(int64_t rows, int64_t heads, int64_t dim) {
    if (norm_sizes(rows, heads, dim) != SSD_OK) return 0;
    return size_t(cls_norm_parts(rows * heads, dim)) * size_t(dim) * 4;
}

int gated_norm_bwd(const gated_norm_inputs* in, const void* dy, int64_t dy_row, int64_t dy_head, const float* rstd,
                   void* dx, void* dz, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    const int st = gated_check(in);
    if (st != SSD_OK) return st;
    if (!dy || !rstd || !dx || (in->z && !dz)) return SSD_ERR_NULL;
    if (!strides_ok({dy_row, dy_head})) return SSD_ERR_SHAPE;
    for (const void* p : {dy, static_cast<const void*>(dx), static_cast<const void*>(dz)})
        if (!aligned(p, elem_size(in->dtype))) return SSD_ERR_ALIGN;
    if (!aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(workspace, 16)) return SSD_ERR_ALIGN;
    if (dweight && (!workspace || workspace_bytes < gated_norm_bwd_workspace_size(in->rows, in->heads, in->dim)))
        return SSD_ERR_WORKSPACE;
    return launched(cls_gated_norm_launch(*in, dy, dy_row, dy_head, const_cast<float*>(rstd), nullptr, dx,
                                          in->z ? dz : nullptr, dweight, static_cast<float*>(workspace),
                                          static_cast<hipStream_t>(stream)));
}

int residual_norm_fwd(const residual_norm_inputs* in, void* y, void* r, float* rstd, void* stream) {
    if (!in || !in->x || !y || !r) return SSD_ERR_NULL;
    const int st = residual_check(in);
    if (st != SSD_OK) return st;
    if (!aligned(y, elem_size(in->dtype)) || !aligned(r, elem_size(in->stream_dtype)) || !aligned(rstd, 4))
        return SSD_ERR_ALIGN;
    return launched(cls_residual_norm_fwd_launch(*in, y, r, rstd, static_cast<hipStream_t>(stream)));
}

size_t residual_norm_bwd_workspace_size(int64_t rows, int64_t dim) {
    if (norm_sizes(rows, 1, dim) != SSD_OK) return 0;
    return size_t(cls_norm_parts(rows, dim)) * size_t(dim) * 8;
}

int residual_norm_bwd(const residual_norm_inputs* in, const residual_norm_grads* g, void* workspace,
                      size_t workspace_bytes, void* stream) {
    const int st = residual_check(in);
    if (st != SSD_OK) return st;
    if (!g || !g->dy || !g->r || !g->rstd || !g->dresidual || (g->dscale && !in->x)) return SSD_ERR_NULL;
    if (!strides_ok({g->dy_row, g->dr_row, g->r_row})) return SSD_ERR_SHAPE;
    for (const void* p : {g->dy, static_cast<const void*>(g->dx)})
        if (!aligned(p, elem_size(in->dtype))) return SSD_ERR_ALIGN;
    for (const void* p : {g->dr, g->r, static_cast<const void*>(g->dresidual)})
        if (!aligned(p, elem_size(in->stream_dtype))) return SSD_ERR_ALIGN;
    if (!aligned(g->rstd, 4) || !aligned(g->dweight, 4) || !aligned(g->dscale, 4) || !aligned(workspace, 16))
        return SSD_ERR_ALIGN;
    if ((g->dweight || g->dscale) &&
        (!workspace || workspace_bytes < residual_norm_bwd_workspace_size(in->rows, in->dim)))
        return SSD_ERR_WORKSPACE;
    return launched(cls_residual_norm_bwd_launch(*in, *g, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
