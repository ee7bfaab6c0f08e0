// Python binding of include/gated_delta.h, in the manner of selective_binding.cpp:
// checks, allocations and the call, on torch's current stream of the inputs' device.
#include "../../include/gated_delta.h"
#include "common.hpp"

#include <cmath>

namespace {

// ---------------------------------------------------------------------------
// gated delta rule
// ---------------------------------------------------------------------------
gated_delta_inputs delta_inputs(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g, const Tensor& beta,
                                const Maybe& h0, const Maybe& seqlens, const std::optional<double>& scale, bool step) {
    gated_delta_inputs s{};
    s.dtype = check_lead("v", v, step ? 3 : 4, step ? "batch, heads, dv" : "batch, seqlen, heads, dv");
    const at::Device dev = v.device();
    const at::ScalarType kind = v.scalar_type();
    check_dims("q", q, step ? 3 : 4, step ? "batch, kheads, dk" : "batch, seqlen, kheads, dk");
    s.batch = v.size(0);
    s.seqlen = step ? 1 : v.size(1);
    s.heads = v.size(-2);
    s.dv = v.size(-1);
    s.kheads = q.size(-2);
    s.dk = q.size(-1);
    const int64_t keys[] = {s.batch, s.seqlen, s.kheads, s.dk}, keys1[] = {s.batch, s.kheads, s.dk};
    const at::IntArrayRef of = step ? at::IntArrayRef(keys1, 3) : at::IntArrayRef(keys, 4);
    check("q", q, dev, kind, of, true);
    check("k", k, dev, kind, of, true);
    const at::IntArrayRef each = v.sizes().slice(0, step ? 2 : 3);
    check("g", g, dev, at::kFloat, each, true);
    check("beta", beta, dev, at::kFloat, each, true);
    check("h0", h0, dev, at::kFloat, {s.batch, s.heads, s.dv, s.dk});
    check("seqlens", seqlens, dev, at::kInt, {s.batch});
    s.scale = scale ? float(*scale) : s.dk > 0 ? float(1 / std::sqrt(double(s.dk))) : 0.0f;
    s.q = ptr(q); s.k = ptr(k); s.v = ptr(v);
    s.g = ptr<float>(g); s.beta = ptr<float>(beta); s.h0 = ptr<float>(h0); s.seqlens = ptr<int32_t>(seqlens);
    s.q_batch = q.stride(0); s.k_batch = k.stride(0); s.v_batch = v.stride(0);
    s.g_batch = g.stride(0); s.beta_batch = beta.stride(0);
    s.q_head = q.stride(-2); s.k_head = k.stride(-2); s.v_head = v.stride(-2);
    if (!step) {
        s.q_token = q.stride(1); s.k_token = k.stride(1); s.v_token = v.stride(1);
        s.g_token = g.stride(1); s.beta_token = beta.stride(1);
    }
    return s;
}

std::tuple<Tensor, Maybe, Maybe> delta(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g,
                                       const Tensor& beta, const Maybe& h0, const Maybe& seqlens,
                                       const std::optional<double>& scale, bool final_state, bool checkpoints,
                                       const Maybe& out) {
    const gated_delta_inputs s = delta_inputs(q, k, v, g, beta, h0, seqlens, scale, false);
    const at::Device dev = v.device();
    const On on(dev);
    const Tensor y = output(out, v);
    Maybe h, kept;
    if (final_state) h = at::empty({s.batch, s.heads, s.dv, s.dk}, f32(dev));
    if (checkpoints) kept = bytes(gated_delta_checkpoint_size(&s), dev);
    const Tensor ws = bytes(gated_delta_workspace_size(&s), dev);
    ok(gated_delta_fwd(&s, ptr(y), ptr<float>(h), ptr(kept), ptr(ws), size_t(ws.numel()), on.stream), "gated_delta");
    written(out);
    if (followed(q, k, v, g, beta, h0)) {
        const auto got = unrecorded("gated_delta", y, h);
        return {got.first, got.second, kept};
    }
    return {y, h, kept};
}

py::dict delta_bwd(const Tensor& dy, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g,
                   const Tensor& beta, const Maybe& h0, const Maybe& seqlens, const std::optional<double>& scale,
                   const Maybe& checkpoints, const Maybe& dh_final) {
    const gated_delta_inputs s = delta_inputs(q, k, v, g, beta, h0, seqlens, scale, false);
    const at::Device dev = v.device();
    check("dy", dy, dev, v.scalar_type(), v.sizes(), true);
    if (!checkpoints) throw py::value_error("checkpoints: run gated_delta with want_checkpoints=True");
    check("checkpoints", checkpoints, dev, at::kByte, {int64_t(gated_delta_checkpoint_size(&s))});
    check("dh_final", dh_final, dev, at::kFloat, {s.batch, s.heads, s.dv, s.dk});
    const On on(dev);
    py::dict got;
    const auto add = [&](const char* name, const Tensor& like) {
        const Tensor t = dense_like(like);
        got[name] = t;
        return ptr(t);
    };
    gated_delta_grads d{};
    d.dy = ptr(dy); d.dy_batch = dy.stride(0); d.dy_token = dy.stride(1); d.dy_head = dy.stride(2);
    d.dh_final = ptr<float>(dh_final);
    d.checkpoints = ptr(checkpoints);
    d.dq = add("dq", q);
    d.dk = add("dk", k);
    d.dv = add("dv", v);
    d.dg = static_cast<float*>(add("dg", g));
    d.dbeta = static_cast<float*>(add("dbeta", beta));
    if (h0) d.dh0 = static_cast<float*>(add("dh0", *h0));
    const Tensor ws = bytes(gated_delta_bwd_workspace_size(&s), dev);
    ok(gated_delta_bwd(&s, &d, ptr(ws), size_t(ws.numel()), on.stream), "gated_delta_bwd");
    return got;
}

Tensor delta_step(const Tensor& h, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g,
                  const Tensor& beta, const std::optional<double>& scale, const Maybe& out) {
    const gated_delta_inputs s = delta_inputs(q, k, v, g, beta, std::nullopt, std::nullopt, scale, true);
    check("h", h, v.device(), at::kFloat, {s.batch, s.heads, s.dv, s.dk});
    const On on(v.device());
    const Tensor y = output(out, v);
    ok(gated_delta_step(&s, ptr<float>(h), ptr(y), on.stream), "gated_delta_step");
    written(h);
    written(out);
    if (followed(h, q, k, v, g, beta)) return unrecorded("gated_delta_step", {y})[0];
    return y;
}

// ---------------------------------------------------------------------------
// norms
// ---------------------------------------------------------------------------
// A tensor [..., heads, dim] whose leading dimensions are one run of rows: its row stride.
int64_t row_stride(const char* name, const Tensor& t, int64_t tail) {
    int64_t stride = 0, rows = 1;  // of the rows so far
    for (int64_t d = t.dim() - tail - 1; d >= 0; --d) {
        if (t.size(d) == 1) continue;
        if (rows == 1) stride = t.stride(d);
        else if (t.stride(d) != stride * rows)
            throw py::value_error(std::string(name) + "'s rows must lie at one distance in memory");
        rows *= t.size(d);
    }
    return stride;
}

gated_norm_inputs gated_inputs(const Tensor& x, const Maybe& weight, const Maybe& z, double eps, bool gate_first) {
    gated_norm_inputs s{};
    s.dtype = element_code("x", x);
    if (x.dim() < 2) throw py::value_error("x must be [..., heads, dim]");
    s.dtype = check_lead("x", x, x.dim(), "..., heads, dim");
    check("z", z, x.device(), x.scalar_type(), x.sizes(), true);
    s.dim = x.size(-1);
    s.heads = x.size(-2);
    s.rows = 1;
    for (int64_t d = 0; d < x.dim() - 2; ++d) s.rows *= x.size(d);
    check("weight", weight, x.device(), at::kFloat, {s.dim});
    s.gate_first = gate_first ? 1 : 0;
    s.eps = float(eps);
    s.x = ptr(x); s.z = ptr(z); s.weight = ptr<float>(weight);
    s.x_row = row_stride("x", x, 2); s.x_head = x.stride(-2);
    if (z) {
        s.z_row = row_stride("z", *z, 2);
        s.z_head = z->stride(-2);
    }
    return s;
}

std::pair<Tensor, Maybe> gated(const Tensor& x, const Maybe& weight, const Maybe& z, double eps, bool gate_first,
                               bool want_rstd, const Maybe& out) {
    const gated_norm_inputs s = gated_inputs(x, weight, z, eps, gate_first);
    const On on(x.device());
    const Tensor y = output(out, x);
    Maybe rstd;
    if (want_rstd) rstd = at::empty(x.sizes().slice(0, size_t(x.dim() - 1)), f32(x.device()));
    ok(gated_norm_fwd(&s, ptr(y), ptr<float>(rstd), on.stream), "gated_norm");
    written(out);
    if (followed(x, weight, z)) return {unrecorded("gated_norm", {y})[0], rstd};
    return {y, rstd};
}

py::dict gated_bwd(const Tensor& dy, const Tensor& x, const Maybe& weight, const Maybe& z, const Maybe& rstd,
                   bool gate_first) {
    const gated_norm_inputs s = gated_inputs(x, weight, z, 0.0, gate_first);
    const at::Device dev = x.device();
    check("dy", dy, dev, x.scalar_type(), x.sizes(), true);
    if (!rstd) throw py::value_error("rstd: run gated_norm with want_rstd=True");
    check("rstd", rstd, dev, at::kFloat, x.sizes().slice(0, size_t(x.dim() - 1)));
    const int64_t dy_row = row_stride("dy", dy, 2);
    const On on(dev);
    py::dict got;
    const Tensor dx = dense_like(x);
    Maybe dz, dweight, ws;
    got["dx"] = dx;
    if (weight) got["dweight"] = *(dweight = dense_like(*weight));
    if (z) got["dz"] = *(dz = dense_like(x));
    const size_t need = gated_norm_bwd_workspace_size(s.rows, s.heads, s.dim);
    if (need) ws = bytes(need, dev);
    ok(gated_norm_bwd(&s, ptr(dy), dy_row, dy.stride(-2), ptr<float>(rstd), ptr(dx), ptr(dz), ptr<float>(dweight),
                      ptr(ws), need, on.stream),
       "gated_norm_bwd");
    return got;
}

// `name`: that of the tensor which the others are held to.
residual_norm_inputs residual_inputs(const char* name, const Tensor& x, const Maybe& weight, const Maybe& scale, double eps) {
    residual_norm_inputs s{};
    s.dtype = element_code(name, x);
    if (x.dim() < 1) throw py::value_error(std::string(name) + " must be [..., dim]");
    s.dtype = check_lead(name, x, x.dim(), "..., dim");
    s.dim = x.size(-1);
    s.rows = 1;
    for (int64_t d = 0; d < x.dim() - 1; ++d) s.rows *= x.size(d);
    check("weight", weight, x.device(), at::kFloat, {s.dim});
    check("scale", scale, x.device(), at::kFloat, {s.dim});
    s.eps = float(eps);
    s.x = ptr(x); s.scale = ptr<float>(scale); s.weight = ptr<float>(weight);
    s.x_row = row_stride(name, x, 1);
    return s;
}

// The stream's type: fp32 or that of the activations.
at::ScalarType stream_kind(const char* name, const Tensor& t, const Tensor& x) {
    const at::ScalarType k = t.scalar_type();
    if (k != at::kFloat && k != x.scalar_type())
        throw py::type_error(std::string(name) + " must be torch.float32 or " + type_text(x.scalar_type()) + " (got " +
                             type_text(k) + ")");
    return k;
}

std::tuple<Tensor, Tensor, Maybe> residual(const Tensor& x, const Maybe& res, const Maybe& weight, const Maybe& scale,
                                           double eps, bool want_rstd) {
    residual_norm_inputs s = residual_inputs("x", x, weight, scale, eps);
    const at::Device dev = x.device();
    const at::ScalarType kind = res ? stream_kind("residual", *res, x) : x.scalar_type();
    check("residual", res, dev, kind, x.sizes(), true);
    s.stream_dtype = kind == at::kFloat ? int32_t(SSD_F32) : s.dtype;
    s.residual = ptr(res);
    if (res) s.residual_row = row_stride("residual", *res, 1);
    const On on(dev);
    const Tensor y = dense_like(x), r = at::empty(x.sizes(), x.options().dtype(kind));
    Maybe rstd;
    if (want_rstd) rstd = at::empty(x.sizes().slice(0, size_t(x.dim() - 1)), f32(dev));
    ok(residual_norm_fwd(&s, ptr(y), ptr(r), ptr<float>(rstd), on.stream), "residual_norm");
    if (followed(x, res, weight, scale)) {
        const std::vector<Tensor> got = unrecorded("residual_norm", {y, r});
        return {got[0], got[1], rstd};
    }
    return {y, r, rstd};
}

py::dict residual_bwd(const Tensor& dy, const Tensor& r, const Maybe& weight, const Tensor& rstd, const Maybe& dr,
                      const Maybe& x, const Maybe& scale) {
    residual_norm_inputs s = residual_inputs("dy", dy, weight, scale, 0.0);
    const at::Device dev = dy.device();
    const at::ScalarType kind = stream_kind("r", r, dy);
    s.stream_dtype = kind == at::kFloat ? int32_t(SSD_F32) : s.dtype;
    check("r", r, dev, kind, dy.sizes(), true);
    check("dr", dr, dev, kind, dy.sizes(), true);
    check("rstd", rstd, dev, at::kFloat, dy.sizes().slice(0, size_t(dy.dim() - 1)));
    if (scale && !x) throw py::value_error("x: the gradient of scale needs it");
    check("x", x, dev, dy.scalar_type(), dy.sizes(), true);
    residual_norm_grads g{};
    g.dy_row = s.x_row;
    s.x = ptr(x);
    s.x_row = x ? row_stride("x", *x, 1) : 0;
    g.r_row = row_stride("r", r, 1);
    g.dr_row = dr ? row_stride("dr", *dr, 1) : 0;
    const On on(dev);
    py::dict got;
    const Tensor dres = at::empty(dy.sizes(), dy.options().dtype(kind)), dx = dense_like(dy);
    Maybe dweight, dscale, ws;
    got["dresidual"] = dres;
    got["dx"] = dx;
    if (weight) got["dweight"] = *(dweight = dense_like(*weight));
    if (scale) got["dscale"] = *(dscale = dense_like(*scale));
    g.dy = ptr(dy); g.dr = ptr(dr); g.r = ptr(r); g.rstd = ptr<float>(rstd);
    g.dresidual = ptr(dres); g.dx = ptr(dx); g.dweight = ptr<float>(dweight); g.dscale = ptr<float>(dscale);
    const size_t need = residual_norm_bwd_workspace_size(s.rows, s.dim);
    if (need) ws = bytes(need, dev);
    ok(residual_norm_bwd(&s, &g, ptr(ws), need, on.stream), "residual_norm_bwd");
    return got;
}

}  // namespace

void bind_gated_delta(py::module_& m) {
    m.def("gated_delta", &delta);
    m.def("gated_delta_bwd", &delta_bwd);
    m.def("gated_delta_step", &delta_step);
    m.def("gated_norm", &gated);
    m.def("gated_norm_bwd", &gated_bwd);
    m.def("residual_norm", &residual);
    m.def("residual_norm_bwd", &residual_bwd);
}
