// Python binding of include/selective_scan.h: checks tensors, allocates outputs
// and workspaces with torch and calls the C ABI on torch's current stream of the
// inputs' device.  It holds no computation and no state.  Native because a call
// has up to a dozen tensors to check, which in Python takes longer than the
// smallest kernels run: one decode token of a sequence took 10.5 us a call, and
// takes 4 to 5 (3 of them the launch).
#include <torch/extension.h>

#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>

#include <optional>
#include <string>
#include <tuple>
#include <type_traits>
#include <utility>
#include <vector>

#include "../../include/selective_scan.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

std::string type_text(at::ScalarType k) {
    switch (k) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kHalf: return "torch.float16";
        case at::kDouble: return "torch.float64";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        default: return at::toString(k);
    }
}

// t is on `dev` with this type and shape, contiguous or (strided) its last dimension adjacent.
void check(const char* name, const Tensor& t, at::Device dev, at::ScalarType kind, at::IntArrayRef shape,
           bool strided = false) {
    const std::string n(name);
    if (t.device() != dev)
        throw py::value_error(n + " must be on one GPU with the other tensors (got " + t.device().str() + ")");
    if (t.scalar_type() != kind)
        throw py::type_error(n + " must be " + type_text(kind) + " (got " + type_text(t.scalar_type()) + ")");
    if (t.sizes() != shape)
        throw py::value_error(n + " must have shape " + shape_text(shape) + " (got " + shape_text(t.sizes()) + ")");
    if (t.is_contiguous() || (strided && (t.size(-1) == 1 || t.stride(-1) == 1))) return;
    throw py::value_error(strided ? n + "'s last dimension must be adjacent in memory" : n + " must be contiguous");
}

void check(const char* name, const Maybe& t, at::Device dev, at::ScalarType kind, at::IntArrayRef shape,
           bool strided = false) {
    if (t) check(name, *t, dev, kind, shape, strided);
}

void check_dims(const char* name, const Tensor& t, int64_t dims, const char* text) {
    if (t.dim() != dims) throw py::value_error(std::string(name) + " must be [" + text + "]");
}

// The tensor that the others are held to.
int32_t check_activation(const char* name, const Tensor& t, bool step) {
    const at::ScalarType k = t.scalar_type();
    if (k != at::kFloat && k != at::kBFloat16 && k != at::kHalf)
        throw py::type_error(std::string(name) + " must be float32, bfloat16 or float16");
    check_dims(name, t, step ? 2 : 3, step ? "batch, channels" : "batch, seqlen, channels");
    if (!t.is_cuda())
        throw py::value_error(std::string(name) + " must be on a GPU (got " + t.device().str() + ")");
    check(name, t, t.device(), k, t.sizes(), true);
    return k == at::kFloat ? SSD_F32 : k == at::kBFloat16 ? SSD_BF16 : SSD_F16;
}

template <typename T = void>
T* ptr(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* ptr(const Maybe& t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

void ok(int status, const char* what) {
    if (status == SSD_OK) return;
    const py::object e = py::module_::import("chunked_linear_scan_amd").attr("SSDError");
    PyErr_SetObject(e.ptr(), e(status, what).ptr());
    throw py::error_already_set();
}

// Whether autograd follows one of the tensors now.
template <typename... T>
bool followed(const T&... tensors) {
    const auto needs = [](const auto& t) {
        if constexpr (std::is_same_v<std::decay_t<decltype(t)>, Maybe>) return t && t->requires_grad();
        else return t.requires_grad();
    };
    return at::GradMode::is_enabled() && (needs(tensors) || ...);
}

// The outputs of a call on such tensors: the same values, through which a backward pass raises.
std::vector<Tensor> unrecorded(const char* what, const std::vector<Tensor>& outputs) {
    const py::object f = py::module_::import("chunked_linear_scan_amd.selective").attr("_unrecorded");
    return f(what, outputs).cast<std::vector<Tensor>>();
}
std::pair<Tensor, Maybe> unrecorded(const char* what, const Tensor& output, const Maybe& state) {
    if (!state) return {unrecorded(what, {output})[0], state};
    const std::vector<Tensor> got = unrecorded(what, {output, *state});
    return {got[0], got[1]};
}

// The launches' device is current for the scope's life.
struct On {
    c10::DeviceGuard guard;
    void* stream;
    explicit On(at::Device d) : guard(d), stream(c10::hip::getCurrentHIPStream(d.index()).stream()) {}
};

// Tells autograd that a tensor was written in place (one of inference mode counts no versions).
void written(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(const Maybe& t) {
    if (t) written(*t);
}

Tensor dense_like(const Tensor& t) { return at::empty(t.sizes(), t.options()); }

Tensor output(const Maybe& out, const Tensor& like) {
    if (!out) return dense_like(like);
    check("out", *out, like.device(), like.scalar_type(), like.sizes());
    return *out;
}

Tensor bytes(size_t n, at::Device dev) {
    return at::empty({int64_t(n)}, at::TensorOptions().dtype(at::kByte).device(dev));
}

at::TensorOptions f32(at::Device dev) { return at::TensorOptions().dtype(at::kFloat).device(dev); }

// ---------------------------------------------------------------------------
// selective scan
// ---------------------------------------------------------------------------
selective_scan_inputs scan_inputs(const Tensor& u, const Tensor& dt, const Tensor& A, const Tensor& B, const Tensor& C,
                                  const Maybe& D, const Maybe& z, const Maybe& dt_bias, const Maybe& h0,
                                  const Maybe& seqlens, bool softplus, bool step) {
    selective_scan_inputs s{};
    s.dtype = check_activation("u", u, step);
    const at::Device dev = u.device();
    const at::ScalarType kind = u.scalar_type();
    check("dt", dt, dev, kind, u.sizes(), true);
    check("z", z, dev, kind, u.sizes(), true);
    check_dims("A", A, 2, "channels, dstate");
    check_dims("B", B, step ? 3 : 4, step ? "batch, ngroups, dstate" : "batch, seqlen, ngroups, dstate");
    s.batch = u.size(0);
    s.seqlen = step ? 1 : u.size(1);
    s.channels = u.size(-1);
    s.dstate = A.size(1);
    s.ngroups = B.size(-2);
    check("A", A, dev, at::kFloat, {s.channels, s.dstate});
    const int64_t bc[] = {s.batch, s.seqlen, s.ngroups, s.dstate}, bc1[] = {s.batch, s.ngroups, s.dstate};
    const at::IntArrayRef rows = step ? at::IntArrayRef(bc1, 3) : at::IntArrayRef(bc, 4);
    check("B", B, dev, kind, rows, true);
    check("C", C, dev, kind, rows, true);
    check("D", D, dev, at::kFloat, {s.channels});
    check("dt_bias", dt_bias, dev, at::kFloat, {s.channels});
    check("h0", h0, dev, at::kFloat, {s.batch, s.channels, s.dstate});
    check("seqlens", seqlens, dev, at::kInt, {s.batch});
    s.softplus = softplus ? 1 : 0;
    s.u = ptr(u); s.dt = ptr(dt); s.z = ptr(z); s.B = ptr(B); s.C = ptr(C);
    s.A = ptr<float>(A); s.D = ptr<float>(D); s.dt_bias = ptr<float>(dt_bias); s.h0 = ptr<float>(h0);
    s.seqlens = ptr<int32_t>(seqlens);
    const Tensor& zz = z ? *z : u;
    s.u_batch = u.stride(0); s.dt_batch = dt.stride(0); s.z_batch = zz.stride(0);
    s.B_batch = B.stride(0); s.C_batch = C.stride(0);
    s.B_group = B.stride(-2); s.C_group = C.stride(-2);
    if (!step) {
        s.u_token = u.stride(1); s.dt_token = dt.stride(1); s.z_token = zz.stride(1);
        s.B_token = B.stride(1); s.C_token = C.stride(1);
    }
    return s;
}

std::vector<int64_t> checkpoint_shape(const selective_scan_inputs& s) {
    const int64_t size = int64_t(selective_scan_checkpoint_size(s.batch, s.seqlen, s.channels, s.dstate));
    const int64_t tile = 4 * s.batch * s.channels * s.dstate;
    return {s.batch, tile > 0 ? size / tile : 0, s.dstate, s.channels};
}

std::tuple<Tensor, Maybe, Maybe> scan(const Tensor& u, const Tensor& dt, const Tensor& A, const Tensor& B, const Tensor& C,
                                      const Maybe& D, const Maybe& z, const Maybe& dt_bias, const Maybe& h0,
                                      const Maybe& seqlens, bool softplus, bool final_state, bool checkpoints,
                                      const Maybe& out) {
    const selective_scan_inputs s = scan_inputs(u, dt, A, B, C, D, z, dt_bias, h0, seqlens, softplus, false);
    const On on(u.device());
    const Tensor y = output(out, u);
    Maybe h, kept, ws;
    if (final_state) h = at::empty({s.batch, s.channels, s.dstate}, f32(u.device()));
    if (checkpoints) kept = at::empty(checkpoint_shape(s), f32(u.device()));
    const size_t need = selective_scan_workspace_size(s.batch, s.seqlen, s.channels, s.dstate, s.ngroups);
    if (need) ws = bytes(need, u.device());
    ok(selective_scan_fwd(&s, ptr(y), ptr<float>(h), ptr(kept), ptr(ws), need, on.stream), "selective_scan");
    written(out);
    if (followed(u, dt, A, B, C, D, z, dt_bias, h0)) {
        const auto got = unrecorded("selective_scan", y, h);
        return {got.first, got.second, kept};
    }
    return {y, h, kept};
}

py::dict scan_bwd(const Tensor& dy, const Tensor& u, const Tensor& dt, const Tensor& A, const Tensor& B, const Tensor& C,
                  const Maybe& D, const Maybe& z, const Maybe& dt_bias, const Maybe& h0, const Maybe& seqlens,
                  bool softplus, const Maybe& checkpoints, const Maybe& dh_final) {
    const selective_scan_inputs s = scan_inputs(u, dt, A, B, C, D, z, dt_bias, h0, seqlens, softplus, false);
    const at::Device dev = u.device();
    check("dy", dy, dev, u.scalar_type(), u.sizes(), true);
    if (!checkpoints) throw py::value_error("checkpoints: run selective_scan with want_checkpoints=True");
    check("checkpoints", checkpoints, dev, at::kFloat, checkpoint_shape(s));
    check("dh_final", dh_final, dev, at::kFloat, {s.batch, s.channels, s.dstate});
    const On on(dev);
    py::dict got;
    selective_scan_grads g{};
    const auto add = [&](const char* name, const Tensor& like) {
        const Tensor t = dense_like(like);
        got[name] = t;
        return ptr(t);
    };
    g.dy = ptr(dy); g.dy_batch = dy.stride(0); g.dy_token = dy.stride(1);
    g.dh_final = ptr<float>(dh_final);
    g.checkpoints = ptr(checkpoints);
    g.du = add("du", u);
    g.ddt = add("ddt", u);
    g.dA = static_cast<float*>(add("dA", A));
    g.dB = add("dB", B);
    g.dC = add("dC", C);
    if (D) g.dD = static_cast<float*>(add("dD", *D));
    if (z) g.dz = add("dz", u);
    if (dt_bias) g.ddt_bias = static_cast<float*>(add("ddt_bias", *dt_bias));
    if (h0) g.dh0 = static_cast<float*>(add("dh0", *h0));
    const size_t need = selective_scan_bwd_workspace_size(s.batch, s.seqlen, s.channels, s.dstate, s.ngroups);
    const Tensor ws = bytes(need > 16 ? need : 16, dev);
    ok(selective_scan_bwd(&s, &g, ptr(ws), size_t(ws.numel()), on.stream), "selective_scan_bwd");
    return got;
}

Tensor scan_step(const Tensor& h, const Tensor& u, const Tensor& dt, const Tensor& A, const Tensor& B, const Tensor& C,
                 const Maybe& D, const Maybe& z, const Maybe& dt_bias, bool softplus, const Maybe& out) {
    const selective_scan_inputs s =
        scan_inputs(u, dt, A, B, C, D, z, dt_bias, std::nullopt, std::nullopt, softplus, true);
    check("h", h, u.device(), at::kFloat, {s.batch, s.channels, s.dstate});
    const On on(u.device());
    const Tensor y = output(out, u);
    ok(selective_scan_step(&s, ptr<float>(h), ptr(y), on.stream), "selective_scan_step");
    written(h);
    written(out);
    if (followed(h, u, dt, A, B, C, D, z, dt_bias)) return unrecorded("selective_scan_step", {y})[0];
    return y;
}

// ---------------------------------------------------------------------------
// short convolution
// ---------------------------------------------------------------------------
short_conv_inputs conv_inputs(const Tensor& x, const Tensor& weight, const Maybe& bias, const Maybe& initial_state,
                              const Maybe& seqlens, bool silu, bool step) {
    short_conv_inputs s{};
    s.dtype = check_activation("x", x, step);
    const at::Device dev = x.device();
    check_dims("weight", weight, 2, "channels, width");
    s.batch = x.size(0);
    s.seqlen = step ? 1 : x.size(1);
    s.channels = x.size(-1);
    s.width = weight.size(1);
    check("weight", weight, dev, at::kFloat, {s.channels, s.width});
    check("bias", bias, dev, at::kFloat, {s.channels});
    check("initial_state", initial_state, dev, x.scalar_type(), {s.batch, s.width - 1, s.channels});
    check("seqlens", seqlens, dev, at::kInt, {s.batch});
    s.silu = silu ? 1 : 0;
    s.x = ptr(x);
    s.x_batch = x.stride(0);
    s.x_token = step ? 0 : x.stride(1);
    s.weight = ptr<float>(weight); s.bias = ptr<float>(bias);
    s.initial_state = ptr(initial_state);
    s.seqlens = ptr<int32_t>(seqlens);
    return s;
}

std::pair<Tensor, Maybe> conv(const Tensor& x, const Tensor& weight, const Maybe& bias, const Maybe& initial_state,
                              const Maybe& seqlens, bool silu, bool final_state, const Maybe& out) {
    const short_conv_inputs s = conv_inputs(x, weight, bias, initial_state, seqlens, silu, false);
    const On on(x.device());
    const Tensor y = output(out, x);
    Maybe last;
    if (final_state) last = at::empty({s.batch, s.width > 0 ? s.width - 1 : 0, s.channels}, x.options());
    ok(short_conv_fwd(&s, ptr(y), ptr(last), on.stream), "short_conv");
    written(out);
    if (followed(x, weight, bias, initial_state)) return unrecorded("short_conv", y, last);
    return {y, last};
}

py::dict conv_bwd(const Tensor& dy, const Tensor& x, const Tensor& weight, const Maybe& bias, const Maybe& initial_state,
                  const Maybe& seqlens, bool silu, const Maybe& dfinal) {
    const short_conv_inputs s = conv_inputs(x, weight, bias, initial_state, seqlens, silu, false);
    const at::Device dev = x.device();
    check("dy", dy, dev, x.scalar_type(), x.sizes(), true);
    check("dfinal_state", dfinal, dev, x.scalar_type(), {s.batch, s.width - 1, s.channels});
    const On on(dev);
    py::dict got;
    const Tensor dx = dense_like(x), dweight = dense_like(weight);
    Maybe dbias, dinitial;
    got["dx"] = dx;
    got["dweight"] = dweight;
    if (bias) got["dbias"] = *(dbias = dense_like(*bias));
    if (initial_state) got["dinitial_state"] = *(dinitial = dense_like(*initial_state));
    const size_t need = short_conv_bwd_workspace_size(s.batch, s.seqlen, s.channels, s.width);
    const Tensor ws = bytes(need > 16 ? need : 16, dev);
    ok(short_conv_bwd(&s, ptr(dy), dy.stride(0), dy.stride(1), ptr(dfinal), ptr(dx), ptr<float>(dweight),
                      ptr<float>(dbias), ptr(dinitial), ptr(ws), size_t(ws.numel()), on.stream),
       "short_conv_bwd");
    return got;
}

Tensor conv_step(const Tensor& state, const Tensor& x, const Tensor& weight, const Maybe& bias, bool silu,
                 const Maybe& out) {
    const short_conv_inputs s = conv_inputs(x, weight, bias, std::nullopt, std::nullopt, silu, true);
    check("state", state, x.device(), x.scalar_type(), {s.batch, s.width - 1, s.channels});
    const On on(x.device());
    const Tensor y = output(out, x);
    ok(short_conv_step(&s, ptr(state), ptr(y), on.stream), "short_conv_step");
    written(state);
    written(out);
    if (followed(state, x, weight, bias)) return unrecorded("short_conv_step", {y})[0];
    return y;
}

// ---------------------------------------------------------------------------
// 8-bit cache of states
// ---------------------------------------------------------------------------
struct CacheArgs {
    std::vector<int64_t> states;  // the shape of the states that the slots name
    int64_t batch, rows, dstate, nslots;
    int format;
};

CacheArgs cache_args(const Tensor& cache, const Tensor& scales, const Tensor& slots) {
    const at::ScalarType k = cache.scalar_type();
    if (k != at::kChar && k != at::kFloat8_e4m3fn) throw py::type_error("cache must be int8 or float8_e4m3fn");
    if (cache.dim() < 2) throw py::value_error("cache must be [slots, ..., dstate]");
    if (!cache.is_cuda()) throw py::value_error("cache must be on a GPU (got " + cache.device().str() + ")");
    const at::Device dev = cache.device();
    check("cache", cache, dev, k, cache.sizes());
    check("scales", scales, dev, at::kFloat, cache.sizes().slice(0, size_t(cache.dim() - 1)));
    check_dims("slots", slots, 1, "batch");
    check("slots", slots, dev, at::kInt, {slots.size(0)});
    CacheArgs a{cache.sizes().vec(), slots.size(0), 1, cache.size(-1), cache.size(0),
                k == at::kChar ? int(SSD_I8) : int(SSD_E4M3)};
    a.states[0] = a.batch;
    for (int64_t d = 1; d + 1 < cache.dim(); ++d) a.rows *= cache.size(d);
    return a;
}

void cache_write(const Tensor& h, const Tensor& cache, const Tensor& scales, const Tensor& slots) {
    const CacheArgs a = cache_args(cache, scales, slots);
    check("h", h, cache.device(), at::kFloat, a.states);
    const On on(cache.device());
    ok(state_cache_write(ptr<float>(h), ptr<int32_t>(slots), a.batch, a.rows, a.dstate, a.nslots, a.format, ptr(cache),
                         ptr<float>(scales), on.stream),
       "state_cache_write");
    written(cache);
    written(scales);
}

Tensor cache_read(const Tensor& cache, const Tensor& scales, const Tensor& slots, const Maybe& out) {
    const CacheArgs a = cache_args(cache, scales, slots);
    if (out) check("out", *out, cache.device(), at::kFloat, a.states);
    const On on(cache.device());
    const Tensor h = out ? *out : at::empty(a.states, f32(cache.device()));
    ok(state_cache_read(ptr(cache), ptr<float>(scales), ptr<int32_t>(slots), a.batch, a.rows, a.dstate, a.nslots,
                        a.format, ptr<float>(h), on.stream),
       "state_cache_read");
    written(out);
    return h;
}

}  // namespace

PYBIND11_MODULE(_selective_binding, m) {
    m.def("selective_scan", &scan);
    m.def("selective_scan_bwd", &scan_bwd);
    m.def("selective_scan_step", &scan_step);
    m.def("short_conv", &conv);
    m.def("short_conv_bwd", &conv_bwd);
    m.def("short_conv_step", &conv_step);
    m.def("state_cache_write", &cache_write);
    m.def("state_cache_read", &cache_read);
}
