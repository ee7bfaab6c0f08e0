// What the binding's translation units share: checks of tensors, pointers,
// status codes, the stream of a call, and what autograd has to be told.
#pragma once

#include <torch/extension.h>

#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>

#include <optional>
#include <string>
#include <tuple>
#include <type_traits>
#include <utility>
#include <vector>

#include "../../include/chunked_linear_scan.h"

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

// The C ABI's code of an activation's element type.
int32_t element_code(const char* name, const Tensor& t) {
    const at::ScalarType k = t.scalar_type();
    if (k != at::kFloat && k != at::kBFloat16 && k != at::kHalf)
        throw py::type_error(std::string(name) + " must be float32, bfloat16 or float16");
    return k == at::kFloat ? SSD_F32 : k == at::kBFloat16 ? SSD_BF16 : SSD_F16;
}

// The tensor that the others are held to: its type, dimensions (as `text` has them) and device.
int32_t check_lead(const char* name, const Tensor& t, int64_t dims, const char* text) {
    const int32_t code = element_code(name, t);
    check_dims(name, t, dims, text);
    if (!t.is_cuda())
        throw py::value_error(std::string(name) + " must be on a GPU (got " + t.device().str() + ")");
    check(name, t, t.device(), t.scalar_type(), t.sizes(), true);
    return code;
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

}  // namespace
