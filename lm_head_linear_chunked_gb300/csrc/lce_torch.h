// What the torch sides of the operators share: the library's addresses, checks
// of tensors, allocation, and the raising of errors.
#pragma once

#include <ATen/core/Tensor.h>
#include <ATen/TracerMode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/SmallVector.h>
#include <c10/util/accumulate.h>
#include <torch/csrc/autograd/forward_grad.h>
#include <torch/csrc/utils/pybind.h>

#include <string>
#include <vector>

#include "lce.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace lce_torch {

struct Library {
    decltype(&lce_layer_norm_forward) norm_forward;
    decltype(&lce_layer_norm_backward) norm_backward;
    decltype(&lce_layer_norm_workspace_size) norm_workspace;
    decltype(&lce_balance_forward) balance_forward;
    decltype(&lce_balance_fused) balance_fused;
    decltype(&lce_balance_backward) balance_backward;
    decltype(&lce_balance_workspace_size) balance_workspace;
    decltype(&lce_beam_select) beam_select;
    decltype(&lce_beam_workspace_size) beam_workspace;
    decltype(&lce_beam_reorder) beam_reorder;
    decltype(&lce_rms_norm_forward) rms_forward;
    decltype(&lce_rms_norm_fp8) rms_fp8;
    decltype(&lce_rms_norm_backward) rms_backward;
    decltype(&lce_rms_norm_workspace_size) rms_workspace;
    decltype(&lce_embedding_forward) embedding_forward;
    decltype(&lce_embedding_backward) embedding_backward;
    decltype(&lce_embedding_workspace_size) embedding_workspace;
    decltype(&lce_expert_rows) expert_rows;
    decltype(&lce_expert_plan) expert_plan;
    decltype(&lce_expert_plan_workspace_size) expert_plan_workspace;
    decltype(&lce_expert_dispatch) expert_dispatch;
    decltype(&lce_expert_dispatch_backward) expert_dispatch_backward;
    decltype(&lce_expert_combine) expert_combine;
    decltype(&lce_expert_combine_backward) expert_combine_backward;
};
extern Library lib;
extern PyObject *lce_error, *traced_error;  // kept for the life of the process
void bind_rows(py::module_& m);             // the operators of lce_torch_rows.cpp

namespace {

inline void check(lce_status_t status, const char* where) {
    if (status == LCE_OK) return;
    const py::object e = py::reinterpret_borrow<py::object>(lce_error)(static_cast<int>(status), where);
    PyErr_SetObject(lce_error, e.ptr());
    throw py::error_already_set();
}

inline std::string text(at::IntArrayRef v) {
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}

inline int type_code(const Tensor& t, const char* what) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return LCE_BF16;
        case at::kHalf: return LCE_F16;
        case at::kFloat: return LCE_F32;
        default: throw py::type_error(std::string(what) + " must be bfloat16, float16 or float32, got " + toString(t.scalar_type()));
    }
}

inline void check_shape(const Tensor& t, at::IntArrayRef shape, const char* what) {
    if (t.sizes() != shape)
        throw py::value_error(std::string(what) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
}

inline void check_type(const Tensor& t, at::ScalarType type, const char* what) {
    if (t.scalar_type() != type)
        throw py::type_error(std::string(what) + " must be " + toString(type) + ", got " + toString(t.scalar_type()));
}

inline void on_cuda(const at::Device& device) {
    if (!device.is_cuda()) throw py::value_error("tensors must be on a CUDA device, got " + device.str());
}
inline void on_device(const Tensor& t, const at::Device& device, const char* what) {
    if (t.device() != device) throw py::value_error(std::string(what) + " is on " + t.device().str() + ", expected " + device.str());
}
inline void on_device(const OptTensor& t, const at::Device& device, const char* what) {
    if (t) on_device(*t, device, what);
}

// The calls below work on addresses.  A forward-mode tangent would be lost
// without a word (there are no forward-mode derivatives), and torch.jit.trace
// would record the allocation of the outputs without the call that fills them.
inline void no_tangent(const Tensor& t, const char* what) {
    if (t.unsafeGetTensorImpl()->autograd_meta() && t._fw_grad(/*level=*/0).defined()) {
        PyErr_SetString(PyExc_NotImplementedError,
                        (std::string(what) + " has a forward-mode tangent: this operator has no forward-mode derivative").c_str());
        throw py::error_already_set();
    }
}
inline void no_tangent(const OptTensor& t, const char* what) {
    if (t) no_tangent(*t, what);
}
inline void not_traced(const char* name) {
    if (at::tracer::impl::is_dispatch_enabled()) {
        PyErr_SetString(traced_error, (std::string(name) + " cannot be traced").c_str());
        throw py::error_already_set();
    }
}

// The current stream: outputs and workspaces belong to it.
inline lce_stream_t stream_of(const at::Device& device) {
    return reinterpret_cast<lce_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
}

template <typename T>
T* ptr(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }
inline void* ptr(const OptTensor& t) { return t ? t->data_ptr() : nullptr; }

// Outputs and workspaces, straight from the allocator: the dispatcher's way to
// it takes as long as the rest of a small call.  A trace has to see them.
inline Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device& device) {
    if (!device.is_cuda() || at::tracer::impl::is_dispatch_enabled()) return at::empty(shape, at::TensorOptions().dtype(type).device(device));
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
}
// Two tensors of one type out of one allocation.
inline std::pair<Tensor, Tensor> empty_pair(at::IntArrayRef a, at::IntArrayRef b, at::ScalarType type, const at::Device& device) {
    const int64_t size = static_cast<int64_t>(c10::elementSize(type)), step = 256 / size;
    const int64_t first = (c10::multiply_integers(a) + step - 1) / step * step;
    const Tensor both = empty({first + c10::multiply_integers(b)}, type, device);
    auto part = [&](at::IntArrayRef shape, int64_t offset) {
        auto t = c10::make_intrusive<c10::TensorImpl>(c10::Storage(both.storage()), both.key_set(), both.dtype());
        t->set_sizes_contiguous(shape);
        t->set_storage_offset(offset);
        return Tensor(std::move(t));
    };
    return {part(a, 0), part(b, first)};
}
inline Tensor like(const Tensor& t) { return empty(t.sizes(), t.scalar_type(), t.device()); }

// t as rows of its last dimension: t itself where its rows are contiguous and
// evenly spaced, else a contiguous copy.
inline Tensor rows_of(const Tensor& t, int64_t* stride) {
    const int64_t width = t.size(-1);
    *stride = width;
    if (t.is_neg()) return t.resolve_neg().contiguous();  // memory that stands for other values
    if (t.is_contiguous()) return t;
    if (t.dim() == 2 && t.stride(1) == 1 && t.stride(0) >= width) {
        *stride = t.stride(0);
        return t;
    }
    return t.contiguous();
}

inline int64_t width(const Tensor& x) {
    if (x.dim() == 0 || x.size(-1) == 0) throw py::value_error("x needs a last dimension of at least one element");
    return x.size(-1);
}

inline void check_affine(const Tensor& x, int64_t H, const Tensor& t, const char* what) {
    if (t.dim() != 1 || t.size(0) != H) check_shape(t, {H}, what);
    if (t.scalar_type() != x.scalar_type()) check_type(t, at::kFloat, what);
    if (!t.is_contiguous()) throw py::value_error(std::string(what) + " must be contiguous");
}

}  // namespace
}  // namespace lce_torch
