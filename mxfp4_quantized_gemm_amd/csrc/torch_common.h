// What the torch binding's parts share: checks of tensors, streams, and the norm
// and 8-bit operators that attention's block calls too.
#pragma once
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/extension.h>

#include <optional>
#include <tuple>

#include "../../include/mxfp4.h"

namespace mx {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
typedef std::optional<Tensor> Maybe;

inline int dtype_of(const Tensor& t, const char* name) {
  const auto s = t.scalar_type();
  TORCH_CHECK_TYPE(s == at::kFloat || s == at::kBFloat16 || s == at::kHalf, name,
                   " must be float32, bfloat16 or float16, got ", s);
  return s == at::kFloat ? MXFP4_DT_F32 : s == at::kBFloat16 ? MXFP4_DT_BF16 : MXFP4_DT_F16;
}

// Raises the package's MXFP4Error for a status other than MXFP4_OK. The GIL is held.
inline void check(int status, const char* where) {
  if (status == MXFP4_OK) return;
  const py::object cls = py::module_::import("mxfp4_quantized_gemm_amd").attr("MXFP4Error");
  const py::object e = cls(status, where);
  PyErr_SetObject(cls.ptr(), e.ptr());
  throw py::error_already_set();
}

// torch.jit.trace would record the outputs' allocation alone: replays of it would
// return memory that nothing wrote.
inline void no_trace(const char* where) {
  TORCH_CHECK(!torch::jit::tracer::isTracing(), where, " cannot be recorded by torch.jit.trace");
}

// A forward-mode tangent of an input would be dropped, which is a derivative of
// zero. (no_grad() does not switch forward mode off.)
inline void no_tangent(const char* where, std::initializer_list<const Tensor*> inputs) {
  for (const Tensor* t : inputs)
    TORCH_CHECK(t == nullptr || !t->defined() || !t->_fw_grad(0).defined(), where,
                " has no forward-mode derivative");
}

// Codes and their products have no gradient, in their scales and bias neither:
// a call that autograd would have to record is refused.
inline void no_gradient(const char* where, std::initializer_list<const Tensor*> inputs) {
  no_trace(where);
  no_tangent(where, inputs);
  if (!at::GradMode::is_enabled()) return;
  for (const Tensor* t : inputs)
    TORCH_CHECK(t == nullptr || !t->requires_grad(), where,
                " has no gradient: call it under torch.no_grad() or on detached tensors");
}

inline hipStream_t stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

inline bool has(const Maybe& t) { return t.has_value() && t->defined(); }
inline const Tensor* ptr(const Maybe& t) { return has(t) ? &*t : nullptr; }

inline void on_gpu(const Tensor& t, const char* name, const Tensor* like = nullptr) {
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must live in GPU memory");
  TORCH_CHECK_VALUE(like == nullptr || t.device() == like->device(), name, " must be on ",
                    like ? like->device() : t.device(), ", is on ", t.device());
}

// t [..., cols] as [rows][cols] with a unit column stride and rows that do not
// overlap: a view where it has them, a copy where not.
struct Rows {
  Tensor t;
  int64_t rows, cols, ld;
  const void* p() const { return t.const_data_ptr(); }
};

inline Rows rows_of(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.dim() >= 1, name, " must have a dimension");
  Rows r{t, 0, t.size(-1), 0};
  if (t.dim() != 2) {
    int64_t n = 1;
    for (int64_t i = 0; i + 1 < t.dim(); ++i) n *= t.size(i);
    r.t = t.reshape({n, r.cols});
  }
  r.rows = r.t.size(0);
  if ((r.t.stride(1) != 1 && r.cols > 1) || (r.t.stride(0) < r.cols && r.rows > 1))
    r.t = r.t.clone(at::MemoryFormat::Contiguous);
  r.ld = r.rows > 1 ? r.t.stride(0) : r.cols;
  return r;
}

inline const float* floats(const Tensor& t, int64_t n, const char* name, const Tensor& like) {
  on_gpu(t, name, &like);
  TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, name, " must be float32, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.numel() == n && t.is_contiguous(), name, " must hold ", n, " contiguous values, holds ",
                    t.numel());
  return t.const_data_ptr<float>();
}

inline int64_t padded(int64_t cols) { return (cols + 127) / 128 * 128; }

struct Operand {  // int8 codes [rows][cols rounded up to 128] and a scale a row
  Tensor codes, scales;
};
Operand norm_int8(const Tensor& x, const Maybe& weight, double eps, const Maybe& residual, Tensor* h);
Operand quantize(const Tensor& x, const Maybe& gate);
Tensor product(const Operand& x, const Tensor& w, const Tensor& sw, const Maybe& bias, at::ScalarType out);
void check_weight(const Tensor& w, int64_t cols, const char* name);
// What product() refuses of a weight, for calls that change something before it.
void check_product(const Tensor& w, const Tensor& sw, const Tensor& like, const char* name);
Tensor as(const Tensor& y, const Tensor& x);  // y [rows][N] with x's leading dimensions

void bind_attention(pybind11::module_& m);  // torch_attention.cpp

}  // namespace mx
