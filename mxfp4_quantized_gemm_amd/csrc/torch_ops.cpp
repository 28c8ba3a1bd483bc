// Torch binding of the norm and 8-bit operators (module _ops): checks tensors,
// allocates outputs and workspaces with torch's allocator on the current
// stream of the tensors' device, and calls the C ABI (include/mxfp4.h). It
// computes nothing itself. These operators run once per layer and token when
// one token is decoded, and take a few microseconds on the GPU then; a binding
// in Python (ctypes) cost 8 us a call and the norm's gradient 135 us.
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/extension.h>

#include <optional>
#include <tuple>

#include "../../include/mxfp4.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
typedef std::optional<Tensor> Maybe;

int dtype_of(const Tensor& t, const char* name) {
  const auto s = t.scalar_type();
  TORCH_CHECK_TYPE(s == at::kFloat || s == at::kBFloat16 || s == at::kHalf, name,
                   " must be float32, bfloat16 or float16, got ", s);
  return s == at::kFloat ? MXFP4_DT_F32 : s == at::kBFloat16 ? MXFP4_DT_BF16 : MXFP4_DT_F16;
}

// Raises the package's MXFP4Error for a status other than MXFP4_OK. The GIL is held.
void check(int status, const char* where) {
  if (status == MXFP4_OK) return;
  const py::object cls = py::module_::import("mxfp4_quantized_gemm_amd").attr("MXFP4Error");
  const py::object e = cls(status, where);
  PyErr_SetObject(cls.ptr(), e.ptr());
  throw py::error_already_set();
}

// torch.jit.trace would record the outputs' allocation alone: replays of it would
// return memory that nothing wrote.
void no_trace(const char* where) {
  TORCH_CHECK(!torch::jit::tracer::isTracing(), where, " cannot be recorded by torch.jit.trace");
}

// A forward-mode tangent of an input would be dropped, which is a derivative of
// zero. (no_grad() does not switch forward mode off.)
void no_tangent(const char* where, std::initializer_list<const Tensor*> inputs) {
  for (const Tensor* t : inputs)
    TORCH_CHECK(t == nullptr || !t->defined() || !t->_fw_grad(0).defined(), where,
                " has no forward-mode derivative");
}

// Codes and their products have no gradient, in their scales and bias neither:
// a call that autograd would have to record is refused.
void no_gradient(const char* where, std::initializer_list<const Tensor*> inputs) {
  no_trace(where);
  no_tangent(where, inputs);
  if (!at::GradMode::is_enabled()) return;
  for (const Tensor* t : inputs)
    TORCH_CHECK(t == nullptr || !t->requires_grad(), where,
                " has no gradient: call it under torch.no_grad() or on detached tensors");
}

hipStream_t stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

bool has(const Maybe& t) { return t.has_value() && t->defined(); }
const Tensor* ptr(const Maybe& t) { return has(t) ? &*t : nullptr; }

void on_gpu(const Tensor& t, const char* name, const Tensor* like = nullptr) {
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

Rows rows_of(const Tensor& t, const char* name) {
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

const float* floats(const Tensor& t, int64_t n, const char* name, const Tensor& like) {
  on_gpu(t, name, &like);
  TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, name, " must be float32, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.numel() == n && t.is_contiguous(), name, " must hold ", n, " contiguous values, holds ",
                    t.numel());
  return t.const_data_ptr<float>();
}

int64_t padded(int64_t cols) { return (cols + 127) / 128 * 128; }

// ------------------------------------------------------------------ norm
// x, residual and weight of a norm, checked.
struct Norm {
  Rows x, res;
  bool added;
  const void* w = nullptr;
  int dtype, wtype;
  Norm(const Tensor& x_, const Maybe& residual, const Maybe& weight) : added(has(residual)) {
    TORCH_CHECK_VALUE(x_.dim() >= 1, "x must have a dimension");
    if (added)
      TORCH_CHECK_VALUE(residual->sizes() == x_.sizes(), "residual must be ", x_.sizes(), ", got ",
                        residual->sizes());
    if (has(weight)) TORCH_CHECK_VALUE(weight->dim() == 1, "weight must have one dimension");
    on_gpu(x_, "x");
    dtype = wtype = dtype_of(x_, "x");
    x = rows_of(x_, "x");
    if (added) {
      on_gpu(*residual, "residual", &x_);
      TORCH_CHECK_TYPE(residual->scalar_type() == x_.scalar_type(), "residual must be ", x_.scalar_type(),
                       ", got ", residual->scalar_type());
      res = rows_of(*residual, "residual");
    }
    if (has(weight)) {
      on_gpu(*weight, "weight", &x_);
      wtype = dtype_of(*weight, "weight");
      TORCH_CHECK_VALUE(weight->numel() == x.cols && weight->is_contiguous(), "weight must hold ", x.cols,
                        " contiguous values, holds ", weight->numel());
      w = weight->const_data_ptr();
    }
  }
  const void* res_p() const { return added ? res.p() : nullptr; }
  int64_t res_ld() const { return added ? res.ld : x.cols; }
};

Tensor like_rows(const Tensor& x) { return at::empty_like(x, x.options(), at::MemoryFormat::Contiguous); }

struct NormOut {
  Tensor y, h, rstd;  // h and rstd undefined where not asked for
};

NormOut norm_forward(const Tensor& x, const Maybe& residual, const Maybe& weight, double eps, bool want_rstd) {
  const Norm n(x, residual, weight);
  const c10::DeviceGuard guard(x.device());
  NormOut o;
  if (n.added) o.h = like_rows(x);
  o.y = like_rows(x);
  if (want_rstd) o.rstd = at::empty({n.x.rows}, x.options().dtype(at::kFloat));
  check(mxfp4_rmsnorm(n.x.p(), n.x.ld, n.res_p(), n.res_ld(), n.w, n.wtype, n.x.rows, n.x.cols, (float)eps,
                      n.dtype, n.added ? o.h.data_ptr() : nullptr, n.x.cols, o.y.data_ptr(), n.x.cols,
                      want_rstd ? o.rstd.data_ptr<float>() : nullptr, stream_of(x)),
        "mxfp4_rmsnorm");
  return o;
}

struct RMSNormFunction : torch::autograd::Function<RMSNormFunction> {
  static variable_list forward(AutogradContext* ctx, const Tensor& x, const Maybe& residual, const Maybe& weight,
                               double eps) {
    const NormOut o = norm_forward(x, residual, weight, eps, true);
    const bool added = o.h.defined();
    ctx->set_materialize_grads(false);
    ctx->save_for_backward({added ? o.h : x, has(weight) ? *weight : Tensor(), o.rstd});
    ctx->saved_data["added"] = added;
    if (added) return {o.y, o.h};
    return {o.y};
  }

  // Runs on a thread of the autograd engine, without the GIL.
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    TORCH_CHECK(!at::GradMode::is_enabled(), "rms_norm has no second derivative");
    const auto saved = ctx->get_saved_variables();
    const Tensor &h = saved[0], &weight = saved[1], &rstd = saved[2];
    const bool added = ctx->saved_data["added"].toBool();
    // the edges are those of the tensors that were given
    const bool want_w = weight.defined() && ctx->needs_input_grad(added ? 2 : 1);
    const Tensor &dy = grads[0], dh = added && grads.size() > 1 ? grads[1] : Tensor();
    Tensor dx, dw, ws;
    if (!dy.defined()) {  // y was not used
      dx = dh;
      if (want_w) dw = at::zeros_like(weight);
    } else {
      no_tangent("the gradient of rms_norm", {&dy, &dh});
      const c10::DeviceGuard guard(h.device());
      const Rows rh = rows_of(h, "h"), ry = rows_of(dy, "dy");
      const bool more = dh.defined();
      const Rows rd = more ? rows_of(dh, "dh") : Rows{};
      dx = like_rows(h);
      size_t bytes = 0;
      if (want_w) {
        dw = at::empty_like(weight);
        bytes = mxfp4_rmsnorm_bwd_workspace_bytes(rh.rows, rh.cols);
        ws = at::empty({(int64_t)bytes}, h.options().dtype(at::kByte));
      }
      const int st = mxfp4_rmsnorm_bwd(
          ry.p(), ry.ld, more ? rd.p() : nullptr, more ? rd.ld : rh.cols, rh.p(), rh.ld,
          weight.defined() ? weight.const_data_ptr() : nullptr,
          weight.defined() ? dtype_of(weight, "weight") : dtype_of(h, "h"), rstd.const_data_ptr<float>(),
          rh.rows, rh.cols, dtype_of(h, "h"), dx.data_ptr(), rh.cols, want_w ? dw.data_ptr() : nullptr,
          want_w ? ws.data_ptr() : nullptr, bytes, stream_of(h));
      TORCH_CHECK(st == MXFP4_OK, "mxfp4_rmsnorm_bwd: ", mxfp4_status_string(st), " (", st, ")");
    }
    return {dx, added ? dx : Tensor(), dw, Tensor()};
  }
};

py::object rms_norm(const Tensor& x, const Maybe& weight, double eps, const Maybe& residual) {
  no_trace("rms_norm");
  no_tangent("rms_norm", {&x, ptr(weight), ptr(residual)});
  const bool grad = at::GradMode::is_enabled() &&
                    (x.requires_grad() || (has(residual) && residual->requires_grad()) ||
                     (has(weight) && weight->requires_grad()));
  if (grad) {
    const variable_list o = RMSNormFunction::apply(x, residual, weight, eps);
    return o.size() == 2 ? py::object(py::make_tuple(o[0], o[1])) : py::cast(o[0]);
  }
  const NormOut o = norm_forward(x, residual, weight, eps, false);
  return o.h.defined() ? py::object(py::make_tuple(o.y, o.h)) : py::cast(o.y);
}

struct Operand {
  Tensor codes, scales;
};

Operand new_operand(const Rows& x) {
  return {at::empty({x.rows, padded(x.cols)}, x.t.options().dtype(at::kChar)),
          at::empty({x.rows}, x.t.options().dtype(at::kFloat))};
}

Operand norm_int8(const Tensor& x, const Maybe& weight, double eps, const Maybe& residual, Tensor* h) {
  no_gradient("rms_norm_int8", {&x, ptr(weight), ptr(residual)});
  const Norm n(x, residual, weight);
  const c10::DeviceGuard guard(x.device());
  Operand o = new_operand(n.x);
  if (n.added) *h = like_rows(x);
  check(mxfp4_rmsnorm_int8(n.x.p(), n.x.ld, n.res_p(), n.res_ld(), n.w, n.wtype, n.x.rows, n.x.cols,
                           (float)eps, n.dtype, n.added ? h->data_ptr() : nullptr, n.x.cols,
                           o.codes.data_ptr(), o.codes.size(1), o.scales.data_ptr<float>(), stream_of(x)),
        "mxfp4_rmsnorm_int8");
  return o;
}

py::tuple rms_norm_int8(const Tensor& x, const Maybe& weight, double eps, const Maybe& residual) {
  Tensor h;
  const Operand o = norm_int8(x, weight, eps, residual, &h);
  return h.defined() ? py::make_tuple(o.codes, o.scales, h) : py::make_tuple(o.codes, o.scales);
}

// ------------------------------------------------------------ 8 bits
Operand quantize(const Tensor& x, const Maybe& gate) {
  no_gradient("int8_quantize", {&x, ptr(gate)});
  if (has(gate)) TORCH_CHECK_VALUE(gate->sizes() == x.sizes(), "gate must be ", x.sizes(), ", got ", gate->sizes());
  on_gpu(x, "x");
  const int dtype = dtype_of(x, "x");
  const Rows r = rows_of(x, "x");
  Rows g{};
  if (has(gate)) {
    on_gpu(*gate, "gate", &x);
    TORCH_CHECK_TYPE(gate->scalar_type() == x.scalar_type(), "gate must be ", x.scalar_type(), ", got ",
                     gate->scalar_type());
    g = rows_of(*gate, "gate");
  }
  const c10::DeviceGuard guard(x.device());
  Operand o = new_operand(r);
  check(mxfp4_int8_quantize(r.p(), r.ld, has(gate) ? g.p() : nullptr, has(gate) ? g.ld : r.cols, r.rows,
                            r.cols, dtype, o.codes.data_ptr(), o.codes.size(1), o.scales.data_ptr<float>(),
                            stream_of(x)),
        "mxfp4_int8_quantize");
  return o;
}

py::tuple int8_quantize(const Tensor& x, const Maybe& gate) {
  const Operand o = quantize(x, gate);
  return py::make_tuple(o.codes, o.scales);
}

// Codes [rows][>= K] of which the first K columns are multiplied.
const void* codes_of(const Tensor& t, int64_t K, const char* name, const Tensor* like, int64_t* ld) {
  on_gpu(t, name, like);
  TORCH_CHECK_TYPE(t.scalar_type() == at::kChar, name, " must be int8, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == 2 && t.size(1) >= K, name, " must be [rows][", K, "], got ", t.sizes());
  TORCH_CHECK_VALUE((t.stride(1) == 1 || K == 1) && (t.stride(0) >= K || t.size(0) <= 1), name,
                    " must have a unit column stride and rows that do not overlap");
  *ld = t.size(0) > 1 ? t.stride(0) : padded(K);  // one row has no pitch
  return t.const_data_ptr();
}

Tensor gemm(const Tensor& a, const Tensor& sa, const Tensor& b, const Tensor& sb, const Maybe& bias, int64_t K,
            at::ScalarType out) {
  no_gradient("int8_gemm", {&sa, &sb, ptr(bias)});
  int64_t lda, ldb;
  const void* pa = codes_of(a, K, "a", nullptr, &lda);
  const void* pb = codes_of(b, K, "b", &a, &ldb);
  const int64_t M = a.size(0), N = b.size(0);
  const float *psa = floats(sa, M, "a_scales", a), *psb = floats(sb, N, "b_scales", a);
  const float* pbias = has(bias) ? floats(*bias, N, "bias", a) : nullptr;
  const c10::DeviceGuard guard(a.device());
  const Tensor c = at::empty({M, N}, a.options().dtype(out));
  const int dtype = dtype_of(c, "out_dtype");
  const size_t bytes = mxfp4_int8_gemm_workspace_bytes(M, N, K);
  Tensor ws;
  if (bytes) ws = at::empty({(int64_t)bytes}, a.options().dtype(at::kByte));
  check(mxfp4_int8_gemm(pa, lda, psa, pb, ldb, psb, pbias, M, N, K, c.data_ptr(), N, dtype,
                        bytes ? ws.data_ptr() : nullptr, bytes, stream_of(a)),
        "mxfp4_int8_gemm");
  return c;
}

Tensor int8_gemm(const Tensor& a, const Tensor& sa, const Tensor& b, const Tensor& sb, const Maybe& bias,
                 at::ScalarType out) {
  TORCH_CHECK_VALUE(a.dim() == 2 && b.dim() == 2 && a.size(1) == b.size(1), "a and b must be [M][K] and [N][K], got ",
                    a.sizes(), " and ", b.sizes());
  return gemm(a, sa, b, sb, bias, a.size(1), out);
}

// The product of quantized rows with a weight that is padded as they are (then
// over the zero codes too), or that has just the rows' own columns.
Tensor product(const Operand& x, const Tensor& w, const Tensor& sw, const Maybe& bias, at::ScalarType out) {
  return gemm(x.codes, x.scales, w, sw, bias, w.size(1), out);
}

void check_weight(const Tensor& w, int64_t cols, const char* name) {
  TORCH_CHECK_VALUE(w.dim() == 2 && (w.size(1) == cols || w.size(1) == padded(cols)), name, " must have ", cols,
                    " or ", padded(cols), " columns, got ", w.sizes());
}

Tensor as(const Tensor& y, const Tensor& x) {  // y [rows][N] with x's leading dimensions
  if (x.dim() == 2) return y;
  auto s = x.sizes().vec();
  s.back() = y.size(1);
  return y.view(s);
}

Tensor int8_linear(const Tensor& x, const Tensor& w, const Tensor& sw, const Maybe& bias,
                   std::optional<at::ScalarType> out) {
  TORCH_CHECK_VALUE(x.dim() >= 1, "x must have a dimension");
  check_weight(w, x.size(-1), "weight codes");
  no_gradient("int8_linear", {&x, &sw, ptr(bias)});
  const Operand q = quantize(x, {});
  return as(product(q, w, sw, bias, out.value_or(x.scalar_type())), x);
}

py::tuple int8_mlp(const Tensor& x, const Maybe& weight, double eps, const Tensor& gu, const Tensor& gus,
                   const Tensor& down, const Tensor& downs, const Maybe& residual) {
  TORCH_CHECK_VALUE(x.dim() >= 1, "x must have a dimension");
  check_weight(gu, x.size(-1), "gate_up codes");
  TORCH_CHECK_VALUE(gu.size(0) % 2 == 0, "gate_up must have an even number of rows, got ", gu.size(0));
  const int64_t F = gu.size(0) / 2;
  check_weight(down, F, "down codes");
  no_gradient("int8_mlp", {&x, ptr(weight), ptr(residual), &gus, &downs});
  Tensor h;
  const Operand q = norm_int8(x, weight, eps, residual, &h);
  const Tensor mid = product(q, gu, gus, {}, x.scalar_type());
  const Operand z = quantize(mid.narrow(1, F, F), mid.narrow(1, 0, F));
  const Tensor y = as(product(z, down, downs, {}, x.scalar_type()), x);
  return py::make_tuple(y, h.defined() ? h : x);
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  namespace p = pybind11;
  m.def("rms_norm", &rms_norm, p::arg("x"), p::arg("weight"), p::arg("eps"), p::arg("residual"));
  m.def("rms_norm_int8", &rms_norm_int8, p::arg("x"), p::arg("weight"), p::arg("eps"), p::arg("residual"));
  m.def("int8_quantize", &int8_quantize, p::arg("x"), p::arg("gate"));
  m.def("int8_gemm", &int8_gemm, p::arg("a"), p::arg("a_scales"), p::arg("b"), p::arg("b_scales"),
        p::arg("bias"), p::arg("out_dtype"));
  m.def("int8_linear", &int8_linear, p::arg("x"), p::arg("w"), p::arg("w_scales"), p::arg("bias"),
        p::arg("out_dtype"));
  m.def("int8_mlp", &int8_mlp, p::arg("x"), p::arg("norm_weight"), p::arg("eps"), p::arg("gate_up"),
        p::arg("gate_up_scales"), p::arg("down"), p::arg("down_scales"), p::arg("residual"));
}
