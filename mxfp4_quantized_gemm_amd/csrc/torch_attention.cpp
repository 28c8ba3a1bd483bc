// Torch binding of attention's operators: as torch_ops.cpp, checks, allocation
// and the autograd node around the C ABI.
#include <cmath>
#include <vector>

#include "torch_common.h"

namespace mx {
namespace {

typedef std::optional<std::vector<int64_t>> Sections;

// t [..., heads, dim] as heads of tokens: a view where its strides allow it.
struct HeadRows {
  Tensor t;
  int64_t tokens, dim;
  mxfp4_heads h;
};

HeadRows heads_of(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.dim() >= 2, name, " must be [..., heads, dim], got ", t.sizes());
  HeadRows r{t, 1, t.size(-1), {}};
  for (int64_t i = 0; i + 2 < t.dim(); ++i) r.tokens *= t.size(i);
  const int64_t heads = t.size(-2);
  if (t.dim() != 3) r.t = t.reshape({r.tokens, heads, r.dim});
  if (r.t.stride(2) != 1 && r.dim > 1) r.t = r.t.clone(at::MemoryFormat::Contiguous);
  r.h = {r.t.const_data_ptr(), heads, r.tokens > 1 ? r.t.stride(0) : 0, heads > 1 ? r.t.stride(1) : 0};
  return r;
}

// Sizes of t's tokens: all but the last two.
at::IntArrayRef tokens_of(const Tensor& t) { return t.sizes().slice(0, t.dim() - 2); }

// Checks that y has x's device, type, tokens and dim.
void like_heads(const Tensor& y, const char* name, const Tensor& x) {
  on_gpu(y, name, &x);
  TORCH_CHECK_TYPE(y.scalar_type() == x.scalar_type(), name, " must be ", x.scalar_type(), ", got ",
                   y.scalar_type());
  TORCH_CHECK_VALUE(y.dim() == x.dim() && tokens_of(y) == tokens_of(x) && y.size(-1) == x.size(-1), name,
                    " must have the tokens and the width of ", x.sizes(), ", got ", y.sizes());
}

const Tensor& whole(const Tensor& t, at::ScalarType type, const char* name, const Tensor& like) {
  on_gpu(t, name, &like);
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  return t;
}

// The rotation of heads with these tokens.
struct Rotation {
  Tensor positions, frequencies;
  mxfp4_rotation r{};
};

Rotation rotation_of(const Tensor& positions, const Tensor& frequencies, const Sections& sections, bool interleaved,
                     at::IntArrayRef lead, int64_t dim, const Tensor& like) {
  Rotation o;
  whole(frequencies, at::kDouble, "frequencies", like);
  whole(positions, at::kLong, "positions", like);
  TORCH_CHECK_VALUE(frequencies.dim() == 1 && 2 * frequencies.numel() <= dim,
                    "frequencies must be one dimension of at most ", dim / 2, " values, got ", frequencies.sizes());
  o.frequencies = frequencies.contiguous();
  o.r.pairs = frequencies.numel();
  o.r.axes = 1;
  o.r.axis_pairs[0] = o.r.pairs;
  o.r.interleaved = interleaved;
  std::vector<int64_t> want(lead.begin(), lead.end());
  if (sections.has_value()) {
    const int64_t n = (int64_t)sections->size();
    int64_t sum = 0;
    bool fine = n >= 1 && n <= 4;
    for (int64_t i = 0; fine && i < n; ++i) {
      fine = (*sections)[i] >= 0 && (*sections)[i] <= o.r.pairs;
      o.r.axis_pairs[i] = (*sections)[i];
      sum += (*sections)[i];
    }
    TORCH_CHECK_VALUE(fine && sum == o.r.pairs, "sections must be 1 to 4 counts of pairs that sum to ", o.r.pairs);
    o.r.axes = (int32_t)n;
    want.insert(want.begin(), n);
  }
  TORCH_CHECK_VALUE(positions.sizes() == at::IntArrayRef(want), "positions must be ", at::IntArrayRef(want), ", got ",
                    positions.sizes());
  o.positions = positions.contiguous();
  o.r.positions = o.positions.const_data_ptr<int64_t>();
  o.r.frequencies = o.frequencies.const_data_ptr<double>();
  return o;
}

struct HeadNorm {
  const void *qw = nullptr, *kw = nullptr;
  int type;
  float eps;
};

HeadNorm head_norm(const Maybe& qw, const Maybe& kw, std::optional<double> eps, int64_t dim, const Tensor& like) {
  HeadNorm n{nullptr, nullptr, dtype_of(like, "q"), -1.f};
  if (eps.has_value()) {
    n.eps = (float)*eps;
    // (one that fp32 has not would be infinity, and every result 0, or 0, and rows of zeros NaN)
    TORCH_CHECK_VALUE(*eps >= 0 && std::isfinite(n.eps) && (n.eps > 0 || *eps == 0),
                      "eps must be 0, a positive number in fp32's range, or None, got ", *eps);
  }
  TORCH_CHECK_VALUE(eps.has_value() || (!has(qw) && !has(kw)), "weights need a norm: eps is None");
  if (has(qw) && has(kw))
    TORCH_CHECK_TYPE(qw->scalar_type() == kw->scalar_type(), "q_weight and k_weight must be of one type, got ",
                     qw->scalar_type(), " and ", kw->scalar_type());
  const auto one = [&](const Maybe& w, const char* name) -> const void* {
    if (!has(w)) return nullptr;
    on_gpu(*w, name, &like);
    n.type = dtype_of(*w, name);
    TORCH_CHECK_VALUE(w->dim() == 1 && w->numel() == dim && w->is_contiguous(), name, " must hold ", dim,
                      " contiguous values, got ", w->sizes());
    return w->const_data_ptr();
  };
  n.qw = one(qw, "q_weight");
  n.kw = one(kw, "k_weight");
  return n;
}

Tensor dense_like(const Tensor& t) { return at::empty(t.sizes(), t.options()); }

// ------------------------------------------------- norm and rotation
// What the node's forward pass takes beside tensors that have gradients.
struct Turn {
  Tensor positions, frequencies;
  std::optional<double> eps;
  Sections sections;
  bool interleaved;
};

// (q', k'), and the heads' factors where `rstd` is given and there is a norm.
std::pair<Tensor, Tensor> turn_forward(const Tensor& q, const Tensor& k, const Maybe& qw, const Maybe& kw,
                                       const Turn& u, Tensor* rstd) {
  on_gpu(q, "q");
  const int dtype = dtype_of(q, "q");
  const HeadRows rq = heads_of(q, "q");
  like_heads(k, "k", q);
  const HeadNorm n = head_norm(qw, kw, u.eps, rq.dim, q);
  const c10::DeviceGuard guard(q.device());
  const HeadRows rk = heads_of(k, "k");
  const Rotation rot = rotation_of(u.positions, u.frequencies, u.sections, u.interleaved, tokens_of(q), rq.dim, q);
  const Tensor qo = dense_like(q), ko = dense_like(k);
  float* r = nullptr;
  if (rstd != nullptr && u.eps.has_value()) {
    *rstd = at::empty({rq.tokens, rq.h.heads + rk.h.heads}, q.options().dtype(at::kFloat));
    r = rstd->data_ptr<float>();
  }
  check(mxfp4_qk_norm_rope(&rq.h, &rk.h, rq.tokens, rq.dim, dtype, &rot.r, n.qw, n.kw, n.type, n.eps, qo.data_ptr(),
                           ko.data_ptr(), r, stream_of(q)),
        "mxfp4_qk_norm_rope");
  return {qo, ko};
}

struct TurnFunction : torch::autograd::Function<TurnFunction> {
  // Without a norm the gradient is dy turned back: the heads themselves are not kept, and may change.
  static variable_list forward(AutogradContext* ctx, const Tensor& q, const Tensor& k, const Maybe& qw,
                               const Maybe& kw, const Turn& u) {
    Tensor rstd;
    const auto o = turn_forward(q, k, qw, kw, u, &rstd);
    const bool norm = u.eps.has_value();
    ctx->set_materialize_grads(false);
    ctx->save_for_backward({norm ? q : Tensor(), norm ? k : Tensor(), has(qw) ? *qw : Tensor(),
                            has(kw) ? *kw : Tensor(), u.positions, u.frequencies, rstd});
    ctx->saved_data["q_sizes"] = q.sizes().vec();
    ctx->saved_data["k_sizes"] = k.sizes().vec();
    ctx->saved_data["eps"] = norm ? c10::IValue(*u.eps) : c10::IValue();
    ctx->saved_data["sections"] = u.sections.has_value() ? c10::IValue(*u.sections) : c10::IValue();
    ctx->saved_data["interleaved"] = u.interleaved;
    return {o.first, o.second};
  }

  // Runs on a thread of the autograd engine, without the GIL.
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    TORCH_CHECK(!at::GradMode::is_enabled(), "qk_norm_rope has no second derivative");
    const auto saved = ctx->get_saved_variables();
    const Tensor &q = saved[0], &k = saved[1], &qw = saved[2], &kw = saved[3];
    const auto &e = ctx->saved_data["eps"], &se = ctx->saved_data["sections"];
    Turn u{saved[4], saved[5], {}, {}, ctx->saved_data["interleaved"].toBool()};
    if (!e.isNone()) u.eps = e.toDouble();
    if (!se.isNone()) u.sections = se.toIntVector();
    // the edges are those of the tensors that were given
    const bool want_qw = qw.defined() && ctx->needs_input_grad(2),
               want_kw = kw.defined() && ctx->needs_input_grad(qw.defined() ? 3 : 2);
    const Tensor &dq = grads[0], &dk = grads[1];
    Tensor rstd = saved[6];
    no_tangent("the gradient of qk_norm_rope", {&dq, &dk});
    const auto q_sizes = ctx->saved_data["q_sizes"].toIntVector(), k_sizes = ctx->saved_data["k_sizes"].toIntVector();
    const auto has_heads = [](const Tensor& dy) { return dy.defined() && dy.size(-2) > 0; };
    if (!has_heads(dq) && !has_heads(dk)) {
      // nothing to turn back (and rstd has no values then, whose address would say that there was no norm)
      const auto zeros = [](bool want, const Tensor& t) { return want ? at::zeros_like(t) : Tensor(); };
      return {zeros(dq.defined(), dq), zeros(dk.defined(), dk), zeros(want_qw, qw), zeros(want_kw, kw), Tensor()};
    }
    const Tensor& like = dq.defined() ? dq : dk;
    const c10::DeviceGuard guard(like.device());
    const at::IntArrayRef lead(q_sizes.data(), q_sizes.size() - 2);
    const int64_t dim = q_sizes.back();
    const HeadNorm n = head_norm(qw.defined() ? Maybe(qw) : Maybe(), kw.defined() ? Maybe(kw) : Maybe(), u.eps,
                                 dim, like);
    const Rotation rot = rotation_of(u.positions, u.frequencies, u.sections, u.interleaved, lead, dim, like);
    // an output that no loss reads has no heads here, and its input no gradient
    HeadRows rq{}, rk{}, rdq{}, rdk{};
    Tensor dqx, dkx, dqw, dkw, ws;
    const auto side = [&](const Tensor& x, const Tensor& dy, const std::vector<int64_t>& sizes, const char* name,
                          HeadRows& rx, HeadRows& rdy, Tensor& dx) {
      if (!dy.defined()) return;
      rdy = heads_of(dy, name);
      dx = at::empty(sizes, dy.options());
      if (x.defined()) rx = heads_of(x, name);
      rx.h.heads = rdy.h.heads;
    };
    side(q, dq, q_sizes, "q", rq, rdq, dqx);
    side(k, dk, k_sizes, "k", rk, rdk, dkx);
    const int64_t tokens = (dq.defined() ? rdq : rdk).tokens, heads = q_sizes[lead.size()];
    if (rstd.defined() && dq.defined() != dk.defined())
      rstd = (dq.defined() ? rstd.narrow(1, 0, heads) : rstd.narrow(1, heads, k_sizes[lead.size()])).contiguous();
    if (want_qw) dqw = dq.defined() ? at::empty_like(qw) : at::zeros_like(qw);
    if (want_kw) dkw = dk.defined() ? at::empty_like(kw) : at::zeros_like(kw);
    const auto out = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    size_t bytes = 0;
    if (want_qw || want_kw) {
      bytes = mxfp4_qk_norm_rope_bwd_workspace_bytes(tokens, rq.h.heads, rk.h.heads, dim);
      ws = at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
    }
    const int st = mxfp4_qk_norm_rope_bwd(&rdq.h, &rdk.h, &rq.h, &rk.h, tokens, dim, dtype_of(like, "dq"), &rot.r,
                                          n.qw, n.kw, n.type, rstd.defined() ? rstd.const_data_ptr<float>() : nullptr,
                                          out(dqx), out(dkx), out(dqw), out(dkw), out(ws), bytes, stream_of(like));
    TORCH_CHECK(st == MXFP4_OK, "mxfp4_qk_norm_rope_bwd: ", mxfp4_status_string(st), " (", st, ")");
    return {dqx, dkx, dqw, dkw, Tensor()};
  }
};

py::tuple qk_norm_rope(const Tensor& q, const Tensor& k, const Tensor& positions, const Tensor& frequencies,
                       const Maybe& qw, const Maybe& kw, std::optional<double> eps, const Sections& sections,
                       bool interleaved) {
  no_gradient("the rotation's frequencies", {&frequencies});
  no_trace("qk_norm_rope");
  no_tangent("qk_norm_rope", {&q, &k, ptr(qw), ptr(kw)});
  const Turn u{positions, frequencies, eps, sections, interleaved};
  if (at::GradMode::is_enabled() && (q.requires_grad() || k.requires_grad() || (has(qw) && qw->requires_grad()) ||
                                     (has(kw) && kw->requires_grad()))) {
    const variable_list o = TurnFunction::apply(q, k, qw, kw, u);
    return py::make_tuple(o[0], o[1]);
  }
  const auto o = turn_forward(q, k, qw, kw, u, nullptr);
  return py::make_tuple(o.first, o.second);
}

// ------------------------------------------------------------- cache
struct Cache {
  const Tensor &k, &ks, &v, &vs;
};

mxfp4_int8_kv cache_of(const Cache& c, int64_t dim) {
  on_gpu(c.k, "cache k");
  on_gpu(c.v, "cache v", &c.k);
  const auto codes = [](const Tensor& t, const char* name) {
    TORCH_CHECK_TYPE(t.scalar_type() == at::kChar, name, " must be int8, got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == 4 && t.is_contiguous(), name,
                      " must be a contiguous [pages][heads][page size][pitch], got ", t.sizes());
  };
  codes(c.k, "cache k");
  codes(c.v, "cache v");
  TORCH_CHECK_VALUE(c.v.sizes() == c.k.sizes(), "cache v must be ", c.k.sizes(), ", got ", c.v.sizes());
  const int64_t pitch = (dim + 63) / 64 * 64;
  TORCH_CHECK_VALUE(dim >= 1 && c.k.size(3) == pitch, "a cache of heads of ", dim, " has a pitch of ", pitch, ", got ",
                    c.k.size(3));
  TORCH_CHECK_VALUE(c.k.size(0) >= 1 && c.k.size(1) >= 1 && c.k.size(2) >= 16 && c.k.size(2) % 16 == 0,
                    "a cache has pages of a multiple of 16 tokens, got ", c.k.sizes());
  const auto scales = [&](const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.dim() == 3 && t.sizes() == c.k.sizes().slice(0, 3), name, " must be ",
                      c.k.sizes().slice(0, 3), ", got ", t.sizes());
    return const_cast<float*>(floats(t, t.numel(), name, c.k));
  };
  mxfp4_int8_kv r{};
  r.k = c.k.data_ptr();
  r.k_scales = scales(c.ks, "cache k_scales");
  r.v = c.v.data_ptr();
  r.v_scales = scales(c.vs, "cache v_scales");
  r.pages = c.k.size(0);
  r.heads = c.k.size(1);
  r.page_size = c.k.size(2);
  r.pitch = c.k.size(3);
  return r;
}

const int64_t* slots_of(const Tensor& slots, at::IntArrayRef lead, const Tensor& like) {
  whole(slots, at::kLong, "slots", like);
  TORCH_CHECK_VALUE(slots.sizes() == lead && slots.is_contiguous(), "slots must be a contiguous ", lead, ", got ",
                    slots.sizes());
  return slots.const_data_ptr<int64_t>();
}

// Autograd counts the changes of what it has saved (scales that a caller's graph reads, say).
void written(const Cache& c) {
  for (const Tensor* t : {&c.k, &c.ks, &c.v, &c.vs})
    if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

void heads_like_cache(const Tensor& t, const char* name, const mxfp4_int8_kv& c) {
  TORCH_CHECK_VALUE(t.size(-2) == c.heads, name, " must have the cache's ", c.heads, " heads, got ", t.sizes());
}

void int8_kv_write(const Tensor& k, const Tensor& v, const Tensor& ck, const Tensor& cks, const Tensor& cv,
                   const Tensor& cvs, const Tensor& slots) {
  no_gradient("int8_kv_write", {&k, &v, &cks, &cvs});
  on_gpu(k, "k");
  const int dtype = dtype_of(k, "k");
  const HeadRows rk = heads_of(k, "k");
  like_heads(v, "v", k);
  on_gpu(ck, "cache k", &k);
  const mxfp4_int8_kv c = cache_of({ck, cks, cv, cvs}, rk.dim);
  heads_like_cache(k, "k", c);
  heads_like_cache(v, "v", c);
  const int64_t* s = slots_of(slots, tokens_of(k), k);
  const c10::DeviceGuard guard(k.device());
  const HeadRows rv = heads_of(v, "v");
  check(mxfp4_int8_kv_write(nullptr, &rk.h, &rv.h, rk.tokens, rk.dim, dtype, nullptr, nullptr, nullptr, dtype, -1.f,
                            &c, s, nullptr, stream_of(k)),
        "mxfp4_int8_kv_write");
  written({ck, cks, cv, cvs});
}

Tensor int8_kv_append(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& ck, const Tensor& cks,
                      const Tensor& cv, const Tensor& cvs, const Tensor& slots, const Tensor& positions,
                      const Tensor& frequencies, const Maybe& qw, const Maybe& kw, std::optional<double> eps,
                      const Sections& sections, bool interleaved) {
  no_gradient("int8_kv_append", {&q, &k, &v, &cks, &cvs, &frequencies, ptr(qw), ptr(kw)});
  on_gpu(q, "q");
  const int dtype = dtype_of(q, "q");
  const HeadRows rq = heads_of(q, "q");
  like_heads(k, "k", q);
  like_heads(v, "v", q);
  on_gpu(ck, "cache k", &q);
  const mxfp4_int8_kv c = cache_of({ck, cks, cv, cvs}, rq.dim);
  heads_like_cache(k, "k", c);
  heads_like_cache(v, "v", c);
  const int64_t* s = slots_of(slots, tokens_of(q), q);
  const HeadNorm n = head_norm(qw, kw, eps, rq.dim, q);
  const c10::DeviceGuard guard(q.device());
  const HeadRows rk = heads_of(k, "k"), rv = heads_of(v, "v");
  const Rotation rot = rotation_of(positions, frequencies, sections, interleaved, tokens_of(q), rq.dim, q);
  const Tensor qo = dense_like(q);
  check(mxfp4_int8_kv_write(&rq.h, &rk.h, &rv.h, rq.tokens, rq.dim, dtype, &rot.r, n.qw, n.kw, n.type, n.eps, &c, s,
                            qo.data_ptr(), stream_of(q)),
        "mxfp4_int8_kv_write");
  written({ck, cks, cv, cvs});
  return qo;
}

py::tuple int8_kv_read(const Tensor& ck, const Tensor& cks, const Tensor& cv, const Tensor& cvs, const Tensor& slots,
                       int64_t dim, at::ScalarType type) {
  no_gradient("int8_kv_read", {&cks, &cvs});
  const mxfp4_int8_kv c = cache_of({ck, cks, cv, cvs}, dim);
  const int64_t* s = slots_of(slots, slots.sizes(), ck);
  const c10::DeviceGuard guard(ck.device());
  auto size = slots.sizes().vec();
  size.push_back(c.heads);
  size.push_back(dim);
  const Tensor k = at::empty(size, ck.options().dtype(type)), v = at::empty(size, ck.options().dtype(type));
  check(mxfp4_int8_kv_read(&c, s, slots.numel(), dim, dtype_of(k, "dtype"), k.data_ptr(), v.data_ptr(),
                           stream_of(ck)),
        "mxfp4_int8_kv_read");
  return py::make_tuple(k, v);
}

// --------------------------------------------------------- attention
// Page tables [batch][columns] and lengths [batch].
struct Tables {
  Tensor pages;
  const int32_t* lengths;
};

Tables tables_of(const Tensor& pages, const Tensor& lengths, int64_t batch, const Tensor& like) {
  whole(pages, at::kInt, "pages", like);
  whole(lengths, at::kInt, "lengths", like);
  TORCH_CHECK_VALUE(pages.dim() == 2 && pages.size(0) == batch, "pages must be [", batch, "][pages of a sequence], got ",
                    pages.sizes());
  TORCH_CHECK_VALUE(lengths.dim() == 1 && lengths.numel() == batch && lengths.is_contiguous(),
                    "lengths must hold ", batch, " contiguous values, got ", lengths.sizes());
  Tables t{pages, lengths.const_data_ptr<int32_t>()};
  if ((pages.stride(1) != 1 && pages.size(1) > 1) || (pages.stride(0) < pages.size(1) && batch > 1))
    t.pages = pages.clone(at::MemoryFormat::Contiguous);
  return t;
}

int64_t pitch_of(const Tables& t, int64_t batch) { return batch > 1 ? t.pages.stride(0) : t.pages.size(1); }

// q.tokens sequences; out [sequences][heads][dim], dense.
void attend(const mxfp4_heads& q, int64_t batch, int64_t dim, int dtype, const mxfp4_int8_kv& c, const Tables& t,
            std::optional<double> scale, int64_t window, const Tensor& out, float* lse) {
  const int64_t table = t.pages.size(1), ld = pitch_of(t, batch);
  const size_t bytes = mxfp4_paged_attention_workspace_bytes(batch, q.heads, c.heads, dim, table, c.page_size);
  Tensor ws;
  if (bytes) ws = at::empty({(int64_t)bytes}, out.options().dtype(at::kByte));
  check(mxfp4_paged_attention(&q, batch, dim, dtype, &c, t.pages.const_data_ptr<int32_t>(), ld, table, t.lengths,
                              (float)scale.value_or(1.0 / std::sqrt((double)dim)), window, out.data_ptr(), lse,
                              bytes ? ws.data_ptr() : nullptr, bytes, stream_of(out)),
        "mxfp4_paged_attention");
}

void check_groups(int64_t q_heads, const mxfp4_int8_kv& c) {
  TORCH_CHECK_VALUE(q_heads >= 1 && q_heads % c.heads == 0, "query heads must be a multiple of the cache's ", c.heads,
                    ", got ", q_heads);
}

py::object paged_attention(const Tensor& q, const Tensor& ck, const Tensor& cks, const Tensor& cv, const Tensor& cvs,
                           const Tensor& pages, const Tensor& lengths, std::optional<double> scale, int64_t window,
                           bool return_lse) {
  no_gradient("paged_attention", {&q, &cks, &cvs});
  on_gpu(q, "q");
  const int dtype = dtype_of(q, "q");
  TORCH_CHECK_VALUE(q.dim() == 3, "q must be [batch][heads][dim], got ", q.sizes());
  TORCH_CHECK_VALUE(window >= 0, "window must be at least 0 (none), got ", window);
  on_gpu(ck, "cache k", &q);
  const mxfp4_int8_kv c = cache_of({ck, cks, cv, cvs}, q.size(2));
  check_groups(q.size(1), c);
  const c10::DeviceGuard guard(q.device());
  const HeadRows r = heads_of(q, "q");
  const Tables t = tables_of(pages, lengths, r.tokens, q);
  const Tensor out = dense_like(q);
  Tensor lse;
  if (return_lse) lse = at::empty({q.size(0), q.size(1)}, q.options().dtype(at::kFloat));
  attend(r.h, r.tokens, r.dim, dtype, c, t, scale, window, out, return_lse ? lse.data_ptr<float>() : nullptr);
  return return_lse ? py::object(py::make_tuple(out, lse)) : py::cast(out);
}

py::tuple int8_attention(const Tensor& x, const Maybe& weight, double eps, const Tensor& qkv, const Tensor& qkvs,
                         const Tensor& o, const Tensor& os, const Tensor& ck, const Tensor& cks, const Tensor& cv,
                         const Tensor& cvs, const Tensor& slots, const Tensor& pages, const Tensor& lengths,
                         const Tensor& positions, const Tensor& frequencies, const Maybe& qw, const Maybe& kw,
                         std::optional<double> qk_eps, int64_t dim, std::optional<double> scale, int64_t window,
                         const Sections& sections, bool interleaved, const Maybe& residual) {
  TORCH_CHECK_VALUE(x.dim() >= 1, "x must have a dimension");
  TORCH_CHECK_VALUE(window >= 0, "window must be at least 0 (none), got ", window);
  on_gpu(x, "x");
  on_gpu(ck, "cache k", &x);
  const int dtype = dtype_of(x, "x");
  const mxfp4_int8_kv c = cache_of({ck, cks, cv, cvs}, dim);
  check_weight(qkv, x.size(-1), "qkv codes");
  TORCH_CHECK_VALUE(qkv.size(0) % dim == 0, "qkv must have heads of ", dim, " rows, got ", qkv.size(0));
  const int64_t H = qkv.size(0) / dim - 2 * c.heads, wide = qkv.size(0);
  check_groups(H, c);
  check_weight(o, H * dim, "out codes");
  no_gradient("int8_attention", {&x, ptr(weight), ptr(residual), &qkvs, &os, &cks, &cvs, &frequencies, ptr(qw), ptr(kw)});
  const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
  const int64_t* s = slots_of(slots, lead, x);
  const HeadNorm n = head_norm(qw, kw, qk_eps, dim, x);
  const Tables t = tables_of(pages, lengths, slots.numel(), x);
  const c10::DeviceGuard guard(x.device());
  const Rotation rot = rotation_of(positions, frequencies, sections, interleaved, lead, dim, x);
  // what the calls behind the write to the cache refuse (an attention of no sequence checks the sizes)
  check_product(o, os, x, "out");
  const mxfp4_heads none{nullptr, H, 0, 0};
  check(mxfp4_paged_attention(&none, 0, dim, dtype, &c, nullptr, pitch_of(t, slots.numel()), t.pages.size(1), nullptr,
                              1.f, window, nullptr, nullptr, nullptr, 0, nullptr),
        "mxfp4_paged_attention");
  Tensor h;
  const Operand in = norm_int8(x, weight, eps, residual, &h);
  const Tensor mid = product(in, qkv, qkvs, {}, x.scalar_type());
  const int64_t B = mid.size(0), size = mid.element_size();
  const char* p = static_cast<const char*>(mid.const_data_ptr());
  const mxfp4_heads q{p, H, wide, dim}, k{p + H * dim * size, c.heads, wide, dim},
      v{p + (H + c.heads) * dim * size, c.heads, wide, dim};
  const Tensor turned = at::empty({B, H * dim}, x.options()), out = at::empty({B, H * dim}, x.options());
  check(mxfp4_int8_kv_write(&q, &k, &v, B, dim, dtype, &rot.r, n.qw, n.kw, n.type, n.eps, &c, s, turned.data_ptr(),
                            stream_of(x)),
        "mxfp4_int8_kv_write");
  written({ck, cks, cv, cvs});
  attend({turned.const_data_ptr(), H, H * dim, dim}, B, dim, dtype, c, t, scale, window, out, nullptr);
  const Tensor y = as(product(quantize(out, {}), o, os, {}, x.scalar_type()), x);
  return py::make_tuple(y, h.defined() ? h : x);
}

}  // namespace

void bind_attention(pybind11::module_& m) {
  namespace p = pybind11;
  m.def("qk_norm_rope", &qk_norm_rope, p::arg("q"), p::arg("k"), p::arg("positions"), p::arg("frequencies"),
        p::arg("q_weight"), p::arg("k_weight"), p::arg("eps"), p::arg("sections"), p::arg("interleaved"));
  m.def("int8_kv_write", &int8_kv_write);
  m.def("int8_kv_append", &int8_kv_append);
  m.def("int8_kv_read", &int8_kv_read);
  m.def("paged_attention", &paged_attention);
  m.def("int8_attention", &int8_attention);
}

}  // namespace mx
