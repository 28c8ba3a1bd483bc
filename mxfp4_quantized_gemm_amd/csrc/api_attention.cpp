// C ABI of attention's operators: argument validation (host only, before any
// HIP call), as api.cpp does for the MXFP4 entry points.
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mxfp4.h"
#include "attention.h"

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 31;
constexpr int64_t kMaxOffset = int64_t(1) << 48;

bool valid_dtype(int t) { return t >= MXFP4_DT_F32 && t <= MXFP4_DT_F16; }
int size_of(int t) { return t == MXFP4_DT_F32 ? 4 : 2; }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ERR_HIP; }
bool dim_ok(int64_t dim) { return dim >= 1 && dim <= mx::kHeadMax; }
bool tokens_ok(int64_t tokens) { return tokens >= 0 && tokens < kMaxTokens; }
bool count_ok(int64_t heads) { return heads >= 0 && heads <= mx::kHeadsMax; }

// Strides whose last offset fits.
bool heads_ok(const mxfp4_heads& x, int64_t tokens) {
  return count_ok(x.heads) && x.token_stride >= 0 && x.head_stride >= 0 &&
         x.token_stride <= kMaxOffset / (tokens > 0 ? tokens : 1) && x.head_stride <= kMaxOffset / mx::kHeadsMax;
}

mx::Heads heads_of(const mxfp4_heads& x) { return {x.p, x.heads, x.token_stride, x.head_stride}; }

// The rotation's sizes, and for tokens > 0 its pointers. NULL is one of no pairs.
int check_rotation(const mxfp4_rotation* r, int64_t tokens, int64_t dim, mxfp4_rotation* out) {
  *out = mxfp4_rotation{};
  out->axes = 1;
  if (r == nullptr) return MXFP4_OK;
  if (r->pairs < 0 || r->pairs > dim / 2) return MXFP4_ERR_SHAPE;
  if (r->pairs == 0) return MXFP4_OK;
  if (r->axes < 1 || r->axes > 4) return MXFP4_ERR_SHAPE;
  int64_t sum = 0;
  for (int i = 0; i < r->axes; ++i) {
    if (r->axis_pairs[i] < 0 || r->axis_pairs[i] > r->pairs) return MXFP4_ERR_SHAPE;
    sum += r->axis_pairs[i];
  }
  if (sum != r->pairs) return MXFP4_ERR_SHAPE;
  if (tokens > 0) {
    if (!r->positions || !r->frequencies) return MXFP4_ERR_NULL;
    if (!aligned(r->positions, 8) || !aligned(r->frequencies, 8)) return MXFP4_ERR_ALIGN;
  }
  *out = *r;
  return MXFP4_OK;
}

// Types of the norm; a call without one (eps < 0) has no weights.
int check_norm(int dtype, int weight_dtype, float eps, const void* qw, const void* kw) {
  if (!valid_dtype(dtype) || (weight_dtype != dtype && weight_dtype != MXFP4_DT_F32)) return MXFP4_ERR_MODE;
  if (isnan(eps) || (eps < 0.f && (qw || kw))) return MXFP4_ERR_MODE;
  if (!aligned(qw, size_of(weight_dtype)) || !aligned(kw, size_of(weight_dtype))) return MXFP4_ERR_ALIGN;
  return MXFP4_OK;
}

mx::HeadNorm norm_of(const void* qw, const void* kw, int dtype, int weight_dtype, float eps) {
  return {qw, kw, weight_dtype == MXFP4_DT_F32 && dtype != MXFP4_DT_F32, eps};
}

int64_t pitch_of(int64_t dim) { return (dim + 63) / 64 * 64; }

int check_cache(const mxfp4_int8_kv* c, int64_t dim) {
  if (c == nullptr) return MXFP4_ERR_NULL;
  if (c->pages < 1 || c->heads < 1 || c->heads > mx::kHeadsMax || c->page_size < mx::kPageUnit ||
      c->page_size % mx::kPageUnit || c->pitch != pitch_of(dim) || c->page_size >= kMaxTokens ||
      c->pages >= (kMaxTokens + c->page_size - 1) / c->page_size)
    return MXFP4_ERR_SHAPE;
  if (!c->k || !c->k_scales || !c->v || !c->v_scales) return MXFP4_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16))
    return MXFP4_ERR_ALIGN;
  return MXFP4_OK;
}

// Positions in a table, and those up to two parts of a line behind its end, are 32-bit numbers.
bool attention_sizes_ok(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t table,
                        int64_t page_size) {
  return tokens_ok(batch) && dim_ok(dim) && kv_heads >= 1 && q_heads >= 1 && q_heads <= mx::kHeadsMax &&
         q_heads % kv_heads == 0 && page_size >= mx::kPageUnit && page_size % mx::kPageUnit == 0 && table >= 0 &&
         table <= (kMaxTokens - 16384) / page_size;
}

}  // namespace

extern "C" {

int mxfp4_qk_norm_rope(const mxfp4_heads* q, const mxfp4_heads* k, int64_t tokens, int64_t dim,
                       int dtype, const mxfp4_rotation* rotation, const void* q_weight,
                       const void* k_weight, int weight_dtype, float eps, void* q_out, void* k_out,
                       float* rstd, hipStream_t stream) {
  if (!q || !k) return MXFP4_ERR_NULL;
  int st = check_norm(dtype, weight_dtype, eps, q_weight, k_weight);
  if (st != MXFP4_OK) return st;
  if (!dim_ok(dim) || !tokens_ok(tokens) || !heads_ok(*q, tokens) || !heads_ok(*k, tokens)) return MXFP4_ERR_SHAPE;
  mxfp4_rotation rot;
  if ((st = check_rotation(rotation, tokens, dim, &rot)) != MXFP4_OK) return st;
  if (tokens == 0 || q->heads + k->heads == 0) return MXFP4_OK;
  if ((q->heads && (!q->p || !q_out)) || (k->heads && (!k->p || !k_out))) return MXFP4_ERR_NULL;
  const int s = size_of(dtype);
  if (!aligned(q->p, s) || !aligned(k->p, s) || !aligned(q_out, s) || !aligned(k_out, s) ||
      !aligned(rstd, 4))
    return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_qk_norm_rope(heads_of(*q), heads_of(*k), tokens, dim, dtype, rot,
                                            norm_of(q_weight, k_weight, dtype, weight_dtype, eps), q_out, k_out,
                                            eps >= 0.f ? rstd : nullptr, stream));
}

size_t mxfp4_qk_norm_rope_bwd_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads,
                                              int64_t dim) {
  return tokens_ok(tokens) && dim_ok(dim) && count_ok(q_heads) && count_ok(k_heads)
             ? mx::qk_norm_rope_bwd_ws(tokens, q_heads, k_heads, dim)
             : 0;
}

int mxfp4_qk_norm_rope_bwd(const mxfp4_heads* dq, const mxfp4_heads* dk, const mxfp4_heads* q,
                           const mxfp4_heads* k, int64_t tokens, int64_t dim, int dtype,
                           const mxfp4_rotation* rotation, const void* q_weight, const void* k_weight,
                           int weight_dtype, const float* rstd, void* dq_out, void* dk_out, void* dq_weight,
                           void* dk_weight, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dq || !dk || !q || !k) return MXFP4_ERR_NULL;
  // (rstd has no values where there is no token or no head)
  const bool weights = dq_weight || dk_weight, norm = rstd != nullptr || tokens == 0 || (q->heads == 0 && k->heads == 0);
  int st = check_norm(dtype, weight_dtype, norm ? 0.f : -1.f, q_weight, k_weight);
  if (st != MXFP4_OK) return st;
  if (weights && !norm) return MXFP4_ERR_MODE;
  if (!dim_ok(dim) || !tokens_ok(tokens) || !heads_ok(*q, tokens) || !heads_ok(*k, tokens) ||
      !heads_ok(*dq, tokens) || !heads_ok(*dk, tokens) || dq->heads != q->heads || dk->heads != k->heads)
    return MXFP4_ERR_SHAPE;
  mxfp4_rotation rot;
  if ((st = check_rotation(rotation, tokens, dim, &rot)) != MXFP4_OK) return st;
  const int s = size_of(dtype), w = size_of(weight_dtype);
  if (!aligned(dq_weight, w) || !aligned(dk_weight, w)) return MXFP4_ERR_ALIGN;
  if (tokens == 0 && !weights) return MXFP4_OK;
  if (tokens > 0) {
    if ((q->heads && (!dq->p || !dq_out || (norm && !q->p))) || (k->heads && (!dk->p || !dk_out || (norm && !k->p))) ||
        (weights && !ws))
      return MXFP4_ERR_NULL;
    if (weights && ws_bytes < mx::qk_norm_rope_bwd_ws(tokens, q->heads, k->heads, dim)) return MXFP4_ERR_WORKSPACE;
  }
  if (!aligned(q->p, s) || !aligned(k->p, s) || !aligned(dq->p, s) || !aligned(dk->p, s) || !aligned(dq_out, s) ||
      !aligned(dk_out, s) || !aligned(rstd, 4) || !aligned(ws, 4))
    return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_qk_norm_rope_bwd(
      heads_of(*dq), heads_of(*dk), heads_of(*q), heads_of(*k), tokens, dim, dtype, rot,
      norm_of(q_weight, k_weight, dtype, weight_dtype, 0.f), rstd, dq_out, dk_out, dq_weight, dk_weight, ws, stream));
}

int mxfp4_int8_kv_write(const mxfp4_heads* q, const mxfp4_heads* k, const mxfp4_heads* v,
                        int64_t tokens, int64_t dim, int dtype, const mxfp4_rotation* rotation,
                        const void* q_weight, const void* k_weight, int weight_dtype, float eps,
                        const mxfp4_int8_kv* cache, const int64_t* slots, void* q_out,
                        hipStream_t stream) {
  if (!k || !v) return MXFP4_ERR_NULL;
  int st = check_norm(dtype, weight_dtype, eps, q_weight, k_weight);
  if (st != MXFP4_OK) return st;
  const mxfp4_heads none = {nullptr, 0, 0, 0}, *qh = q ? q : &none;
  if (!dim_ok(dim) || !tokens_ok(tokens) || !heads_ok(*qh, tokens) || !heads_ok(*k, tokens) || !heads_ok(*v, tokens))
    return MXFP4_ERR_SHAPE;
  if ((st = check_cache(cache, dim)) != MXFP4_OK) return st;
  if (k->heads != cache->heads || v->heads != cache->heads) return MXFP4_ERR_SHAPE;
  mxfp4_rotation rot;
  if ((st = check_rotation(rotation, tokens, dim, &rot)) != MXFP4_OK) return st;
  if (tokens == 0) return MXFP4_OK;
  if (!k->p || !v->p || !slots || (qh->heads && (!qh->p || !q_out))) return MXFP4_ERR_NULL;
  const int s = size_of(dtype);
  if (!aligned(qh->p, s) || !aligned(k->p, s) || !aligned(v->p, s) || !aligned(q_out, s) || !aligned(slots, 8))
    return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_int8_kv_write(heads_of(*qh), heads_of(*k), heads_of(*v), tokens, dim, dtype, rot,
                                             norm_of(q_weight, k_weight, dtype, weight_dtype, eps), *cache, slots,
                                             q_out, stream));
}

int mxfp4_int8_kv_read(const mxfp4_int8_kv* cache, const int64_t* slots, int64_t tokens, int64_t dim,
                       int dtype, void* k, void* v, hipStream_t stream) {
  if (!valid_dtype(dtype)) return MXFP4_ERR_MODE;
  if (!dim_ok(dim) || !tokens_ok(tokens)) return MXFP4_ERR_SHAPE;
  const int st = check_cache(cache, dim);
  if (st != MXFP4_OK || tokens == 0) return st;
  if (!slots || !k || !v) return MXFP4_ERR_NULL;
  const int s = size_of(dtype);
  if (!aligned(slots, 8) || !aligned(k, s) || !aligned(v, s)) return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_int8_kv_read(*cache, slots, tokens, dim, dtype, k, v, stream));
}

size_t mxfp4_paged_attention_workspace_bytes(int64_t batch, int64_t q_heads, int64_t kv_heads,
                                             int64_t dim, int64_t table, int64_t page_size) {
  return attention_sizes_ok(batch, q_heads, kv_heads, dim, table, page_size)
             ? mx::paged_attention_ws(batch, q_heads, kv_heads, dim, table, page_size)
             : 0;
}

int mxfp4_paged_attention(const mxfp4_heads* q, int64_t batch, int64_t dim, int dtype,
                          const mxfp4_int8_kv* cache, const int32_t* pages, int64_t pages_ld,
                          int64_t table, const int32_t* lengths, float scale, int64_t window,
                          void* out, float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!q) return MXFP4_ERR_NULL;
  if (!valid_dtype(dtype)) return MXFP4_ERR_MODE;
  if (!dim_ok(dim)) return MXFP4_ERR_SHAPE;
  const int st = check_cache(cache, dim);
  if (st != MXFP4_OK) return st;
  if (!attention_sizes_ok(batch, q->heads, cache->heads, dim, table, cache->page_size) || !heads_ok(*q, batch) ||
      window < 0 || pages_ld < table || pages_ld > kMaxOffset / (batch > 0 ? batch : 1))
    return MXFP4_ERR_SHAPE;
  if (batch == 0) return MXFP4_OK;
  const size_t need = mx::paged_attention_ws(batch, q->heads, cache->heads, dim, table, cache->page_size);
  if (!q->p || !lengths || !out || (table && !pages) || (need && !ws)) return MXFP4_ERR_NULL;
  if (ws_bytes < need) return MXFP4_ERR_WORKSPACE;
  const int s = size_of(dtype);
  if (!aligned(q->p, s) || !aligned(out, s) || !aligned(lse, 4) || !aligned(pages, 4) || !aligned(lengths, 4) ||
      !aligned(ws, 4))
    return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_paged_attention(heads_of(*q), batch, dim, dtype, *cache, pages, pages_ld, table,
                                               lengths, scale, window, out, lse, ws, stream));
}

}  // extern "C"
