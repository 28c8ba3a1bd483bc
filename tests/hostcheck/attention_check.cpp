// Host-only checks of attention's entry points (api_attention.cpp) against
// stand-ins for their launch layer that record each launch, and of the integer
// arithmetic that the attention kernel shares with the host (attention_plan.h).
// Nothing here touches device memory.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <vector>

#include "../../include/mxfp4.h"
#include "../../mxfp4_quantized_gemm_amd/csrc/attention.h"
#include "../../mxfp4_quantized_gemm_amd/csrc/attention_plan.h"

static int g_launches = 0, g_checks = 0;
static hipError_t g_result = hipSuccess;
static mxfp4_rotation g_rot;
static int64_t g_q_heads;

namespace mx {
hipError_t launch_qk_norm_rope(Heads q, Heads, int64_t, int64_t, int, const mxfp4_rotation& rot, HeadNorm, void*,
                               void*, float*, hipStream_t) {
  ++g_launches;
  g_rot = rot;
  g_q_heads = q.heads;
  return g_result;
}
hipError_t launch_qk_norm_rope_bwd(Heads, Heads, Heads, Heads, int64_t, int64_t, int, const mxfp4_rotation& rot,
                                   HeadNorm, const float*, void*, void*, void*, void*, void*, hipStream_t) {
  ++g_launches;
  g_rot = rot;
  return g_result;
}
size_t qk_norm_rope_bwd_ws(int64_t tokens, int64_t, int64_t, int64_t dim) { return (size_t)(tokens < 4 ? tokens : 4) * dim * 8; }
hipError_t launch_int8_kv_write(Heads q, Heads, Heads, int64_t, int64_t, int, const mxfp4_rotation& rot, HeadNorm,
                                const mxfp4_int8_kv&, const int64_t*, void*, hipStream_t) {
  ++g_launches;
  g_rot = rot;
  g_q_heads = q.heads;
  return g_result;
}
hipError_t launch_int8_kv_read(const mxfp4_int8_kv&, const int64_t*, int64_t, int64_t, int, void*, void*, hipStream_t) {
  ++g_launches;
  return g_result;
}
hipError_t launch_paged_attention(Heads, int64_t, int64_t, int, const mxfp4_int8_kv&, const int32_t*, int64_t, int64_t,
                                  const int32_t*, float, int64_t, void*, float*, void*, hipStream_t) {
  ++g_launches;
  return g_result;
}
size_t paged_attention_ws(int64_t, int64_t, int64_t, int64_t, int64_t table, int64_t page_size) {
  return table * page_size > kUnit ? 1024 : 0;
}
}  // namespace mx

#define CHECK(cond)                                                  \
  do {                                                               \
    ++g_checks;                                                      \
    if (!(cond)) {                                                   \
      printf("FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond);       \
      exit(1);                                                       \
    }                                                                \
  } while (0)

static void* at(uintptr_t a) { return reinterpret_cast<void*>(a); }

static void plan() {
  // the division by a page's sixteenths: every divisor that a page below 2^31
  // tokens has near powers of two and at random, at the borders of each quotient
  std::mt19937_64 rng(1);
  std::vector<uint32_t> ds;
  for (uint32_t s = 0; s < 27; ++s)
    for (int e = -2; e <= 2; ++e) ds.push_back((1u << s) + e);
  for (int i = 0; i < 2000; ++i) ds.push_back(1 + rng() % ((1u << (1 + rng() % 27)) - 1 + 1));
  for (uint32_t d : ds) {
    if (d < 1 || d >= 1u << 27) continue;
    const mx::Divisor m = mx::divisor_of(d);
    for (int i = 0; i < 200; ++i) {
      const uint32_t q = (uint32_t)(rng() % (((1u << 27) - 1) / d + 1));
      for (int64_t x : {(int64_t)q * d - 1, (int64_t)q * d, (int64_t)q * d + d - 1, (int64_t)(rng() % (1u << 27))})
        if (x >= 0 && x < 1 << 27) CHECK(mx::divided((uint32_t)x, m) == (uint32_t)x / d);
    }
    CHECK(mx::divided((1u << 27) - 1, m) == ((1u << 27) - 1) / d);
  }
  // spans: every token that counts lies in a unit, none of the units is empty
  const int big = 0x7fffffff - 1023;
  for (int most : {0, 16, 48, 1 << 20, big})
    for (int n : {-5, 0, 1, 15, 16, 17, 127, 128, 129, 4097, 1 << 20, big, 0x7fffffff})
      for (int w : {0, 1, 2, 16, 17, 100, 4096, big - 1}) {
        const mx::Span s = mx::span_of(n, most, w);
        CHECK(s.n == std::min(std::max(n, 0), most));
        CHECK(s.first == (w ? std::max(s.n - w, 0) : 0));
        CHECK(s.start % 16 == 0 && s.start <= s.first && s.first - s.start < 16);
        CHECK((int64_t)s.start + (int64_t)s.units * mx::kUnit >= s.n);
        CHECK(s.units == 0 ? s.n == 0 : (int64_t)s.start + (int64_t)(s.units - 1) * mx::kUnit < s.n);
      }
  // shares: all units once, in order, none empty; the owner is the one that has a unit
  for (int i = 0; i < 3000; ++i) {
    const int64_t W = 1 + rng() % 600, U = W + (i % 3 ? rng() % 5000 : rng() % (int64_t(1) << 44));
    CHECK(mx::share(0, U, W) == 0 && mx::share(W, U, W) == U);
    for (int k = 0; k < 20; ++k) {
      const int64_t w = rng() % W, lo = mx::share(w, U, W), hi = mx::share(w + 1, U, W);
      CHECK(lo < hi && mx::owner(lo, U, W) == w && mx::owner(hi - 1, U, W) == w);
      const int64_t u = rng() % U, o = mx::owner(u, U, W);
      CHECK(o >= 0 && o < W && mx::share(o, U, W) <= u && u < mx::share(o + 1, U, W));
    }
  }
}

int main() {
  plan();
  void *p = at(0x10000), *odd = at(0x10001);
  const mxfp4_heads h{p, 4, 512, 64}, none{nullptr, 0, 0, 0};
  mxfp4_rotation r{(const int64_t*)p, (const double*)p, 32, 1, 0, {32, 0, 0, 0}};
  mxfp4_int8_kv c{p, (float*)p, p, (float*)p, 8, 4, 16, 64};
  // a launch for a good call, and its error handed on
  CHECK(mxfp4_qk_norm_rope(&h, &h, 3, 64, 1, &r, p, p, 1, 1e-6f, p, p, nullptr, nullptr) == MXFP4_OK && g_launches == 1);
  CHECK(g_rot.pairs == 32 && g_q_heads == 4);
  CHECK(mxfp4_qk_norm_rope(&h, &none, 3, 64, 1, nullptr, nullptr, nullptr, 1, -1.f, p, nullptr, nullptr, nullptr) == MXFP4_OK);
  CHECK(g_launches == 2 && g_rot.pairs == 0 && g_rot.axes == 1);
  g_result = hipErrorInvalidValue;
  CHECK(mxfp4_qk_norm_rope(&h, &h, 3, 64, 1, &r, p, p, 1, 1e-6f, p, p, nullptr, nullptr) == MXFP4_ERR_HIP);
  CHECK(mxfp4_paged_attention(&h, 2, 64, 1, &c, (int32_t*)p, 4, 4, (int32_t*)p, 1.f, 0, p, nullptr, p, 1024, nullptr) ==
        MXFP4_OK + MXFP4_ERR_HIP);
  g_result = hipSuccess;
  g_launches = 0;
  // strides and sizes at the borders of their range
  for (int64_t bad : {int64_t(-1), int64_t(1) << 62, INT64_MAX, INT64_MIN}) {
    mxfp4_heads x = h;
    x.token_stride = bad;
    CHECK(mxfp4_qk_norm_rope(&x, &h, 3, 64, 1, &r, p, p, 1, 0.f, p, p, nullptr, nullptr) == MXFP4_ERR_SHAPE);
    x = h;
    x.head_stride = bad;
    CHECK(mxfp4_qk_norm_rope(&h, &x, 3, 64, 1, &r, p, p, 1, 0.f, p, p, nullptr, nullptr) == MXFP4_ERR_SHAPE);
    x = h;
    x.heads = bad;
    CHECK(mxfp4_qk_norm_rope(&h, &x, 3, 64, 1, &r, p, p, 1, 0.f, p, p, nullptr, nullptr) == MXFP4_ERR_SHAPE);
    CHECK(mxfp4_qk_norm_rope(&h, &h, bad, 64, 1, &r, p, p, 1, 0.f, p, p, nullptr, nullptr) == MXFP4_ERR_SHAPE);
    CHECK(mxfp4_qk_norm_rope(&h, &h, 3, bad, 1, &r, p, p, 1, 0.f, p, p, nullptr, nullptr) == MXFP4_ERR_SHAPE);
    CHECK(mxfp4_int8_kv_read(&c, (int64_t*)p, bad, 64, 1, p, p, nullptr) == MXFP4_ERR_SHAPE);
    mxfp4_rotation t = r;
    t.pairs = bad;
    CHECK(mxfp4_qk_norm_rope(&h, &h, 3, 64, 1, &t, p, p, 1, 0.f, p, p, nullptr, nullptr) == MXFP4_ERR_SHAPE);
    t = r;
    t.axis_pairs[0] = bad;
    CHECK(mxfp4_qk_norm_rope(&h, &h, 3, 64, 1, &t, p, p, 1, 0.f, p, p, nullptr, nullptr) == MXFP4_ERR_SHAPE);
    mxfp4_int8_kv k = c;
    k.pages = bad;
    CHECK(mxfp4_int8_kv_read(&k, (int64_t*)p, 3, 64, 1, p, p, nullptr) == MXFP4_ERR_SHAPE);
    k = c;
    k.page_size = bad;
    CHECK(mxfp4_int8_kv_read(&k, (int64_t*)p, 3, 64, 1, p, p, nullptr) == MXFP4_ERR_SHAPE);
    k = c;
    k.heads = bad;
    CHECK(mxfp4_int8_kv_read(&k, (int64_t*)p, 3, 64, 1, p, p, nullptr) == MXFP4_ERR_SHAPE);
    k = c;
    k.pitch = bad;
    CHECK(mxfp4_int8_kv_read(&k, (int64_t*)p, 3, 64, 1, p, p, nullptr) == MXFP4_ERR_SHAPE);
    const auto attend = [&](int64_t batch, int64_t ld, int64_t table, int64_t window) {
      return mxfp4_paged_attention(&h, batch, 64, 1, &c, (int32_t*)p, ld, table, (int32_t*)p, 1.f, window, p, nullptr, p,
                                   1 << 20, nullptr);
    };
    CHECK(attend(bad, 4, 4, 0) == MXFP4_ERR_SHAPE && attend(2, bad, 4, 0) == MXFP4_ERR_SHAPE &&
          attend(2, 4, bad, 0) == MXFP4_ERR_SHAPE);
    CHECK(bad > 0 || attend(2, 4, 4, bad) == MXFP4_ERR_SHAPE);
    CHECK(mxfp4_paged_attention_workspace_bytes(bad, 4, 4, 64, 4, 16) == 0);
    CHECK(mxfp4_paged_attention_workspace_bytes(2, bad, 4, 64, 4, 16) == 0);
    CHECK(mxfp4_paged_attention_workspace_bytes(2, 4, bad, 64, 4, 16) == 0);
    CHECK(mxfp4_paged_attention_workspace_bytes(2, 4, 4, bad, 4, 16) == 0);
    CHECK(mxfp4_paged_attention_workspace_bytes(2, 4, 4, 64, bad, 16) == 0);
    CHECK(mxfp4_paged_attention_workspace_bytes(2, 4, 4, 64, 4, bad) == 0);
    CHECK(mxfp4_qk_norm_rope_bwd_workspace_bytes(bad, 4, 4, 64) == 0);
    CHECK(mxfp4_qk_norm_rope_bwd_workspace_bytes(4, 4, 4, bad) == 0);
  }
  CHECK(g_launches == 0);
  // a cache of all the slots there may be, and one more page
  c.pages = ((int64_t(1) << 31) - 1) / 16;
  CHECK(mxfp4_int8_kv_read(&c, (int64_t*)p, 3, 64, 1, p, p, nullptr) == MXFP4_OK && g_launches == 1);
  ++c.pages;
  CHECK(mxfp4_int8_kv_read(&c, (int64_t*)p, 3, 64, 1, p, p, nullptr) == MXFP4_ERR_SHAPE);
  c.pages = 8;
  CHECK(mxfp4_int8_kv_read(&c, (int64_t*)odd, 3, 64, 1, p, p, nullptr) == MXFP4_ERR_ALIGN && g_launches == 1);
  printf("%d checks passed\n", g_checks);
  return 0;
}
