// Host-only check of the C ABI of the norm and 8-bit operators (api_int8.cpp),
// built with the address and undefined-behaviour sanitizers against stand-ins
// for their launch layer: refusals at the limits of sizes, pitches and
// alignments return the documented status before any launch, valid calls at
// the limits hand their arguments on, and a failed launch maps to
// MXFP4_ERR_HIP. Exit status 0 when every case holds; the first failing case
// is printed.
#include <stdio.h>
#include <stdlib.h>

#include "../../include/mxfp4.h"
#include "../../mxfp4_quantized_gemm_amd/csrc/norm_int8.h"

namespace {
int g_cases = 0;
int g_launches = 0;
hipError_t g_result = hipSuccess;
int64_t g_rows, g_cols, g_k;
size_t g_ws = 0;  // what int8_gemm_ws answers

hipError_t launched(int64_t rows, int64_t cols, int64_t k = 0) {
  ++g_launches;
  g_rows = rows;
  g_cols = cols;
  g_k = k;
  return g_result;
}
}  // namespace

namespace mx {
hipError_t launch_rmsnorm(CMat, CMat, const void*, int, int64_t rows, int64_t cols, float, int, Mat, Mat, float*,
                          hipStream_t) {
  return launched(rows, cols);
}
hipError_t launch_rmsnorm_int8(CMat, CMat, const void*, int, int64_t rows, int64_t cols, float, int, Mat, Mat, float*,
                               hipStream_t) {
  return launched(rows, cols);
}
hipError_t launch_rmsnorm_bwd(CMat, CMat, CMat, const void*, int, const float*, int64_t rows, int64_t cols, int, Mat,
                              void*, void*, hipStream_t) {
  return launched(rows, cols);
}
size_t rmsnorm_bwd_ws(int64_t, int64_t cols) { return (size_t)cols * 4; }
hipError_t launch_int8_quantize(CMat, CMat, int64_t rows, int64_t cols, int, Mat, float*, hipStream_t) {
  return launched(rows, cols);
}
hipError_t launch_int8_gemm(CMat, const float*, CMat, const float*, const float*, int64_t M, int64_t N, int64_t K, Mat,
                            int, void*, hipStream_t) {
  return launched(M, N, K);
}
size_t int8_gemm_ws(int64_t, int64_t, int64_t) { return g_ws; }
}  // namespace mx

#define CHECK(cond)                                                               \
  do {                                                                            \
    ++g_cases;                                                                    \
    if (!(cond)) {                                                                \
      fprintf(stderr, "int8_check: %s:%d: failed: %s\n", __FILE__, __LINE__, #cond); \
      exit(1);                                                                    \
    }                                                                             \
  } while (0)
// Refused with `st`, and nothing launched.
#define REFUSED(st, call)            \
  do {                               \
    const int before = g_launches;   \
    CHECK((call) == (st));           \
    CHECK(g_launches == before);     \
  } while (0)
// Taken, and launched once with these sizes.
#define TAKEN(call, r, c)                                                      \
  do {                                                                         \
    const int before = g_launches;                                             \
    CHECK((call) == MXFP4_OK);                                                 \
    CHECK(g_launches == before + 1 && g_rows == (int64_t)(r) && g_cols == (int64_t)(c)); \
  } while (0)

namespace {

constexpr int64_t kBig[] = {INT64_MIN, INT64_MIN + 1, -1, INT64_MAX, INT64_MAX - 1, int64_t(1) << 62, int64_t(1) << 48};

// Stand-in device addresses: never dereferenced.
alignas(256) unsigned char g_mem[4096];
void* at(size_t off) { return g_mem + off; }
float* floats(size_t off) { return static_cast<float*>(at(off)); }

struct Norm {
  const void* x = at(0);
  int64_t x_ld = 64;
  const void* res = at(0);
  int64_t res_ld = 64;
  const void* w = at(0);
  int wt = 1;
  int64_t rows = 4, cols = 64;
  int dt = 1;
  void* h = at(0);
  int64_t h_ld = 64;
  void* out = at(0);
  int64_t out_ld = 64;
  float* stat = floats(0);
  int norm() const {
    return mxfp4_rmsnorm(x, x_ld, res, res_ld, w, wt, rows, cols, 1e-5f, dt, h, h_ld, out, out_ld, stat, nullptr);
  }
  int codes() const {
    return mxfp4_rmsnorm_int8(x, x_ld, res, res_ld, w, wt, rows, cols, 1e-5f, dt, h, h_ld, out, out_ld, stat, nullptr);
  }
  int quantize() const { return mxfp4_int8_quantize(x, x_ld, res, res_ld, rows, cols, dt, out, out_ld, stat, nullptr); }
  void pitch(int64_t ld) { x_ld = res_ld = h_ld = out_ld = ld; }
};

template <class Call>
void row_cases(Call call, bool norm) {
  for (int64_t v : kBig) {
    Norm a;
    a.rows = v;
    REFUSED(MXFP4_ERR_SHAPE, call(a));
    a = Norm();
    a.cols = v;
    REFUSED(MXFP4_ERR_SHAPE, call(a));
    for (int64_t Norm::* ld : {&Norm::x_ld, &Norm::res_ld, &Norm::out_ld}) {
      a = Norm();
      a.*ld = v;
      REFUSED(MXFP4_ERR_SHAPE, call(a));
    }
    a = Norm();
    a.dt = (int)v;
    if (a.dt < 0 || a.dt > 2) REFUSED(MXFP4_ERR_MODE, call(a));
  }
  Norm a;
  a.cols = 32768;
  a.pitch(32768);
  TAKEN(call(a), 4, 32768);
  a.cols = 32769;
  a.pitch(32769);
  REFUSED(MXFP4_ERR_SHAPE, call(a));
  a = Norm();
  a.rows = (int64_t(1) << 31) - 1;
  TAKEN(call(a), a.rows, 64);
  a.rows += 1;
  REFUSED(MXFP4_ERR_SHAPE, call(a));
  // the largest pitch of two rows, and one past it
  a = Norm();
  a.rows = 2;
  a.pitch(int64_t(1) << 47);
  TAKEN(call(a), 2, 64);
  a.x_ld += 1;
  REFUSED(MXFP4_ERR_SHAPE, call(a));
  // 2^40 elements, and one row more
  a = Norm();
  a.cols = 32768;
  a.rows = int64_t(1) << 25;
  a.pitch(32768);
  CHECK(call(a) == (a.rows <= (int64_t(1) << 40) / a.cols ? MXFP4_OK : MXFP4_ERR_SHAPE));
  a.rows += 1;
  REFUSED(MXFP4_ERR_SHAPE, call(a));
  // nothing to do: no pointer is looked at
  a = Norm();
  a.rows = 0;
  a.x = a.res = a.w = nullptr;
  a.h = a.out = nullptr;
  a.stat = nullptr;
  REFUSED(MXFP4_OK, call(a));
  for (size_t off = 1; off < 4; ++off) {
    a = Norm();
    a.dt = a.wt = 0;
    a.x = at(off);
    REFUSED(MXFP4_ERR_ALIGN, call(a));
    a = Norm();
    a.stat = reinterpret_cast<float*>(at(off));
    REFUSED(MXFP4_ERR_ALIGN, call(a));
  }
  if (norm) {
    a = Norm();
    a.wt = 2;
    REFUSED(MXFP4_ERR_MODE, call(a));
    a = Norm();
    a.h_ld = 63;
    REFUSED(MXFP4_ERR_SHAPE, call(a));
    a.h = nullptr;  // then its pitch is not looked at
    TAKEN(call(a), 4, 64);
  }
  g_result = hipErrorInvalidValue;
  CHECK(call(Norm()) == MXFP4_ERR_HIP);
  g_result = hipSuccess;
}

void gradient_cases() {
  const size_t need = mxfp4_rmsnorm_bwd_workspace_bytes(4, 64);
  CHECK(need == 256);
  for (int64_t v : kBig) {
    CHECK(mxfp4_rmsnorm_bwd_workspace_bytes(v, 64) == 0);
    CHECK(mxfp4_rmsnorm_bwd_workspace_bytes(4, v) == 0);
  }
  struct Args {
    int64_t rows = 4, cols = 64, ld = 64;
    void* dw = at(0);
    void* ws = at(0);
    size_t bytes = 256;
    int operator()() const {
      return mxfp4_rmsnorm_bwd(at(0), ld, at(0), ld, at(0), ld, at(0), 1, floats(0), rows, cols, 1, at(0), ld, dw, ws,
                               bytes, nullptr);
    }
  } a;
  TAKEN(a(), 4, 64);
  for (int64_t v : kBig) {
    Args b;
    b.rows = v;
    REFUSED(MXFP4_ERR_SHAPE, b());
    b = Args();
    b.cols = v;
    REFUSED(MXFP4_ERR_SHAPE, b());
    b = Args();
    b.ld = v;
    REFUSED(MXFP4_ERR_SHAPE, b());
  }
  a.bytes = 255;
  REFUSED(MXFP4_ERR_WORKSPACE, a());
  a.ws = nullptr;
  REFUSED(MXFP4_ERR_NULL, a());
  a.dw = nullptr;  // not wanted: no workspace
  TAKEN(a(), 4, 64);
  a.rows = 0;
  REFUSED(MXFP4_OK, a());
  a.dw = at(0);  // set to zero by a launch
  TAKEN(a(), 0, 64);
}

void product_cases() {
  struct Args {
    int64_t M = 4, N = 8, K = 64, lda = 64, ldb = 64, ldc = 8;
    int dt = 1;
    void* ws = nullptr;
    size_t bytes = 0;
    int operator()() const {
      return mxfp4_int8_gemm(at(0), lda, floats(0), at(0), ldb, floats(0), nullptr, M, N, K, at(0), ldc, dt, ws, bytes,
                             nullptr);
    }
  } a;
  TAKEN(a(), 4, 8);
  for (int64_t v : kBig) {
    for (int64_t Args::* f : {&Args::M, &Args::N, &Args::K, &Args::lda, &Args::ldb, &Args::ldc}) {
      Args b;
      b.*f = v;
      REFUSED(MXFP4_ERR_SHAPE, b());
    }
    CHECK(mxfp4_int8_gemm_workspace_bytes(v, 8, 64) == 0);
    CHECK(mxfp4_int8_gemm_workspace_bytes(4, v, 64) == 0);
    CHECK(mxfp4_int8_gemm_workspace_bytes(4, 8, v) == 0);
  }
  // the longest sum, the most rows, the most tiles
  a.K = a.lda = a.ldb = 131071;
  TAKEN(a(), 4, 8);
  CHECK(g_k == 131071);
  a.K = a.lda = a.ldb = 131072;
  REFUSED(MXFP4_ERR_SHAPE, a());
  a = Args();
  a.M = (int64_t(1) << 26) - 1;
  TAKEN(a(), a.M, 8);
  a.M += 1;
  REFUSED(MXFP4_ERR_SHAPE, a());
  a = Args();
  a.M = 64 * 4096;
  a.N = a.ldc = 64 * 2047;
  TAKEN(a(), a.M, a.N);
  a.N = a.ldc = 64 * 2048;
  REFUSED(MXFP4_ERR_SHAPE, a());
  // empty products
  for (int64_t Args::* f : {&Args::M, &Args::N}) {
    a = Args();
    a.*f = 0;
    REFUSED(MXFP4_OK, a());
    CHECK(mxfp4_int8_gemm_workspace_bytes(a.M, a.N, 64) == 0);
  }
  // a workspace that is asked for
  g_ws = 4096;
  CHECK(mxfp4_int8_gemm_workspace_bytes(4, 8, 64) == 4096);
  a = Args();
  REFUSED(MXFP4_ERR_NULL, a());
  a.ws = at(0);
  a.bytes = 4095;
  REFUSED(MXFP4_ERR_WORKSPACE, a());
  a.bytes = 4096;
  TAKEN(a(), 4, 8);
  for (size_t off : {1, 4, 8}) {
    a.ws = at(off);
    REFUSED(MXFP4_ERR_ALIGN, a());
  }
  g_ws = 0;
  g_result = hipErrorInvalidValue;
  CHECK(Args()() == MXFP4_ERR_HIP);
  g_result = hipSuccess;
}

}  // namespace

int main() {
  row_cases([](const Norm& a) { return a.norm(); }, true);
  row_cases([](const Norm& a) { return a.codes(); }, true);
  row_cases([](const Norm& a) { return a.quantize(); }, false);
  gradient_cases();
  product_cases();
  printf("%d checks passed\n", g_cases);
  return 0;
}
