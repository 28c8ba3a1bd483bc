// C ABI of the norm and 8-bit operators: argument validation (host only,
// before any HIP call), as api.cpp does for the MXFP4 entry points.
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/mxfp4.h"
#include "norm_int8.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxK = 131071;               // 2^14 K < 2^31: the int32 sums stay exact
constexpr int64_t kMaxDim = int64_t(1) << 26;   // a product's rows of A and of B, and
constexpr int64_t kMaxTiles = int64_t(1) << 23; // its 64 x 64 tiles: grids stay below 2^32 threads

bool valid_dtype(int t) { return t >= MXFP4_DT_F32 && t <= MXFP4_DT_F16; }
int size_of(int t) { return t == MXFP4_DT_F32 ? 4 : 2; }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ERR_HIP; }

// A row operator's sizes: up to 2^31 - 1 rows of 1 to mx::kRowMax columns.
bool rows_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows < kMaxRows && cols >= 1 && cols <= mx::kRowMax && rows <= kMaxElems / cols;
}

// A pitch: at least the columns, and such that the last row's offset fits.
bool pitch_ok(int64_t ld, int64_t rows, int64_t cols) {
  return ld >= cols && ld <= (int64_t(1) << 48) / (rows > 0 ? rows : 1);
}

// The norm's arguments that its two forms share.
int check_norm(const void* x, int64_t x_ld, const void* res, int64_t res_ld, const void* weight,
               int weight_dtype, int64_t rows, int64_t cols, int dtype, const void* h,
               int64_t h_ld, const void* out, int64_t out_ld, int out_size) {
  if (!valid_dtype(dtype) || (weight_dtype != dtype && weight_dtype != MXFP4_DT_F32))
    return MXFP4_ERR_MODE;
  if (!rows_ok(rows, cols) || !pitch_ok(x_ld, rows, cols) || !pitch_ok(out_ld, rows, cols) ||
      (res && !pitch_ok(res_ld, rows, cols)) || (h && !pitch_ok(h_ld, rows, cols)))
    return MXFP4_ERR_SHAPE;
  if (rows == 0) return MXFP4_OK;
  if (!x || !out) return MXFP4_ERR_NULL;
  const int s = size_of(dtype);
  if (!aligned(x, s) || !aligned(res, s) || !aligned(h, s) || !aligned(weight, size_of(weight_dtype)) ||
      !aligned(out, out_size))
    return MXFP4_ERR_ALIGN;
  return MXFP4_OK;
}

}  // namespace

extern "C" {

int mxfp4_rmsnorm(const void* x, int64_t x_ld, const void* residual, int64_t residual_ld,
                  const void* weight, int weight_dtype, int64_t rows, int64_t cols, float eps,
                  int dtype, void* h, int64_t h_ld, void* y, int64_t y_ld, float* rstd,
                  hipStream_t stream) {
  const int st = check_norm(x, x_ld, residual, residual_ld, weight, weight_dtype, rows, cols,
                            dtype, h, h_ld, y, y_ld, valid_dtype(dtype) ? size_of(dtype) : 4);
  if (st != MXFP4_OK || rows == 0) return st;
  if (!aligned(rstd, 4)) return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_rmsnorm({x, x_ld}, {residual, residual_ld}, weight, weight_dtype,
                                       rows, cols, eps, dtype, {h, h_ld}, {y, y_ld}, rstd,
                                       stream));
}

int mxfp4_rmsnorm_int8(const void* x, int64_t x_ld, const void* residual, int64_t residual_ld,
                       const void* weight, int weight_dtype, int64_t rows, int64_t cols,
                       float eps, int dtype, void* h, int64_t h_ld, void* codes,
                       int64_t codes_ld, float* scales, hipStream_t stream) {
  const int st = check_norm(x, x_ld, residual, residual_ld, weight, weight_dtype, rows, cols,
                            dtype, h, h_ld, codes, codes_ld, 1);
  if (st != MXFP4_OK || rows == 0) return st;
  if (!scales) return MXFP4_ERR_NULL;
  if (!aligned(scales, 4)) return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_rmsnorm_int8({x, x_ld}, {residual, residual_ld}, weight,
                                            weight_dtype, rows, cols, eps, dtype, {h, h_ld},
                                            {codes, codes_ld}, scales, stream));
}

size_t mxfp4_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  return rows_ok(rows, cols) ? mx::rmsnorm_bwd_ws(rows, cols) : 0;
}

int mxfp4_rmsnorm_bwd(const void* dy, int64_t dy_ld, const void* dh, int64_t dh_ld, const void* h,
                      int64_t h_ld, const void* weight, int weight_dtype, const float* rstd,
                      int64_t rows, int64_t cols, int dtype, void* dx, int64_t dx_ld,
                      void* dweight, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!valid_dtype(dtype) || (weight_dtype != dtype && weight_dtype != MXFP4_DT_F32))
    return MXFP4_ERR_MODE;
  if (!rows_ok(rows, cols) || !pitch_ok(dy_ld, rows, cols) || (dh && !pitch_ok(dh_ld, rows, cols)) ||
      !pitch_ok(h_ld, rows, cols) || !pitch_ok(dx_ld, rows, cols))
    return MXFP4_ERR_SHAPE;
  if (rows == 0 && !dweight) return MXFP4_OK;
  if (rows > 0) {
    if (!dy || !h || !rstd || !dx || (dweight && !ws)) return MXFP4_ERR_NULL;
    if (dweight && ws_bytes < mx::rmsnorm_bwd_ws(rows, cols)) return MXFP4_ERR_WORKSPACE;
  }
  const int s = size_of(dtype), w = size_of(weight_dtype);
  if (!aligned(dy, s) || !aligned(dh, s) || !aligned(h, s) || !aligned(dx, s) || !aligned(rstd, 4) ||
      !aligned(weight, w) || !aligned(dweight, w) || !aligned(ws, 4))
    return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_rmsnorm_bwd({dy, dy_ld}, {dh, dh_ld}, {h, h_ld}, weight,
                                           weight_dtype, rstd, rows, cols, dtype, {dx, dx_ld},
                                           dweight, ws, stream));
}

int mxfp4_int8_quantize(const void* x, int64_t x_ld, const void* gate, int64_t gate_ld,
                        int64_t rows, int64_t cols, int dtype, void* codes, int64_t codes_ld,
                        float* scales, hipStream_t stream) {
  if (!valid_dtype(dtype)) return MXFP4_ERR_MODE;
  if (!rows_ok(rows, cols) || !pitch_ok(x_ld, rows, cols) || !pitch_ok(codes_ld, rows, cols) ||
      (gate && !pitch_ok(gate_ld, rows, cols)))
    return MXFP4_ERR_SHAPE;
  if (rows == 0) return MXFP4_OK;
  if (!x || !codes || !scales) return MXFP4_ERR_NULL;
  const int s = size_of(dtype);
  if (!aligned(x, s) || !aligned(gate, s) || !aligned(scales, 4)) return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_int8_quantize({x, x_ld}, {gate, gate_ld}, rows, cols, dtype,
                                             {codes, codes_ld}, scales, stream));
}

static bool gemm_sizes_ok(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 1 || K > kMaxK || M >= kMaxDim || N >= kMaxDim) return false;
  const int64_t tm = (M + 63) / 64, tn = (N + 63) / 64;
  return tn == 0 || tm < kMaxTiles / tn;
}

size_t mxfp4_int8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return gemm_sizes_ok(M, N, K) && M > 0 && N > 0 ? mx::int8_gemm_ws(M, N, K) : 0;
}

int mxfp4_int8_gemm(const void* A, int64_t lda, const float* a_scales, const void* B, int64_t ldb,
                    const float* b_scales, const float* bias, int64_t M, int64_t N, int64_t K,
                    void* C, int64_t ldc, int out_dtype, void* ws, size_t ws_bytes,
                    hipStream_t stream) {
  if (!valid_dtype(out_dtype)) return MXFP4_ERR_MODE;
  if (!gemm_sizes_ok(M, N, K) || !pitch_ok(lda, M, K) || !pitch_ok(ldb, N, K) || !pitch_ok(ldc, M, N))
    return MXFP4_ERR_SHAPE;
  if (M == 0 || N == 0) return MXFP4_OK;
  const size_t need = mx::int8_gemm_ws(M, N, K);
  if (!A || !a_scales || !B || !b_scales || !C || (need && !ws)) return MXFP4_ERR_NULL;
  if (ws_bytes < need) return MXFP4_ERR_WORKSPACE;
  if (!aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(bias, 4) ||
      !aligned(C, size_of(out_dtype)) || (need && !aligned(ws, 16)))
    return MXFP4_ERR_ALIGN;
  return hip_status(mx::launch_int8_gemm({A, lda}, a_scales, {B, ldb}, b_scales, bias, M, N, K,
                                         {C, ldc}, out_dtype, ws, stream));
}

}  // extern "C"
