// Launch interface of the norm and 8-bit operators between their host API
// (api_int8.cpp) and their gfx950 kernels (norm.hip, int8_gemm.hip).
// Arguments are validated by the caller.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace mx {

// A matrix with a row pitch in elements.
struct Mat {
  void* p;
  int64_t ld;
};
struct CMat {
  const void* p;
  int64_t ld;
};

// Widest row of the norm and of the int8 quantizers: 1024 threads of 32
// values (norm.hip).
constexpr int64_t kRowMax = 32768;

// RMS norm of h = x + res (res.p may be NULL), y in the inputs' type; h.p and
// rstd may be NULL (not written); weight NULL is 1.
hipError_t launch_rmsnorm(CMat x, CMat res, const void* weight, int weight_dtype, int64_t rows,
                          int64_t cols, float eps, int dtype, Mat h, Mat y, float* rstd,
                          hipStream_t stream);
// The same with y as int8 codes and a scale a row.
hipError_t launch_rmsnorm_int8(CMat x, CMat res, const void* weight, int weight_dtype,
                               int64_t rows, int64_t cols, float eps, int dtype, Mat h, Mat q,
                               float* scales, hipStream_t stream);
// Gradients: dx (of x and of res alike), and dweight unless it is NULL
// (partial sums in ws, rmsnorm_bwd_ws bytes).
hipError_t launch_rmsnorm_bwd(CMat dy, CMat dh, CMat h, const void* weight, int weight_dtype,
                              const float* rstd, int64_t rows, int64_t cols, int dtype, Mat dx,
                              void* dweight, void* ws, hipStream_t stream);
size_t rmsnorm_bwd_ws(int64_t rows, int64_t cols);

// Int8 codes and a scale a row of x, or of silu(gate) x where gate.p is set.
hipError_t launch_int8_quantize(CMat x, CMat gate, int64_t rows, int64_t cols, int dtype, Mat q,
                                float* scales, hipStream_t stream);

// C[m][n] = (sum_k A[m][k] B[n][k]) sa[m] sb[n] + bias[n]; bias may be NULL.
hipError_t launch_int8_gemm(CMat A, const float* sa, CMat B, const float* sb, const float* bias,
                            int64_t M, int64_t N, int64_t K, Mat C, int out_dtype, void* ws,
                            hipStream_t stream);
// Bytes of partial sums that launch_int8_gemm writes for these sizes.
size_t int8_gemm_ws(int64_t M, int64_t N, int64_t K);

}  // namespace mx
