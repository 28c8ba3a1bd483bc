// Int8 matrix product with a scale for each token and each channel on
// gfx950's int8 MFMA (MI355X):
//   C[m][n] = (sum_k A[m][k] B[n][k]) sa[m] sb[n] + bias[n].
// The sum is exact: int32 accumulators, K <= 131071 so that even -128 * -128
// in every place stays below 2^31. It is rounded to fp32 once, then scaled,
// added to and rounded to C's type, so the result does not depend on the
// order of the sum, on the tiling or on how k is split.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "norm_int8.h"

namespace mx {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;

struct Args {
  const uint8_t *A, *B;
  const float *sa, *sb, *bias;
  void* C;
  int64_t lda, ldb, ldc, M, N, K;
};

// The scaled sum; one rounding in each step.
__device__ __forceinline__ float scaled(int acc, float sa, float sb) {
  return (float)acc * sa * sb;
}

template <int OUT>
__device__ __forceinline__ void put(void* C, int64_t i, float v) {
  if constexpr (OUT == kF32) static_cast<float*>(C)[i] = v;
  if constexpr (OUT == kBF16) static_cast<__bf16*>(C)[i] = (__bf16)v;
  if constexpr (OUT == kF16) static_cast<_Float16*>(C)[i] = (_Float16)v;
}

// ------------------------------------------------------ general kernel
// Any sizes, pitches and alignments: 64 x 64 tiles of C, 4 waves of one 32 x
// 32 MFMA tile each, k in steps of 64 staged through LDS. 16 bytes of a row
// are loaded at once where its address allows it, byte by byte where not and
// at the row's end; rows and bytes past the operands are zero.
namespace gen {

constexpr int BM = 64, BN = 64, KB = 64;
constexpr int PITCH = KB + 16;  // 20 words: 8 lanes' 16-byte reads hit distinct banks

__device__ __forceinline__ u32x4 chunk(const uint8_t* p, int64_t row, int64_t rows, int64_t ld,
                                       int64_t k, int64_t K, bool vec) {
  u32x4 q = {0, 0, 0, 0};
  if (row < rows && k < K) {
    const uint8_t* s = p + row * ld + k;
    if (vec && k + 16 <= K) {
      q = *reinterpret_cast<const u32x4*>(s);
    } else {
      const int n = (int)min(K - k, (int64_t)16);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) q[i >> 2] |= (uint32_t)s[i] << (8 * (i & 3));
    }
  }
  return q;
}

template <int OUT>
__global__ __launch_bounds__(256) void gemm_kernel(Args P, bool vec) {
  __shared__ __attribute__((aligned(16))) uint8_t la[BM * PITCH], lb[BN * PITCH];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t ntn = (P.N + BN - 1) / BN;
  const int64_t m0 = blockIdx.x / ntn * BM, n0 = blockIdx.x % ntn * BN;
  const int wm = wave >> 1, wn = wave & 1;
  const int r = t >> 2, c = (t & 3) * 16;  // the thread's chunk of a tile
  const uint8_t* fa = la + (wm * 32 + (lane & 31)) * PITCH + (lane >> 5) * 16;
  const uint8_t* fb = lb + (wn * 32 + (lane & 31)) * PITCH + (lane >> 5) * 16;
  v16i acc = {};
  u32x4 qa = chunk(P.A, m0 + r, P.M, P.lda, c, P.K, vec);
  u32x4 qb = chunk(P.B, n0 + r, P.N, P.ldb, c, P.K, vec);
  for (int64_t k = 0; k < P.K; k += KB) {
    *reinterpret_cast<u32x4*>(la + r * PITCH + c) = qa;
    *reinterpret_cast<u32x4*>(lb + r * PITCH + c) = qb;
    __syncthreads();
    qa = chunk(P.A, m0 + r, P.M, P.lda, k + KB + c, P.K, vec);
    qb = chunk(P.B, n0 + r, P.N, P.ldb, k + KB + c, P.K, vec);
#pragma unroll
    for (int s = 0; s < KB / 32; ++s)
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(*reinterpret_cast<const v4i*>(fa + 32 * s),
                                                  *reinterpret_cast<const v4i*>(fb + 32 * s), acc,
                                                  0, 0, 0);
    __syncthreads();
  }
  // register e of a lane is row 8 (e / 4) + 4 (lane / 32) + e % 4, column lane % 32
  const int64_t n = n0 + wn * 32 + (lane & 31);
  if (n >= P.N) return;
  const float sb = P.sb[n], bias = P.bias ? P.bias[n] : 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int64_t m = m0 + wm * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
    if (m < P.M) put<OUT>(P.C, m * P.ldc + n, scaled(acc[e], P.sa[m], sb) + bias);
  }
}

template <int OUT>
hipError_t launch(const Args& P, hipStream_t st) {
  const bool vec = (((uintptr_t)P.A | (uintptr_t)P.B) & 15) == 0 && ((P.lda | P.ldb) & 15) == 0;
  const int64_t tiles = ((P.M + BM - 1) / BM) * ((P.N + BN - 1) / BN);
  hipLaunchKernelGGL((gemm_kernel<OUT>), dim3((unsigned)tiles), dim3(256), 0, st, P, vec);
  return hipGetLastError();
}

}  // namespace gen

template <int OUT>
hipError_t launch_out(const Args& P, void* ws, hipStream_t st) {
  return gen::launch<OUT>(P, st);
}

}  // namespace

size_t int8_gemm_ws(int64_t M, int64_t N, int64_t K) { return 0; }

hipError_t launch_int8_gemm(CMat A, const float* sa, CMat B, const float* sb, const float* bias,
                            int64_t M, int64_t N, int64_t K, Mat C, int out_dtype, void* ws,
                            hipStream_t stream) {
  const Args P{static_cast<const uint8_t*>(A.p), static_cast<const uint8_t*>(B.p), sa, sb, bias,
               C.p, A.ld, B.ld, C.ld, M, N, K};
  switch (out_dtype) {
    case kBF16: return launch_out<kBF16>(P, ws, stream);
    case kF16: return launch_out<kF16>(P, ws, stream);
    default: return launch_out<kF32>(P, ws, stream);
  }
}

}  // namespace mx
