// RMS norm with the residual's addition, its gradient, and the int8 row
// quantizers for gfx950 (MI355X).
//
//   h = round_T(x + res)                   the residual stream, held in its type T
//   r = 1 / sqrt(mean(h^2) + eps)          one factor a row
//   y = (h r) w
//   codes: a = max |v| of the row's values v (y; x; or silu(gate) x),
//          scale = a / 127, q = rint(v (127 / a)); a = 0: scale 0, codes 0;
//          a row that holds a NaN or an infinity: scale NaN, codes 0
//   gradient of (y, h): with g = dy w and u = h r,
//          dx = dres = r (g - u mean(g u)) + dh,  dw = sum over rows of dy u
//
// Each is one pass over HBM: a row's values stay in registers between its
// sums and its output. Precision: products and factors in fp32; the sum of
// squares in fp64, because h^2 leaves fp32's range for |h| above 2^64, and so
// that r is the same fp32 number whatever the order of the sum (but for a row
// in about 10^8 whose factor lies within 2^-50 of a rounding border); the int8
// codes can then be checked bit for bit against a plain implementation. The
// gradient's sums are in fp32: a row's in at most 32 steps a thread, a weight's
// over a work-group's rows and then over the work-groups.
//
// HBM bounds all of them (8192 x 4096 bf16): norm 43 us for 268 MB (6.2 TB/s;
// torch's copy on the same card 5.1), norm to codes 40, codes of x 18, gated
// codes 26, gradient 47.5 and 4 for the weight's second pass.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "norm_int8.h"
#include "rows.h"

namespace mx {
namespace {

// silu(g) u = g u / (1 + exp(-g)), by the hardware's base-2 exponential and
// reciprocal (each within about one ulp; the rounded argument g log2(e) adds
// at most |g| 2^-24 to the relative error): far below half a step of a code.
// Past t = -g log2(e) = kFar the exponential and the reciprocal leave fp32's
// range, though g u 2^-t need not (any u): there 1 / (1 + 2^t) is 2^-kFar h h
// with h = 2^((kFar - t) / 2), and the factors are taken in an order in which
// none leaves the range before the result does (kFar - t is exact). 512 x 14336
// bf16: 7.4 us with this branch and 7.6 without; 9.6 where all waves take it.
constexpr float kFar = 120.f;
__device__ __forceinline__ float exponent(float g) { return g * -1.44269504f; }
__device__ __forceinline__ float swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(exponent(g))) * u;
}
__device__ __forceinline__ float swiglu_far(float g, float u) {
  const float h = __builtin_amdgcn_exp2f(0.5f * (kFar - exponent(g)));
  return g * 0x1p-120f * (h * u) * h;
}

constexpr int kNorm = 0, kNormInt8 = 1, kQuant = 2, kSwiglu = 3;

struct RowArgs {
  const void *x, *res, *w;  // res: the residual (norm) or the gate (swiglu)
  void *h, *out;
  float* stat;  // rstd (norm, may be NULL) or scales
  int64_t x_ld, res_ld, h_ld, out_ld, rows;
  double inv_cols;  // 1 / cols
  int cols;
  float eps;
  bool wide;  // fp32 weight beside 16-bit inputs
};

template <int T, bool EVEN, int TPR, int R, int OP>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void row_kernel(RowArgs A) {
  constexpr int V = 16 / Type<T>::S;
  constexpr int NW = TPR < 256 ? 4 : TPR / 64;
  __shared__ double red64[NW];
  __shared__ uint32_t red32[NW];
  // below 256 threads a row, a work-group takes 256 / TPR rows
  const int t = TPR < 256 ? threadIdx.x % TPR : threadIdx.x;
  const int64_t group = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t row = TPR < 256 ? group * (256 / TPR) + threadIdx.x / TPR : group;
  if (row >= A.rows) return;  // no barrier follows below 256 threads a row; else whole work-groups
  typedef Row<T, EVEN, TPR, R> X;
  float v[R][V];
  X::load(A.x, row * A.x_ld, A.cols, t, v);
  if constexpr (OP == kSwiglu) {
    float g[R][V];
    X::load(A.res, row * A.res_ld, A.cols, t, g);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float far = 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k) far = fmaxf(far, exponent(g[i][k]));
      if (far <= kFar) {
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] = swiglu(g[i][k], v[i][k]);
      } else {  // a gate below -83: hardly ever
#pragma unroll
        for (int k = 0; k < V; ++k)
          v[i][k] = exponent(g[i][k]) > kFar ? swiglu_far(g[i][k], v[i][k]) : swiglu(g[i][k], v[i][k]);
      }
    }
  }
  if constexpr (OP == kNorm || OP == kNormInt8) {
    if (A.res != nullptr) {
      float b[R][V];
      X::load(A.res, row * A.res_ld, A.cols, t, b);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] = round_to<T>(v[i][k] + b[i][k]);
    }
    if (A.h != nullptr) X::store(A.h, row * A.h_ld, A.cols, t, v);
    float w[R][V];
    load_weight<T, EVEN, TPR, R>(A.w, A.wide, A.cols, t, w);
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) s = fma((double)v[i][k], (double)v[i][k], s);
    s = reduce_row<TPR>(s, red64, t, add64);
    const float r = (float)rsqrt64(fma(s, A.inv_cols, (double)A.eps));
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) v[i][k] = v[i][k] * r * w[i][k];
    if constexpr (OP == kNorm) {
      if (A.stat != nullptr && t == 0) A.stat[row] = r;
      X::store(A.out, row * A.out_ld, A.cols, t, v);
    }
  }
  if constexpr (OP != kNorm)
    write_codes<T, EVEN, TPR, R>(v, red32, static_cast<uint8_t*>(A.out) + row * A.out_ld, A.out_ld,
                           A.stat + row, A.cols, t);
}

// ------------------------------------------------------------- gradient
struct BwdArgs {
  const void *dy, *dh, *h, *w;
  const float* rstd;
  void* dx;
  float* part;  // [gridDim.x][cols] partial sums of dw, or NULL
  int64_t dy_ld, dh_ld, h_ld, dx_ld, rows;
  int cols;
  bool wide;
};

// Work-groups walk the rows in turn (up to a wave a row, several rows at a time):
// the weight's gradient is summed over a work-group's rows in registers, and
// the work-groups' partial sums by a second kernel, in a fixed order (no
// atomics). One work-group's partial sums cost as much traffic as two rows in
// 16 bits, so there are no more of them than keep the loads going: 8192 x 4096
// bf16 took 62.2 us with 1024 work-groups of 256 threads and 58.2 with 512,
// 4096 x 16384 146 with 1024 of 1024 threads and 112 with 256.
template <int T, bool EVEN, int TPR, int R>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void bwd_kernel(BwdArgs A) {
  constexpr int V = 16 / Type<T>::S;
  constexpr int RPG = TPR < 256 ? 256 / TPR : 1;  // rows at a time
  __shared__ float red[2][TPR < 64 ? 1 : TPR / 64];
  __shared__ float meet[RPG > 1 ? RPG * TPR * R * V : 1];
  // 32 values a thread (or 16 and the shifts of an odd width) at 1024 threads
  // leave no registers for the weight and its gradient, nor for dh in flight
  // during the sum: the weight and dh are then loaded where they are used, and
  // the gradient is summed in LDS (1024 x 30000 bf16: 92 us, 182 with spills)
  constexpr bool KEEP = R * V <= 16 && (EVEN || TPR < 1024);
  __shared__ float own[KEEP ? 1 : TPR * R * V];
  const int t = threadIdx.x % TPR, part = threadIdx.x / TPR;
  typedef Row<T, EVEN, TPR, R> X;
  float w[R][V], dw[R][V];
  if constexpr (KEEP) load_weight<T, EVEN, TPR, R>(A.w, A.wide, A.cols, t, w);
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if constexpr (KEEP)
        dw[i][k] = 0.f;
      else
        own[(i * V + k) * TPR + t] = 0.f;  // a thread touches its own slots only
    }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPG + part; row < A.rows;
       row += (int64_t)gridDim.x * RPG, turn ^= 1) {
    float g[R][V], u[R][V], d[R][V];
    X::load(A.dy, row * A.dy_ld, A.cols, t, g);
    X::load(A.h, row * A.h_ld, A.cols, t, u);
    if constexpr (!KEEP) {
      const void* p = A.w;
      asm volatile("" : "+s"(p));  // else the compiler hoists the loads, and spills
      load_weight<T, EVEN, TPR, R>(p, A.wide, A.cols, t, w);
    }
    const float r = A.rstd[row];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        u[i][k] *= r;
        if constexpr (KEEP) {
          dw[i][k] = fmaf(g[i][k], u[i][k], dw[i][k]);
        } else {
          float& a = own[(i * V + k) * TPR + t];
          a = fmaf(g[i][k], u[i][k], a);
        }
        g[i][k] *= w[i][k];
        s = fmaf(g[i][k], u[i][k], s);
      }
    const auto load_dh = [&]() {
      if (A.dh != nullptr) {
        X::load(A.dh, row * A.dh_ld, A.cols, t, d);
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) d[i][k] = 0.f;
      }
    };
    if constexpr (KEEP) load_dh();
    // two sets of slots: a row's slots are written again two rows later,
    // after the barrier of the row between
    s = reduce_row<TPR>(s, red[turn], t, add32) / (float)A.cols;
    if constexpr (!KEEP) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) g[i][k] = r * (g[i][k] - u[i][k] * s);
      load_dh();
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) d[i][k] += g[i][k];
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) d[i][k] = fmaf(r, g[i][k] - u[i][k] * s, d[i][k]);
    }
    X::store(A.dx, row * A.dx_ld, A.cols, t, d);
  }
  if (A.part == nullptr) return;
  if constexpr (RPG > 1) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) meet[part * TPR * R * V + (t + TPR * i) * V + k] = dw[i][k];
    __syncthreads();
    for (int c = threadIdx.x; c < A.cols; c += 256) {
      float v = meet[c];
#pragma unroll
      for (int q = 1; q < RPG; ++q) v += meet[q * TPR * R * V + c];
      A.part[(int64_t)blockIdx.x * A.cols + c] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = (t + TPR * i) * V + k;
        if (c < A.cols)
          A.part[(int64_t)blockIdx.x * A.cols + c] = KEEP ? dw[i][k] : own[KEEP ? 0 : (i * V + k) * TPR + t];
      }
  }
}

// dw[c] = sum over the parts p of part[p][c]: 32 half-waves of a work-group
// take every 32nd part of 32 columns, then their sums meet in order.
template <int T>
__global__ __launch_bounds__(1024) void dw_kernel(const float* part, int parts, int cols, void* dw) {
  __shared__ float red[32][32];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 16
    for (int p = q; p < parts; p += 32) s += part[(int64_t)p * cols + c];
  }
  red[q][lane] = s;
  __syncthreads();
  if (q == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 32; ++k) s += red[k][lane];
    put1<T>(dw, c, s);
  }
}

// A grid dimension holds below 2^32 threads: many rows go into two dimensions.
constexpr int64_t kGridX = int64_t(1) << 20;

template <int T, bool EVEN, int TPR, int E, int OP>
hipError_t go(const RowArgs& A, hipStream_t st) {
  constexpr int per = TPR < 256 ? 256 / TPR : 1;
  const int64_t groups = (A.rows + per - 1) / per, gx = groups < kGridX ? groups : kGridX;
  const dim3 grid((unsigned)gx, (unsigned)((groups + gx - 1) / gx)), blk(TPR < 256 ? 256 : TPR);
  hipLaunchKernelGGL((row_kernel<T, EVEN, TPR, E * Type<T>::S / 16, OP>), grid, blk, 0, st, A);
  return hipGetLastError();
}

// Threads a row and values a thread: a quarter of a wave up to 128 columns
// (the width of an attention head: 65536 x 128 bf16 took 26.6 us with a wave a
// row), one wave up to 1024, 4 waves up to 8192, 16 waves up to kRowMax.
template <int T, bool EVEN, int OP>
hipError_t go_width(const RowArgs& A, hipStream_t st) {
  if (A.cols <= 128) return go<T, EVEN, 16, 8, OP>(A, st);
  if (A.cols <= 256) return go<T, EVEN, 32, 8, OP>(A, st);
  if (A.cols <= 512) return go<T, EVEN, 64, 8, OP>(A, st);
  if (A.cols <= 1024) return go<T, EVEN, 64, 16, OP>(A, st);
  if (A.cols <= 4096) return go<T, EVEN, 256, 16, OP>(A, st);
  if (A.cols <= 8192) return go<T, EVEN, 256, 32, OP>(A, st);
  if (A.cols <= 16384) return go<T, EVEN, 1024, 16, OP>(A, st);
  return go<T, EVEN, 1024, 32, OP>(A, st);
}

template <int T, int OP>
hipError_t go_vec(const RowArgs& A, hipStream_t st) {
  return A.cols % (16 / Type<T>::S) == 0 ? go_width<T, true, OP>(A, st) : go_width<T, false, OP>(A, st);
}

template <int OP>
hipError_t go_type(const RowArgs& A, int dtype, hipStream_t st) {
  switch (dtype) {
    case kBF16: return go_vec<kBF16, OP>(A, st);
    case kF16: return go_vec<kF16, OP>(A, st);
    default: return go_vec<kF32, OP>(A, st);
  }
}

// Work-groups of the gradient (4 waves up to 4096 columns, 8 or 16 above), and
// the rows that each takes at a time.
int64_t bwd_groups(int64_t rows, int64_t cols) {
  const int64_t most = cols <= 256 ? 2048 : cols <= 512 ? 1024 : cols <= 4096 ? 512 : 256;
  const int64_t at_a_time = cols <= 128 ? 16 : cols <= 256 ? 8 : cols <= 1024 ? 4 : 1;
  const int64_t need = (rows + at_a_time - 1) / at_a_time;
  return need < most ? need : most;
}

template <int T, bool EVEN, int TPR, int E>
hipError_t go_bwd(const BwdArgs& A, hipStream_t st) {
  hipLaunchKernelGGL((bwd_kernel<T, EVEN, TPR, E * Type<T>::S / 16>), dim3((unsigned)bwd_groups(A.rows, A.cols)),
                     dim3(TPR < 256 ? 256 : TPR), 0, st, A);
  return hipGetLastError();
}

template <int T, bool EVEN>
hipError_t go_bwd_width(const BwdArgs& A, hipStream_t st) {
  if (A.cols <= 128) return go_bwd<T, EVEN, 16, 8>(A, st);
  if (A.cols <= 256) return go_bwd<T, EVEN, 32, 8>(A, st);
  if (A.cols <= 512) return go_bwd<T, EVEN, 64, 8>(A, st);
  if (A.cols <= 1024) return go_bwd<T, EVEN, 64, 16>(A, st);
  if (A.cols <= 4096) return go_bwd<T, EVEN, 256, 16>(A, st);
  if (A.cols <= 8192) return go_bwd<T, EVEN, 512, 16>(A, st);
  if (A.cols <= 16384) return go_bwd<T, EVEN, 1024, 16>(A, st);
  return go_bwd<T, EVEN, 1024, 32>(A, st);
}

template <int T>
hipError_t go_bwd_vec(const BwdArgs& A, hipStream_t st) {
  return A.cols % (16 / Type<T>::S) == 0 ? go_bwd_width<T, true>(A, st) : go_bwd_width<T, false>(A, st);
}

RowArgs row_args(CMat x, CMat res, const void* w, int wdt, int64_t rows, int64_t cols, float eps,
                 int dtype, Mat h, Mat out, float* stat) {
  return RowArgs{x.p, res.p, w, h.p, out.p, stat, x.ld, res.ld, h.ld, out.ld, rows,
                 1.0 / (double)cols, (int)cols, eps,
                 w != nullptr && wdt == kF32 && dtype != kF32};
}

}  // namespace

hipError_t launch_rmsnorm(CMat x, CMat res, const void* weight, int weight_dtype, int64_t rows,
                          int64_t cols, float eps, int dtype, Mat h, Mat y, float* rstd,
                          hipStream_t stream) {
  return go_type<kNorm>(row_args(x, res, weight, weight_dtype, rows, cols, eps, dtype, h, y, rstd),
                        dtype, stream);
}

hipError_t launch_rmsnorm_int8(CMat x, CMat res, const void* weight, int weight_dtype,
                               int64_t rows, int64_t cols, float eps, int dtype, Mat h, Mat q,
                               float* scales, hipStream_t stream) {
  return go_type<kNormInt8>(
      row_args(x, res, weight, weight_dtype, rows, cols, eps, dtype, h, q, scales), dtype, stream);
}

hipError_t launch_int8_quantize(CMat x, CMat gate, int64_t rows, int64_t cols, int dtype, Mat q,
                                float* scales, hipStream_t stream) {
  const RowArgs A =
      row_args(x, gate, nullptr, kF32, rows, cols, 0.f, dtype, Mat{nullptr, 0}, q, scales);
  return gate.p ? go_type<kSwiglu>(A, dtype, stream) : go_type<kQuant>(A, dtype, stream);
}

size_t rmsnorm_bwd_ws(int64_t rows, int64_t cols) {
  return (size_t)bwd_groups(rows, cols) * (size_t)cols * sizeof(float);
}

hipError_t launch_rmsnorm_bwd(CMat dy, CMat dh, CMat h, const void* weight, int weight_dtype,
                              const float* rstd, int64_t rows, int64_t cols, int dtype, Mat dx,
                              void* dweight, void* ws, hipStream_t stream) {
  const BwdArgs A{dy.p,  dh.p,  h.p,  weight, rstd,      dx.p, dweight ? static_cast<float*>(ws) : nullptr,
                  dy.ld, dh.ld, h.ld, dx.ld,  rows, (int)cols, weight && weight_dtype == kF32 && dtype != kF32};
  if (rows > 0) {
    const hipError_t e = dtype == kBF16  ? go_bwd_vec<kBF16>(A, stream)
                         : dtype == kF16 ? go_bwd_vec<kF16>(A, stream)
                                         : go_bwd_vec<kF32>(A, stream);
    if (e != hipSuccess) return e;
  }
  if (dweight == nullptr) return hipSuccess;
  const dim3 grid((unsigned)((cols + 31) / 32)), blk(1024);
  const int parts = (int)bwd_groups(rows, cols);
  const float* p = static_cast<const float*>(ws);
  if (weight_dtype == kBF16)
    hipLaunchKernelGGL((dw_kernel<kBF16>), grid, blk, 0, stream, p, parts, (int)cols, dweight);
  else if (weight_dtype == kF16)
    hipLaunchKernelGGL((dw_kernel<kF16>), grid, blk, 0, stream, p, parts, (int)cols, dweight);
  else
    hipLaunchKernelGGL((dw_kernel<kF32>), grid, blk, 0, stream, p, parts, (int)cols, dweight);
  return hipGetLastError();
}

}  // namespace mx
