// Launch interface of attention's operators between their host API
// (api_attention.cpp) and their gfx950 kernels (heads.hip, attention.hip).
// Arguments are validated by the caller; the sizes' limits are here.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mxfp4.h"

namespace mx {

constexpr int64_t kHeadMax = 256;    // widest head: 32 threads of 8 values (heads.hip)
constexpr int64_t kHeadsMax = 1024;  // heads of a tensor
constexpr int64_t kPageUnit = 16;    // a page is a multiple: a matrix instruction's tokens lie in one page

// Heads [tokens][heads][dim] with a unit stride in dim.
struct Heads {
  const void* p;
  int64_t heads, ts, hs;
};

// The norm (eps < 0: none; not looked at by the gradient) and the weights of queries and keys (NULL: 1).
struct HeadNorm {
  const void *qw, *kw;
  bool wide;  // fp32 weights beside 16-bit heads
  float eps;
};

hipError_t launch_qk_norm_rope(Heads q, Heads k, int64_t tokens, int64_t dim, int dtype,
                               const mxfp4_rotation& rot, HeadNorm n, void* qo, void* ko, float* rstd,
                               hipStream_t stream);
// Gradients dx of q and k, and of the weights unless both are NULL (partial
// sums in ws, qk_norm_rope_bwd_ws bytes). rstd NULL: no norm.
hipError_t launch_qk_norm_rope_bwd(Heads dq, Heads dk, Heads q, Heads k, int64_t tokens, int64_t dim,
                                   int dtype, const mxfp4_rotation& rot, HeadNorm n, const float* rstd,
                                   void* dqx, void* dkx, void* dqw, void* dkw, void* ws, hipStream_t stream);
size_t qk_norm_rope_bwd_ws(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim);

// Queries to qo, keys and values to the cache's slots; q.heads may be 0.
hipError_t launch_int8_kv_write(Heads q, Heads k, Heads v, int64_t tokens, int64_t dim, int dtype,
                                const mxfp4_rotation& rot, HeadNorm n, const mxfp4_int8_kv& cache,
                                const int64_t* slots, void* qo, hipStream_t stream);
hipError_t launch_int8_kv_read(const mxfp4_int8_kv& cache, const int64_t* slots, int64_t tokens,
                               int64_t dim, int dtype, void* k, void* v, hipStream_t stream);

hipError_t launch_paged_attention(Heads q, int64_t batch, int64_t dim, int dtype,
                                  const mxfp4_int8_kv& cache, const int32_t* pages, int64_t pages_ld,
                                  int64_t table, const int32_t* lengths, float scale, int64_t window,
                                  void* out, float* lse, void* ws, hipStream_t stream);
size_t paged_attention_ws(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim,
                          int64_t table, int64_t page_size);

}  // namespace mx
