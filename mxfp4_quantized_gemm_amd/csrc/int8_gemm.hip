// Int8 matrix product with a scale for each token and each channel on
// gfx950's int8 MFMA (MI355X):
//   C[m][n] = (sum_k A[m][k] B[n][k]) sa[m] sb[n] + bias[n].
// The sum is exact: int32 accumulators, K <= 131071 so that even -128 * -128
// in every place stays below 2^31. It is rounded to fp32 once, then scaled,
// added to and rounded to C's type, so the result does not depend on the
// order of the sum, on the tiling or on how k is split.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

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

// The scaled sum: the int32 sum, its product with sa and the whole round to
// fp32 once each. Every kernel ends in this, so they agree bit for bit.
__device__ __forceinline__ float scaled(int acc, float sa, float sb, float bias) {
  return fmaf((float)acc * sa, sb, bias);
}

template <int OUT>
__device__ __forceinline__ void put(void* C, int64_t i, float v) {
  if constexpr (OUT == kF32) static_cast<float*>(C)[i] = v;
  if constexpr (OUT == kBF16) static_cast<__bf16*>(C)[i] = (__bf16)v;
  if constexpr (OUT == kF16) static_cast<_Float16*>(C)[i] = (_Float16)v;
}

template <int OUT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  if constexpr (OUT == kBF16) {
    const b2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    const h2 v = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, v);
  }
}

// ------------------------------------------------------ general kernel
// Any sizes, pitches and alignments (within the entry point's limits): 64 x 64 tiles of C, 4 waves of one 32 x
// 32 MFMA tile each, k in steps of 64 staged through LDS. 16 bytes of a row
// are loaded at once where its address allows it, byte by byte where not and
// at the row's end; rows and bytes past the operands are zero. It is far from the
// DMA kernels: 2048 x 6144 x 4112 in 157 us (their 2048 x 6144 x 4096: 58), and by
// bytes, where rows are not 16-byte aligned, x 4100 in 2.3 ms.
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
  const uint32_t ntn = (uint32_t)((P.N + BN - 1) / BN), tm = blockIdx.x / ntn;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)(blockIdx.x - tm * ntn) * BN;
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
    if (m < P.M) put<OUT>(P.C, m * P.ldc + n, scaled(acc[e], P.sa[m], sb, bias));
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

// ------------------------------------------------ LDS DMA building blocks
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes,
                                           0x00020000);
}

// One LDS DMA instruction: lane l's B bytes (4 or 16) at buffer offset voff +
// soff land at lds + B l. A lane whose voff lies past the resource's bytes
// reads zero.
template <int B, int NT = 0>
__device__ __forceinline__ void dma(rsrc_t r, uint8_t* lds, uint32_t voff, uint32_t soff) {
  static_assert(B == 4 || B == 16, "dwords or four of them");
  if constexpr (B == 4)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 4, voff, soff, 0, 0);
  else if constexpr (NT)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, voff, soff, 0, 2);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, voff, soff, 0, 0);
}

// s_waitcnt with vmcnt (and lgkmcnt 0 where LG) constrained.
template <int N, bool LG = false>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | ((LG ? 0 : 15) << 8));
}

// Rows of an operand from row r0 on, at most n of them, as a buffer.
__device__ __forceinline__ rsrc_t rows_rsrc(const uint8_t* p, int64_t r0, int64_t rows, int64_t n,
                                            int64_t ld) {
  return make_rsrc(p + r0 * ld, min(rows - r0, n) * ld);
}

// k-tiles are 128 bytes of every operand row, row-major in LDS, 16-byte chunk
// c of row r at slot c ^ ((r >> 1) & 7): a DMA instruction (8 whole rows) stays
// contiguous, 8 lanes fetch a whole 128-byte row, and the 16 lanes of a
// fragment read (one chunk of rows r .. r + 15) land on distinct banks.
constexpr int KB = 128;

// Offset of lane l's chunk in DMA block u (rows 8 u .. 8 u + 7).
__device__ __forceinline__ uint32_t dma_off(int u, int lane, int64_t ld) {
  const int row = 8 * u + (lane >> 3);
  return (uint32_t)(row * ld + (((lane & 7) ^ ((row >> 1) & 7)) << 4));
}

// LDS offset of the fragment of k-step s: chunk 2 s + lane / 32 of row lane % 32.
__device__ __forceinline__ uint32_t frag_off(int s, int lane) {
  const int l32 = lane & 31, h = lane >> 5;
  return (uint32_t)(l32 * KB + (((2 * s + h) ^ ((l32 >> 1) & 7)) << 4));
}

// Work-group id -> output tile. Consecutive ids go round-robin over the 8
// XCDs; each XCD gets a contiguous range of logical tiles, walked in groups
// of 4 tile-rows, so that the tiles resident on one XCD share operand rows in
// its L2. (There are at most 2^23 tiles. Divisions of 64 bits cost 1 us before the
// first load: 64 x 1024 x 1024 6.0 -> 5.0, 333 x 1537 x 2816 11.5 -> 10.1.)
__device__ __forceinline__ void tile_of(uint32_t wg, uint32_t nwg, uint32_t ntm, uint32_t ntn,
                                        uint32_t& tm, uint32_t& tn) {
  const uint32_t per = nwg / 8;
  uint32_t lg = wg;
  if (wg < per * 8) lg = (wg % 8) * per + wg / 8;
  const uint32_t width = 4 * ntn, g = lg / width, first = g * 4;
  const uint32_t gs = min(ntm - first, 4u), r = lg - g * width;
  tn = r / gs;
  tm = first + r - tn * gs;
}

// ------------------------------------------------------------- epilogue
// The tiled kernels give the MFMA the weight's rows first, so that a lane's
// registers 4 q .. 4 q + 3 are four consecutive columns (8 q + 4 (lane / 32)) of
// row lane % 32 of C. Tiles go out through LDS, each wave its own 2.5 KiB:
// lanes then store 16 bytes each of 64 or 128 consecutive bytes of a row, at
// any alignment. (8192 x 28672 x 4096 bf16, us: 128-byte rows 830, 64-byte rows
// 872, 4-byte stores straight from the registers after exchanges between
// lanes 843; with a width of 4097 164 / 196 / 168. Kept in the caches instead
// of past them 848. The middle sizes gained from 64-byte rows over 2-byte
// stores: 1024 x 6144 x 4096 35.9 -> 32.6, 512 x 4096 x 4096 32.5 -> 29.2.)
constexpr int kI32 = 3;                  // partial sums of a split of k
constexpr int kStage = 32 * (64 + 16);   // rows padded by 16 bytes: banks spread

// A tile's scales and bias in LDS, filled by DMA (rows past the end are 0).
struct Factors {
  const float *sa, *sb, *bias;
};

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Staged rows of RB bytes (32 of 64 or 16 of 128) to C from row m0, column n0.
template <int OUT, int RB>
__device__ __forceinline__ void store_rows(const uint8_t* stage, void* C, int64_t ldc, int64_t m0,
                                           int64_t n0, int64_t M, int64_t N, int lane) {
  typedef u32x4 u32x4_2 __attribute__((aligned(2)));  // C may start at any element
  constexpr int S = OUT == kBF16 || OUT == kF16 ? 2 : 4, V = 16 / S, L = RB / 16;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 64 / L * h + lane / L;
    const u32x4 q = *reinterpret_cast<const u32x4*>(stage + r * (RB + 16) + lane % L * 16);
    const int64_t m = m0 + r, n = n0 + lane % L * V;
    uint8_t* p = static_cast<uint8_t*>(C) + (m * ldc + n) * S;
    if (m < M && n + V <= N) {
      if constexpr (OUT == kI32)
        *reinterpret_cast<u32x4_2*>(p) = q;  // read again soon
      else
        __builtin_nontemporal_store(q, reinterpret_cast<u32x4_2*>(p));
    } else if (m < M) {
#pragma unroll
      for (int e = 0; e < V - 1; ++e) {
        const uint32_t d = q[e * S / 4];
        if (n + e < N) {
          if constexpr (S == 4)
            reinterpret_cast<uint32_t*>(p)[e] = d;
          else
            reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(d >> (16 * (e & 1)));
        }
      }
    }
  }
}

// The lane's four columns of group q of a tile, scaled: 16 bits or 32 each.
template <int OUT>
__device__ __forceinline__ u32x4 four(const v16i& acc, int q, float sa, Factors F, int half) {
  const float4 sb = *reinterpret_cast<const float4*>(F.sb + 8 * q + 4 * half);
  const float4 b = *reinterpret_cast<const float4*>(F.bias + 8 * q + 4 * half);
  const float v0 = scaled(acc[4 * q], sa, sb.x, b.x), v1 = scaled(acc[4 * q + 1], sa, sb.y, b.y);
  const float v2 = scaled(acc[4 * q + 2], sa, sb.z, b.z), v3 = scaled(acc[4 * q + 3], sa, sb.w, b.w);
  if constexpr (OUT == kF32)
    return u32x4{__float_as_uint(v0), __float_as_uint(v1), __float_as_uint(v2), __float_as_uint(v3)};
  else
    return u32x4{pack2<OUT>(v0, v1), pack2<OUT>(v2, v3), 0, 0};
}

// One tile (rows m0 .., columns n0 ..) of C, 64 bytes of every row at a time;
// its rows' scales start at F.sa, its columns' at F.sb and F.bias (not read
// for partial sums). `stage` is the wave's own.
template <int OUT>
__device__ __forceinline__ void put_tile(const v16i& acc, uint8_t* stage, Factors F, void* C, int64_t ldc,
                                         int64_t m0, int64_t n0, int64_t M, int64_t N, int lane) {
  const int half = lane >> 5, l32 = lane & 31;
  uint8_t* row = stage + l32 * (64 + 16);
  if constexpr (OUT == kBF16 || OUT == kF16) {
    const float sa = F.sa[l32];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4 d = four<OUT>(acc, q, sa, F, half);
      *reinterpret_cast<u32x2*>(row + 16 * q + 8 * half) = u32x2{d.x, d.y};
    }
    wave_sync();
    store_rows<OUT, 64>(stage, C, ldc, m0, n0, M, N, lane);
    wave_sync();
  } else {
    const float sa = OUT == kI32 ? 0.f : F.sa[l32];
#pragma unroll
    for (int p = 0; p < 2; ++p) {  // 16 columns each
#pragma unroll
      for (int q = 2 * p; q < 2 * p + 2; ++q) {
        u32x4 d;
        if constexpr (OUT == kI32)
          d = u32x4{(uint32_t)acc[4 * q], (uint32_t)acc[4 * q + 1], (uint32_t)acc[4 * q + 2], (uint32_t)acc[4 * q + 3]};
        else
          d = four<OUT>(acc, q, sa, F, half);
        *reinterpret_cast<u32x4*>(row + 32 * (q & 1) + 16 * half) = d;
      }
      wave_sync();
      store_rows<OUT, 64>(stage, C, ldc, m0, n0 + 16 * p, M, N, lane);
      wave_sync();
    }
  }
}

// Two tiles side by side, 128 bytes of 16 rows at a time: 64 columns of 16
// bits, or each tile's 32 columns of 32 bits in turn.
template <int OUT>
__device__ __forceinline__ void put_pair(const v16i& acc0, const v16i& acc1, uint8_t* stage, Factors F, void* C,
                                         int64_t ldc, int64_t m0, int64_t n0, int64_t M, int64_t N, int lane) {
  const int half = lane >> 5, l32 = lane & 31;
  const float sa = F.sa[l32];
  const Factors F1{F.sa, F.sb + 32, F.bias + 32};
  uint8_t* row = stage + (l32 & 15) * (128 + 16);
  u32x4 d[2][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) d[0][q] = four<OUT>(acc0, q, sa, F, half);
#pragma unroll
  for (int q = 0; q < 4; ++q) d[1][q] = four<OUT>(acc1, q, sa, F1, half);
#pragma unroll
  for (int p = 0; p < 2; ++p) {  // rows 0-15, 16-31
    if constexpr (OUT == kF32) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (l32 >> 4 == p) {
#pragma unroll
          for (int q = 0; q < 4; ++q) *reinterpret_cast<u32x4*>(row + 32 * q + 16 * half) = d[j][q];
        }
        wave_sync();
        store_rows<OUT, 128>(stage, C, ldc, m0 + 16 * p, n0 + 32 * j, M, N, lane);
        wave_sync();
      }
    } else {
      if (l32 >> 4 == p) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<u32x2*>(row + 64 * j + 16 * q + 8 * half) = u32x2{d[j][q].x, d[j][q].y};
      }
      wave_sync();
      store_rows<OUT, 128>(stage, C, ldc, m0 + 16 * p, n0, M, N, lane);
      wave_sync();
    }
  }
}

// Scales and bias of the BM rows from m0 and the BN columns from n0 to LDS
// (sa, then sb, then bias; without a bias zeros), 64 of them an instruction.
template <int BM, int BN, int NW>
__device__ __forceinline__ void fetch_factors(uint8_t* lds, const Args& P, int64_t m0, int64_t n0,
                                              rsrc_t none, int wave, int lane) {
  const int64_t mb = min(P.M - m0, (int64_t)BM) * 4, nb = min(P.N - n0, (int64_t)BN) * 4;
#pragma unroll
  for (int u = 0; u < (BM + 2 * BN) / 64; u += NW) {
    const int blk = u + wave;
    if (blk < BM / 64)
      dma<4>(make_rsrc(P.sa + m0, mb), lds + blk * 256, (blk * 64 + lane) * 4, 0);
    else if (blk < (BM + BN) / 64)
      dma<4>(make_rsrc(P.sb + n0, nb), lds + blk * 256, ((blk - BM / 64) * 64 + lane) * 4, 0);
    else if (blk < (BM + 2 * BN) / 64)
      dma<4>(P.bias ? make_rsrc(P.bias + n0, nb) : none, lds + blk * 256,
             ((blk - (BM + BN) / 64) * 64 + lane) * 4, 0);
  }
}

// ------------------------------------------------------- few tokens (M <= 16 MG)
// The weight's bytes are the work. A work-group owns 16 rows of B and its W
// waves split k: of the chunks of 64 bytes of the 16 rows, 2 c and 2 c + 1 belong
// to wave c % W, loaded straight into registers in the MFMA's layout (lane l:
// row l % 16, 16 bytes at 16 (l / 16)), so W waves read 128 W consecutive bytes
// of each row. A wave keeps U chunks in flight: a chunk's registers are loaded again right
// after its MFMA. Chunks past the end are loads out of the buffer's range
// (zero, no traffic), so that a round of U has no branches. The tokens (A) come
// from the caches. Partial sums meet in LDS. Measured: 4096 x 14336, one token
// in 11.0-11.6 us with B from memory, 5.1-5.3 TB/s. B is read through the caches: past them (it is used
// once) was slower whether it lay in the last-level cache (10.2 against 14.3)
// or not (12.1 against 13.0).
namespace few {

template <int W, int U, int MG, int NG, int OUT>
__global__ __launch_bounds__(64 * W) void gemm_kernel(Args P) {
  __shared__ int red[W][MG * NG][64 * 4];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NG);
  const rsrc_t rb = rows_rsrc(P.B, n0, P.N, 16 * NG, P.ldb), ra = rows_rsrc(P.A, 0, P.M, 16 * MG, P.lda);
  uint32_t va[MG], vb[NG];
#pragma unroll
  for (int g = 0; g < MG; ++g) va[g] = (uint32_t)((16 * g + (lane & 15)) * P.lda + 16 * (lane >> 4));
#pragma unroll
  for (int h = 0; h < NG; ++h) vb[h] = (uint32_t)((16 * h + (lane & 15)) * P.ldb + 16 * (lane >> 4));
  const int chunks = (int)(P.K / 64);
  v4i acc[NG][MG], qb[U][NG], qa[U][MG];
#pragma unroll
  for (int h = 0; h < NG; ++h)
#pragma unroll
    for (int g = 0; g < MG; ++g) acc[h][g] = v4i{0, 0, 0, 0};
  // Work-groups start at different chunks and wrap around: rows whose pitch is
  // a multiple of 4 KiB would else be read at the same place of it by all of
  // them, which is the same few memory channels (one token, us: 8192 x 8192
  // 17.2 -> 11.7, 4096 x 4096 5.4 -> 4.7, 4096 x 14336 as before).
  const int rot = (int)(blockIdx.x / 8 * 4 % (unsigned)chunks);
  auto load = [&](int u, int c) {
    const uint32_t dead = c < chunks ? 0u : 0x80000000u;  // rows are below 2^23 bytes
    const uint32_t so = (uint32_t)(c + rot - (c + rot >= chunks ? chunks : 0)) * 64;
#pragma unroll
    for (int h = 0; h < NG; ++h)
      qb[u][h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rb, vb[h] | dead, so, 0));
#pragma unroll
    for (int g = 0; g < MG; ++g)
      qa[u][g] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(ra, va[g] | dead, so, 0));
  };
  // a wave's loads take the two halves of 128-byte lines one after the other
  static_assert(U % 2 == 0, "pairs of chunks");
  auto chunk = [&](int u) { return 2 * wave + u / 2 * 2 * W + u % 2; };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, chunk(u));
  auto mul = [&](int u) {
#pragma unroll
    for (int h = 0; h < NG; ++h)
#pragma unroll
      for (int g = 0; g < MG; ++g)
        acc[h][g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(qb[u][h], qa[u][g], acc[h][g], 0, 0, 0);
  };
  for (int c = W * U; c < chunks; c += W * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mul(u);
      load(u, c + chunk(u));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) mul(u);
  // register e of lane l is row 4 (l / 16) + e of B, token l % 16
#pragma unroll
  for (int h = 0; h < NG; ++h)
#pragma unroll
    for (int g = 0; g < MG; ++g) *reinterpret_cast<v4i*>(&red[wave][h * MG + g][4 * lane]) = acc[h][g];
  __syncthreads();
  for (int i = t; i < 256 * MG * NG; i += 64 * W) {
    const int n = i % (16 * NG), m = i / (16 * NG);  // neighbouring threads, neighbouring columns
    const int64_t row = m, col = n0 + n;
    if (row >= P.M || col >= P.N) continue;
    const int at = (n >> 4) * MG + (m >> 4), l = 4 * ((m & 15) + 16 * ((n & 15) >> 2)) + (n & 3);
    int s = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[w][at][l];
    put<OUT>(P.C, row * P.ldc + col, scaled(s, P.sa[row], P.sb[col], P.bias ? P.bias[col] : 0.f));
  }
}

template <int W, int U, int MG, int NG, int OUT>
hipError_t launch(const Args& P, hipStream_t st) {
  hipLaunchKernelGGL((gemm_kernel<W, U, MG, NG, OUT>), dim3((unsigned)((P.N + 16 * NG - 1) / (16 * NG))),
                     dim3(64 * W), 0, st, P);
  return hipGetLastError();
}

}  // namespace few

// ------------------------------------------- ring of k-tiles (middle sizes)
// WM x WN waves of TM x TN MFMA tiles; k-tiles run through a ring of NS LDS
// buffers filled by DMA NS - 1 ahead, one barrier a k-tile. Where there
// are fewer output tiles than CUs the k range is split over blockIdx.y: the
// int32 partial sums go to the workspace and a second kernel adds them (the
// sums are exact, so the split does not show in the result).
// What bounds it, while the operands lie in the caches and up to half of the CUs
// work: the LDS, written by DMA at 64 bytes a clock and read at 256, not both at
// once. A k-tile of 64 x 128 (8 waves of 32 x 32) is 384 + 256 clocks beside 256 of
// MFMAs, and takes 0.25-0.28 us on 64 to 128 CUs. Past that it is the operands' way
// to the CUs: with all CUs at work 0.32-0.36 us a k-tile from the caches (24 KB to
// each of 256 CUs: 17-19 TB/s), and 0.44-0.50 us, on 128 CUs too, where the operands
// come from memory (512 x 4096 x 14336, 112 k-tiles: 39 us the one way, 52 the
// other). Tiles that need fewer operand bytes follow; 128 x 128 with 8 waves of 64 x 32 is 512 + 384 (16 waves of
// 32 x 32: 512 + 512; 512 x 6144 x 4096 16.6 against 17.4 us), 128 x 256 with 8
// waves of 64 x 64 is 768 + 512 (16 of 32 x 64: 768 + 768; 1024 x 6144 x 4096
// 27.1 against 28.0). Fragments read a whole k-tile ahead, and rows touched in
// the L2 up to 16 k-tiles ahead by a wave of its own, gained nothing. For few
// tokens it is B from memory: 28672 x 4096, 64 tokens in 21.2 us, 5.7 TB/s.
namespace ring {

template <int WM_, int WN_, int TM_, int TN_, int NS_, int SP_ = 4, int NTB_ = 0>
struct G {
  static constexpr int NTB = NTB_;  // B is read once: do not keep it in the caches
  static constexpr int SP = SP_;  // k-steps that a k-tile's DMAs are spread over
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, NS = NS_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int BM = 32 * WM * TM, BN = 32 * WN * TN;
  static constexpr int NB = (BM + BN) / 8 / NW;  // DMA blocks (8 rows) per wave and k-tile
  static constexpr int STAGE = (BM + BN) * KB;
  static_assert((BM + BN) % (8 * NW) == 0, "DMA blocks divide over the waves");
  static_assert(NS >= 2 && NS <= 6 && (NS - 1) * NB < 64, "vmcnt range");
};

template <class T>
struct Frag {
  v4i a[T::TM], b[T::TN];
};

template <class T>
struct Lane {
  uint32_t off[T::NB];  // DMA offsets
  uint32_t fa[4], fb[4];
};

// DMAs [U0, U1) of the k-tile at byte ko into st; nothing is fetched where it is not live.
template <class T, int U0 = 0, int U1 = T::NB>
__device__ __forceinline__ void fetch(uint8_t* st, rsrc_t ra, rsrc_t rb, rsrc_t none, bool live,
                                      const Lane<T>& L, uint32_t ko, int wave) {
#pragma unroll
  for (int u = U0; u < U1; ++u) {
    const int blk = T::NW * u + wave;  // uniform: blocks of A, then of B
    // (which of the two is known here where A's blocks divide over the waves)
    const bool of_a = T::BM / 8 % T::NW == 0 ? u < T::BM / 8 / T::NW : 8 * blk < T::BM;
    if (of_a)
      dma<16>(live ? ra : none, st + blk * 1024, L.off[u], ko);
    else
      dma<16, T::NTB>(live ? rb : none, st + blk * 1024, L.off[u], ko);
  }
}

template <class T, int S>
__device__ __forceinline__ void read(const uint8_t* st, const Lane<T>& L, Frag<T>& F) {
#pragma unroll
  for (int i = 0; i < T::TM; ++i) F.a[i] = *reinterpret_cast<const v4i*>(st + L.fa[S] + i * 32 * KB);
#pragma unroll
  for (int j = 0; j < T::TN; ++j) F.b[j] = *reinterpret_cast<const v4i*>(st + L.fb[S] + j * 32 * KB);
}

template <class T>
__device__ __forceinline__ void mul(const Frag<T>& F, v16i (&acc)[T::TM][T::TN]) {
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
#pragma unroll
    for (int j = 0; j < T::TN; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(F.b[j], F.a[i], acc[i][j], 0, 0, 0);
}

// Scheduling of a k-step: its LDS reads and DMAs spread over its MFMAs (left
// alone, the compiler bunches them behind the MFMAs). DMAs come after an MFMA:
// a wave waits at a DMA while the load unit is busy, and an MFMA then runs.
template <class T, int R, int NL>
__device__ __forceinline__ void interleave() {
  constexpr int NM = T::TM * T::TN, NR = T::TM + T::TN;
  if constexpr (R < NM) {
    constexpr int r = NR * (R + 1) / NM - NR * R / NM, l = NL * (R + 1) / NM - NL * R / NM;
    if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(0x020, l, 0);
    interleave<T, R + 1, NL>();
  } else {
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Steps k, k + 1, ... (at most N) that lie below end.
template <int N, int I = 0, class F>
__device__ __forceinline__ void steps(F& step, int k, int end) {
  if constexpr (I < N) {
    if (k + I >= end) return;
    step(std::integral_constant<int, I>{}, k + I);
    steps<N, I + 1>(step, k, end);
  }
}

template <class T, int OUT>
__global__ __launch_bounds__(T::NT) void gemm_kernel(Args P, int splits, int* part) {
  constexpr int NS = T::NS, NB = T::NB;
  // separate arrays: the compiler sees that a DMA into one does not feed reads
  // of another, and adds no waits
  __shared__ __attribute__((aligned(16))) uint8_t s0[T::STAGE], s1[T::STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t s2[NS > 2 ? T::STAGE : 16], s3[NS > 3 ? T::STAGE : 16];
  __shared__ __attribute__((aligned(16))) uint8_t s4[NS > 4 ? T::STAGE : 16], s5[NS > 5 ? T::STAGE : 16];
  __shared__ __attribute__((aligned(16))) uint8_t factors[(T::BM + 2 * T::BN) * 4];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;
  const uint32_t ntm = (uint32_t)((P.M + T::BM - 1) / T::BM), ntn = (uint32_t)((P.N + T::BN - 1) / T::BN);
  uint32_t tm, tn;
  tile_of(blockIdx.x, gridDim.x, ntm, ntn, tm, tn);
  const int64_t m0 = (int64_t)tm * T::BM, n0 = (int64_t)tn * T::BN;
  // the split's k-tiles: [k0, k0 + nk), at least one
  const int all = (int)(P.K / KB), z = blockIdx.y;
  const int k0 = all * z / splits, nk = all * (z + 1) / splits - k0;
  // Tiles start at different k-tiles and wrap around, where B streams from
  // memory: rows whose pitch is a multiple of 4 KiB would else be read at the
  // same place of that pitch by all tiles at once, which is the same few memory
  // channels (28672 x 4096, us: 16 tokens 25.4 -> 21.7, 64 tokens 26.8 -> 23.6;
  // 28672 x 8192 48.5 -> 37.9). Other tiles share A's rows in the L2 by running
  // in step (512 x 6144 x 4096: 19.5, rotated 21.1).
  const int rot = T::NTB ? (int)(tn * (uint32_t)nk / ntn) : 0;
  auto at = [&](int k) { return (uint32_t)(k0 + k + rot - (k + rot >= nk ? nk : 0)) * KB; };
  const rsrc_t ra = rows_rsrc(P.A, m0, P.M, T::BM, P.lda), rb = rows_rsrc(P.B, n0, P.N, T::BN, P.ldb);
  const rsrc_t none = make_rsrc(P.A, 0);
  Lane<T> L;
#pragma unroll
  for (int u = 0; u < NB; ++u) {
    const int blk = T::NW * u + wave;
    L.off[u] = 8 * blk < T::BM ? dma_off(blk, lane, P.lda) : dma_off(blk - T::BM / 8, lane, P.ldb);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    L.fa[s] = (uint32_t)(wm * T::TM * 32 * KB) + frag_off(s, lane);
    L.fb[s] = (uint32_t)((T::BM + wn * T::TN * 32) * KB) + frag_off(s, lane);
  }
  v16i acc[T::TM][T::TN];
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
#pragma unroll
    for (int j = 0; j < T::TN; ++j) acc[i][j] = v16i{};

  auto slot = [&](int s) {
    return s == 0 ? s0 : s == 1 ? s1 : s == 2 ? s2 : s == 3 ? s3 : s == 4 ? s4 : s5;
  };
  // the scales and bias, the first NS - 1 k-tiles and the first part of the
  // next; the first k-tile has landed when only the others' DMAs are outstanding
  if (splits == 1) fetch_factors<T::BM, T::BN, T::NW>(factors, P, m0, n0, none, wave, lane);
#pragma unroll
  for (int k = 0; k < NS - 1; ++k)
    fetch<T>(slot(k), ra, rb, none, k < nk, L, at(k), wave);
  fetch<T, 0, NB / T::SP>(slot(NS - 1), ra, rb, none, NS - 1 < nk, L, at(NS - 1), wave);
  wait_vm<(NS - 2) * NB + NB / T::SP>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frag<T> F0, F1;
  read<T, 0>(s0, L, F0);
  // k-tile k in slot S: a k-step's MFMAs run on fragments read during the
  // k-step before. The barrier before the last k-step publishes k-tile k + 1
  // (each wave's own DMAs of it have landed, the later ones stay in flight)
  // and retires slot S (each wave's reads of it are done), which takes k-tile
  // k + NS: the first of its SP parts here, the others with the first k-steps
  // of k-tile k + 1.
  auto part_of = [&](auto S, auto Q, int k) {  // part Q of k-tile k into slot S
    constexpr int u0 = NB * Q.value / T::SP, u1 = NB * (Q.value + 1) / T::SP;
    if constexpr (Q.value < T::SP)
      fetch<T, u0, u1>(slot(S.value), ra, rb, none, k < nk, L, at(k), wave);
  };
  auto count = [](int q) { return q < T::SP ? NB * (q + 1) / T::SP - NB * q / T::SP : 0; };
  auto step = [&](auto S, int k) {
    constexpr std::integral_constant<int, (S.value + NS - 1) % NS> before{};
    uint8_t* st = slot(S.value);
    read<T, 1>(st, L, F1);
    mul<T>(F0, acc);
    part_of(before, std::integral_constant<int, 1>{}, k - 1 + NS);
    interleave<T, 0, count(1)>();
    read<T, 2>(st, L, F0);
    mul<T>(F1, acc);
    part_of(before, std::integral_constant<int, 2>{}, k - 1 + NS);
    interleave<T, 0, count(2)>();
    read<T, 3>(st, L, F1);
    mul<T>(F0, acc);
    part_of(before, std::integral_constant<int, 3>{}, k - 1 + NS);
    interleave<T, 0, count(3)>();
    wait_vm<(NS - 2) * NB, true>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read<T, 0>(slot((S.value + 1) % NS), L, F0);
    part_of(S, std::integral_constant<int, 0>{}, k + NS);
    mul<T>(F1, acc);
    interleave<T, 0, count(0)>();
  };
  // Whole turns of the ring, then the rest: with exits inside the loop the
  // compiler saw ways to its start on which slot 0 was just fetched, and waited
  // there for all DMAs (512 x 6144 x 4096 18.7 -> 17.4, 64 x 28672 x 4096
  // 22.7 -> 21.2).
  int k = 0;
  for (; k + NS <= nk; k += NS) steps<NS>(step, k, k + NS);
  steps<NS - 1>(step, k, nk);
  // The last (empty) DMAs land and every wave is done with the slots: the
  // first ones become the waves' staging of the epilogue.
  wait_vm<0, true>();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  static_assert(T::NW * kStage <= 2 * T::STAGE, "staging fits two slots");
  uint8_t* stage = wave * kStage + kStage <= T::STAGE ? s0 + wave * kStage : s1 + (wave - T::STAGE / kStage) * kStage;
  const float* f = reinterpret_cast<const float*>(factors);
#pragma unroll
  for (int j = 0; j < T::TN; ++j)
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
      const int r = (wm * T::TM + i) * 32, c = (wn * T::TN + j) * 32;
      const Factors F{f + r, f + T::BM + c, f + T::BM + T::BN + c};
      if (splits == 1)
        put_tile<OUT>(acc[i][j], stage, F, P.C, P.ldc, m0 + r, n0 + c, P.M, P.N, lane);
      else
        put_tile<kI32>(acc[i][j], stage, F, part + (int64_t)z * P.M * P.N, P.N, m0 + r, n0 + c, P.M, P.N, lane);
    }
}

// Four columns a thread, at any alignment.
template <int OUT>
__global__ __launch_bounds__(256) void sum_kernel(Args P, int splits, const int* part) {
  typedef v4i v4i_4 __attribute__((aligned(4)));
  typedef u32x4 u32x4_4 __attribute__((aligned(4)));
  typedef u32x2 u32x2_2 __attribute__((aligned(2)));
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, m = blockIdx.y;
  if (n >= P.N) return;
  const float sa = P.sa[m];
  const int* p = part + m * P.N + n;
  if (n + 4 <= P.N) {
    v4i s = {0, 0, 0, 0};
#pragma unroll 4
    for (int z = 0; z < splits; ++z) s += *reinterpret_cast<const v4i_4*>(p + z * P.M * P.N);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = scaled(s[e], sa, P.sb[n + e], P.bias ? P.bias[n + e] : 0.f);
    if constexpr (OUT == kF32)
      *reinterpret_cast<u32x4_4*>(static_cast<float*>(P.C) + m * P.ldc + n) =
          u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    else
      *reinterpret_cast<u32x2_2*>(static_cast<uint16_t*>(P.C) + m * P.ldc + n) =
          u32x2{pack2<OUT>(v[0], v[1]), pack2<OUT>(v[2], v[3])};
  } else {
    for (int e = 0; n + e < P.N; ++e) {
      int s = 0;
      for (int z = 0; z < splits; ++z) s += p[z * P.M * P.N + e];
      put<OUT>(P.C, m * P.ldc + n + e, scaled(s, sa, P.sb[n + e], P.bias ? P.bias[n + e] : 0.f));
    }
  }
}

template <class T, int OUT>
hipError_t launch(const Args& P, int splits, void* ws, hipStream_t st) {
  const int64_t tiles = ((P.M + T::BM - 1) / T::BM) * ((P.N + T::BN - 1) / T::BN);
  hipLaunchKernelGGL((gemm_kernel<T, OUT>), dim3((unsigned)tiles, splits), dim3(T::NT), 0, st, P, splits,
                     static_cast<int*>(ws));
  if (splits > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((sum_kernel<OUT>), dim3((unsigned)((P.N + 1023) / 1024), (unsigned)P.M), dim3(256), 0,
                       st, P, splits, static_cast<const int*>(ws));
  }
  return hipGetLastError();
}

}  // namespace ring

// --------------------------------------------------- large products
// Persistent: one 512-thread work-group per CU walks 256 x 256 output tiles,
// 8 waves (2 x 4) of 128 x 64, that is 4 x 2 MFMA tiles and 128 accumulators
// a lane. Two LDS stages of one k-tile each, filled by DMA: a k-tile's four
// k-steps of 8 MFMAs each run on fragments that were read during the k-step
// before, the next k-tile's DMAs are issued in two halves one k-step apart,
// and the barrier comes before the last k-step, whose MFMAs run after it
// together with the first reads of the next k-tile. The operand stream does
// not stop at a tile's end: the last k-tiles prefetch the next tile's first.
// What bounds it is power: at 8192 x 28672 x 4096 (790-860 us on different
// boxes, 2.25-2.44 POP/s) the clock falls to 1.4 GHz with the MFMAs busy 72 %
// of the time; one tile on an idle chip runs at 87 % and 2.4 GHz. A tile's
// epilogue costs about 6 of its 60 us there.
// The tile's scales and bias come by DMA too (its first k-tile), so that the
// epilogue waits for no load.
namespace big {

constexpr int BM = 256, BN = 256, TM = 4, TN = 2, WN = 4;  // (put_pair takes the two)
constexpr int TILE = BM * KB, STAGE = 2 * TILE;
constexpr int DA = 4;  // DMA blocks of an operand per wave and k-tile

struct Tile {
  rsrc_t a, b;
  int64_t m0, n0;
};

struct Frag {
  v4i a[TM], b[TN];
};

struct Offs {
  uint32_t a[DA], b[DA], fa[4], fb[4];
};

// Half H of k-tile kk into st: of the current tile, of the next one when kk
// runs past the (even) number of k-tiles np, nothing where there is none.
template <int H>
__device__ __forceinline__ void fetch(uint8_t* st, const Tile& c, const Tile& n, bool has_next,
                                      rsrc_t none, const Offs& O, int kk, int nk, int np, int wave) {
  const bool nx = kk >= np;
  const int k = nx ? kk - np : kk;
  const bool live = k < nk && (!nx || has_next);
  const rsrc_t ra = live ? (nx ? n.a : c.a) : none, rb = live ? (nx ? n.b : c.b) : none;
  const uint32_t ko = (uint32_t)k * KB;
#pragma unroll
  for (int u = 2 * H; u < 2 * H + 2; ++u) dma<16>(ra, st + (DA * wave + u) * 1024, O.a[u], ko);
#pragma unroll
  for (int u = 2 * H; u < 2 * H + 2; ++u) dma<16>(rb, st + TILE + (DA * wave + u) * 1024, O.b[u], ko);
}

template <int S>
__device__ __forceinline__ void read(const uint8_t* st, const Offs& O, Frag& F) {
#pragma unroll
  for (int i = 0; i < TM; ++i) F.a[i] = *reinterpret_cast<const v4i*>(st + O.fa[S] + i * 32 * KB);
#pragma unroll
  for (int j = 0; j < TN; ++j) F.b[j] = *reinterpret_cast<const v4i*>(st + O.fb[S] + j * 32 * KB);
}

__device__ __forceinline__ void mul(const Frag& F, v16i (&acc)[TN][TM]) {
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i)
      acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(F.b[j], F.a[i], acc[j][i], 0, 0, 0);
}

// One MFMA, then an LDS read and a DMA where there are any left, and so on.
template <int R, int NR, int NL>
__device__ __forceinline__ void interleave() {
  constexpr int NM = TM * TN;
  if constexpr (R < NM) {
    constexpr int r = R < NR ? (R == NM - 1 ? NR - R : 1) : 0;
    constexpr int l = NL * (R + 1) / NM - NL * R / NM;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
    if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(0x020, l, 0);
    interleave<R + 1, NR, NL>();
  }
}

// k-tile k of the current tile, in st; F0 holds its first fragments. The
// stage nx holds k-tile k + 1 but for its second half.
__device__ __forceinline__ void ktile(uint8_t* st, uint8_t* nx, const Tile& c, const Tile& n,
                                      bool has_next, rsrc_t none, const Offs& O, Frag& F0, Frag& F1,
                                      v16i (&acc)[TN][TM], int k, int nk, int np, int wave) {
  constexpr int NR = TM + TN;
  read<1>(st, O, F1);
  mul(F0, acc);
  fetch<1>(nx, c, n, has_next, none, O, k + 1, nk, np, wave);
  interleave<0, NR, 4>();
  __builtin_amdgcn_sched_barrier(0);
  read<2>(st, O, F0);
  mul(F1, acc);
  interleave<0, NR, 0>();
  __builtin_amdgcn_sched_barrier(0);
  read<3>(st, O, F1);
  mul(F0, acc);
  interleave<0, NR, 0>();
  __builtin_amdgcn_sched_barrier(0);
  wait_vm<0>();
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  read<0>(nx, O, F0);
  fetch<0>(st, c, n, has_next, none, O, k + 2, nk, np, wave);
  mul(F1, acc);
  interleave<0, NR, 4>();
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ Tile tile_at(const Args& P, uint32_t vt, uint32_t ntiles, uint32_t ntm,
                                        uint32_t ntn) {
  Tile T;
  uint32_t tm, tn;
  tile_of(vt, ntiles, ntm, ntn, tm, tn);
  T.m0 = (int64_t)tm * BM;
  T.n0 = (int64_t)tn * BN;
  T.a = rows_rsrc(P.A, T.m0, P.M, BM, P.lda);
  T.b = rows_rsrc(P.B, T.n0, P.N, BN, P.ldb);
  return T;
}

template <int OUT>
__global__ __attribute__((amdgpu_flat_work_group_size(512, 512), amdgpu_waves_per_eu(2)))
void gemm_kernel(Args P) {
  __shared__ __attribute__((aligned(16))) uint8_t st0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t st1[STAGE];
  __shared__ __attribute__((aligned(16))) float sc[2][3 * 256];  // sa, sb, bias of a tile
  __shared__ __attribute__((aligned(16))) uint8_t staging[8 * kStage];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t ntm = (uint32_t)((P.M + BM - 1) / BM), ntn = (uint32_t)((P.N + BN - 1) / BN);
  const uint32_t ntiles = ntm * ntn, step = gridDim.x;
  const int nk = (int)(P.K / KB), np = (nk + 1) & ~1;
  const int arow0 = wm * TM * 32, brow0 = wn * TN * 32;
  const rsrc_t none = make_rsrc(P.A, 0);
  Offs O;
#pragma unroll
  for (int u = 0; u < DA; ++u) {
    O.a[u] = dma_off(DA * wave + u, lane, P.lda);
    O.b[u] = dma_off(DA * wave + u, lane, P.ldb);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    O.fa[s] = (uint32_t)(arow0 * KB) + frag_off(s, lane);
    O.fb[s] = (uint32_t)(TILE + brow0 * KB) + frag_off(s, lane);
  }
  uint32_t vt = blockIdx.x;
  Tile c = tile_at(P, vt, ntiles, ntm, ntn);
  bool has_next = vt + step < ntiles;
  Tile n = has_next ? tile_at(P, vt + step, ntiles, ntm, ntn) : c;
  int turn = 0;

  // k-tile 0 and the first half of k-tile 1; no LDS reads come before this
  // barrier, so no release fence (it would wait for the later DMAs too)
  fetch<0>(st0, c, n, has_next, none, O, 0, nk, np, wave);
  fetch<1>(st0, c, n, has_next, none, O, 0, nk, np, wave);
  fetch<0>(st1, c, n, has_next, none, O, 1, nk, np, wave);
  wait_vm<4>();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  Frag F0, F1;
  read<0>(st0, O, F0);

  v16i acc[TN][TM];
  for (;;) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[j][i] = v16i{};
    // Read after the last k-tile, several barriers later; the buffers
    // alternate, so no wave still reads the one that is filled.
    fetch_factors<BM, BN, 8>(reinterpret_cast<uint8_t*>(sc[turn]), P, c.m0, c.n0, none, wave, lane);
    for (int k = 0; k < np; k += 2) {
      ktile(st0, st1, c, n, has_next, none, O, F0, F1, acc, k, nk, np, wave);
      ktile(st1, st0, c, n, has_next, none, O, F0, F1, acc, k + 1, nk, np, wave);
    }
    const float* f = sc[turn] + arow0;
    const float* g = sc[turn] + 256 + brow0;
#pragma unroll
    for (int i = 0; i < TM; ++i)
      put_pair<OUT>(acc[0][i], acc[1][i], staging + wave * kStage, Factors{f + 32 * i, g, g + 256}, P.C, P.ldc,
                    c.m0 + arow0 + 32 * i, c.n0 + brow0, P.M, P.N, lane);
    if (!has_next) break;
    vt += step;
    c = n;
    has_next = vt + step < ntiles;
    if (has_next) n = tile_at(P, vt + step, ntiles, ntm, ntn);
    turn ^= 1;
  }
  wait_vm<0>();  // the last (empty) DMAs still write LDS: let them land
}

// Compute units of the current device, queried once per device.
int cu_count() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int c = 0;
    n = (hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && c > 0) ? c : 256;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int OUT>
hipError_t launch(const Args& P, hipStream_t st) {
  const int64_t tiles = ((P.M + BM - 1) / BM) * ((P.N + BN - 1) / BN), ncu = cu_count();
  hipLaunchKernelGGL((gemm_kernel<OUT>), dim3((unsigned)(tiles < ncu ? tiles : ncu)), dim3(512), 0, st, P);
  return hipGetLastError();
}

}  // namespace big

// The DMA kernels: 16-byte rows, whole k-tiles, 32-bit offsets within a tile.
bool fast_ok(const Args& P) {
  return (((uintptr_t)P.A | (uintptr_t)P.B) & 15) == 0 && ((P.lda | P.ldb) & 15) == 0 && P.K % KB == 0 &&
         P.lda < (int64_t(1) << 23) && P.ldb < (int64_t(1) << 23);
}

// ----------------------------------------------------------- choice
typedef ring::G<2, 4, 1, 1, 6, 3> R64x128;
typedef ring::G<2, 4, 1, 1, 6, 3, 1> R64x128nt;
typedef ring::G<2, 4, 2, 1, 4, 4> R128x128;
typedef ring::G<2, 4, 2, 2, 3, 3> R128x256;

enum Kind { kFew, kFew2, k64x128, k128x128, k128x256, k256x256 };

struct Plan {
  Kind kind;
  int splits;
};

// From this size on a weight is counted as coming from HBM each time.
constexpr int64_t kPastCache = int64_t(1) << 27;

// The kernel and split with the least expected time, in us, by a model whose
// constants were fitted to the times of all of them at 278 sizes (1 to 3618
// tokens, weights of 45 KB to 320 MB; profiles/int8_gemm_candidates.csv has the
// times): its choice is within
// 0.7% of the fastest on average, 26% at worst (1983 x 3220 x 256, where C's bytes
// rule). Few tokens: a start, and for each round of 256 work-groups and 1024 k
// a time that grows with M; two groups of 16 rows of B to each load of A where
// that still gives most CUs a work-group (us, one group / two: 6144 x 4096, M = 4
// 7.5 / 7.0, M = 16 9.4 / 8.1, M = 64 20.3 / 14.3; 1024 x 4096, M = 16 5.4 /
// 7.4). Tiles: a start, and for each round of 256 tiles c a k-tile and an
// epilogue by the tile's area, but no faster than B from memory, the operands
// of all tiles through the caches, or the arithmetic; a split of k adds a launch
// and its partial sums. Measured, for example, at 1024 x 4096 (N x K) and 64
// tokens: few 11.0, 64 x 128 tiles 8.8, split in eight 8.1; at 6144 x 4096 and
// 512 tokens 22.8 / 16.3 / 22.8 / 39.9 for the four tiles, and at 1024 tokens
// 39.0 / 32.7 / 27.2 / 40.4.
float tiled_us(int64_t M, int64_t N, int64_t K, int bm, int bn, float c, int splits) {
  const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn), nk = K / KB;
  const int64_t rounds = (tiles * splits + 255) / 256;
  float t = (float)rounds * ((float)((nk + splits - 1) / splits) * c + 5.96f * (float)(bm * bn) / 65536.f);
  t = fmaxf(t, (float)N * K / (N * K >= kPastCache ? 8.32e6f : 9.38e6f));
  t = fmaxf(t, (float)(tiles * nk) * ((bm + bn) * KB) / 14.5e6f);
  t = fmaxf(t, (float)tiles * bm * bn * 2.f * K / 2.99e9f);
  return 2.17f + t + (splits > 1 ? 4.08f + (float)splits * M * N * 8.f / 2.38e6f : 0.f);
}

Plan plan_of(int64_t M, int64_t N, int64_t K) {
  Plan best{k64x128, 1};
  float t = tiled_us(M, N, K, 64, 128, 0.347f, 1);
  const auto offer = [&](Kind kind, int splits, float us) {
    if (us < t) {
      t = us;
      best = {kind, splits};
    }
  };
  if (M > 64) {  // (larger tiles would be rows past the end)
    offer(k128x128, 1, tiled_us(M, N, K, 128, 128, 0.462f, 1));
    offer(k128x256, 1, tiled_us(M, N, K, 128, 256, 0.823f, 1));
    offer(k256x256, 1, tiled_us(M, N, K, 256, 256, 1.01f, 1));
  }
  for (int s : {2, 3, 4, 6, 8}) {  // splits of at least 4 k-tiles
    if (s * 4 > K / KB || M > 4096) break;  // (rows are a grid dimension of the sums)
    offer(k64x128, s, tiled_us(M, N, K, 64, 128, 0.347f, s));
    if (M > 64 && s <= 4) offer(k128x128, s, tiled_us(M, N, K, 128, 128, 0.462f, s));
  }
  if (M <= 64)
    for (int g : {1, 2}) {
      const float rounds = (float)((N + 4096 * g - 1) / (4096 * g));
      const float per = g == 1 ? 0.449f + 0.0432f * M : 0.713f + 0.0552f * M;
      const float mem = (float)N * K / (N * K >= kPastCache ? 6.64e6f : 8.81e6f);
      offer(g == 1 ? kFew : kFew2, 1, 2.35f + fmaxf(rounds * K / 1024.f * per, mem));
    }
  return best;
}

template <int OUT>
hipError_t launch_out(const Args& P, void* ws, hipStream_t st) {
  if (!fast_ok(P)) return gen::launch<OUT>(P, st);
  const Plan plan = plan_of(P.M, P.N, P.K);
  switch (plan.kind) {
    case kFew:
      if (P.M <= 16) return few::launch<8, 4, 1, 1, OUT>(P, st);
      if (P.M <= 32) return few::launch<8, 4, 2, 1, OUT>(P, st);
      return few::launch<8, 2, 4, 1, OUT>(P, st);
    case kFew2:
      // few chunks of k leave 8 waves half idle (22741 x 512, M = 1: 4.4 against 5.3)
      if (P.M <= 16 && P.K <= 1024) return few::launch<4, 4, 1, 2, OUT>(P, st);
      if (P.M <= 16) return few::launch<8, 4, 1, 2, OUT>(P, st);
      if (P.M <= 32) return few::launch<4, 4, 2, 2, OUT>(P, st);
      return few::launch<4, 4, 4, 2, OUT>(P, st);
    case k64x128:
      // One tile-row reads B once. A large weight comes from HBM each time, and
      // past the caches is faster (28672 x 4096, M = 64: 23.8 against 28.3 us);
      // a smaller one may still lie in the 256 MB cache (6144 x 4096, used
      // again after two others of its size: 12.2 kept against 17.0).
      if (P.M <= 64 && P.N * P.K >= (int64_t(1) << 26))
        return ring::launch<R64x128nt, OUT>(P, plan.splits, ws, st);
      return ring::launch<R64x128, OUT>(P, plan.splits, ws, st);
    case k128x128: return ring::launch<R128x128, OUT>(P, plan.splits, ws, st);
    case k128x256: return ring::launch<R128x256, OUT>(P, plan.splits, ws, st);
    default: return big::launch<OUT>(P, st);
  }
}

}  // namespace

size_t int8_gemm_ws(int64_t M, int64_t N, int64_t K) {
  if (K % KB) return 0;
  const int splits = plan_of(M, N, K).splits;
  return splits > 1 ? (size_t)splits * (size_t)M * (size_t)N * sizeof(int) : 0;
}

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
