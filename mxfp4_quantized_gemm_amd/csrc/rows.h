// Rows in the registers of a group of threads: loads and stores at any width and
// alignment, sums over the threads, int8 codes with one scale a row. Shared by
// the norms (norm.hip) and the operators on attention's heads (heads.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {
namespace {

constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <int T>
struct Type;  // bytes of a value
template <>
struct Type<kF32> {
  static constexpr int S = 4;
};
template <>
struct Type<kBF16> {
  static constexpr int S = 2;
};
template <>
struct Type<kF16> {
  static constexpr int S = 2;
};

// One value of type T at element i of p, as fp32 (exact), and back (RNE).
template <int T>
__device__ __forceinline__ float get1(const void* p, int64_t i) {
  if constexpr (T == kF32) return static_cast<const float*>(p)[i];
  if constexpr (T == kBF16)
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  if constexpr (T == kF16) return (float)static_cast<const _Float16*>(p)[i];
}

template <int T>
__device__ __forceinline__ float round_to(float v) {
  if constexpr (T == kBF16) return (float)(__bf16)v;
  if constexpr (T == kF16) return (float)(_Float16)v;
  return v;
}

template <int T>
__device__ __forceinline__ void put1(void* p, int64_t i, float v) {
  if constexpr (T == kF32) static_cast<float*>(p)[i] = v;
  if constexpr (T == kBF16) static_cast<__bf16*>(p)[i] = (__bf16)v;
  if constexpr (T == kF16) static_cast<_Float16*>(p)[i] = (_Float16)v;
}

// 16 bytes of type T <-> V = 16 / size values.
template <int T, int V>
__device__ __forceinline__ void unpack(u32x4 q, float (&v)[V]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if constexpr (T == kF32) {
      v[d] = __uint_as_float(q[d]);
    } else if constexpr (T == kBF16) {
      v[2 * d] = __uint_as_float(q[d] << 16);
      v[2 * d + 1] = __uint_as_float(q[d] & 0xffff0000u);
    } else {
      const uint32_t e = q[d];  // a bit_cast of the element itself reads element 0
      const f16x2 h = __builtin_bit_cast(f16x2, e);
      v[2 * d] = (float)h.x;
      v[2 * d + 1] = (float)h.y;
    }
  }
}

template <int T, int V>
__device__ __forceinline__ u32x4 pack(const float (&v)[V]) {
  u32x4 q;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if constexpr (T == kF32) {
      q[d] = __float_as_uint(v[d]);
    } else if constexpr (T == kBF16) {
      const bf16x2 h = {(__bf16)v[2 * d], (__bf16)v[2 * d + 1]};
      q[d] = __builtin_bit_cast(uint32_t, h);
    } else {
      const f16x2 h = {(_Float16)v[2 * d], (_Float16)v[2 * d + 1]};
      q[d] = __builtin_bit_cast(uint32_t, h);
    }
  }
  return q;
}

// Rows may start at any element (odd widths, slices): vectors are loaded and
// stored with the element's alignment, which gfx950 takes in one instruction
// (at most one cache line more).
typedef u32x4 u32x4_2 __attribute__((aligned(2)));
typedef u32x2 u32x2_1 __attribute__((aligned(1)));
typedef uint32_t u32_1 __attribute__((aligned(1)));

// q shifted down by n bytes (0 <= n < 16), zeros from above.
__device__ __forceinline__ u32x4 shift_down(u32x4 q, int n) {
  const uint64_t lo = (uint64_t)q.y << 32 | q.x, hi = (uint64_t)q.w << 32 | q.z;
  const int b = 8 * (n & 7);
  const uint64_t l = n & 8 ? hi : lo, h = n & 8 ? 0 : hi;
  const uint64_t a = l >> b | (b ? h << (64 - b) : 0), c = h >> b;
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)c, (uint32_t)(c >> 32)};
}

// A thread's share of a row: chunk i (i < R) holds the V = 16 bytes' worth of
// consecutive values from column (t + TPR i) V on, so that a load covers TPR V
// consecutive values. Columns past the row read as 0 and are not written.
// EVEN: the width is a multiple of V. If it is not, the chunk in which the row
// ends is loaded as the row's last 16 bytes and shifted, in the same
// instruction as the others (value by value it kept the whole row waiting:
// 1541 x 1111 fp32, backward 12.2 us), and stored value by value.
template <int T, bool EVEN, int TPR, int R>
struct Row {
  static constexpr int S = Type<T>::S, V = 16 / S;
  // The chunks as they lie in memory (EVEN), for a row that is wanted later.
  static __device__ __forceinline__ void load_raw(const void* p, int64_t row0, int cols, int t, u32x4 (&q)[R]) {
    static_assert(EVEN, "chunks of odd rows are shifted");
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (t + TPR * i) * V;
      q[i] = u32x4{0, 0, 0, 0};
      if (c < cols) q[i] = *reinterpret_cast<const u32x4_2*>(static_cast<const uint8_t*>(p) + (row0 + c) * S);
    }
  }
  static __device__ __forceinline__ void load(const void* p, int64_t row0, int cols, int t,
                                              float (&v)[R][V]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (t + TPR * i) * V;
      u32x4 q = {0, 0, 0, 0};
      if (EVEN) {
        if (c < cols)
          q = *reinterpret_cast<const u32x4_2*>(static_cast<const uint8_t*>(p) + (row0 + c) * S);
      } else if (cols >= V) {
        const int back = max(c + V - cols, 0);
        if (c < cols) {
          q = *reinterpret_cast<const u32x4_2*>(static_cast<const uint8_t*>(p) + (row0 + c - back) * S);
        }
        if (i == cols / V / TPR) q = shift_down(q, back * S & 15);  // (the same i for all threads)
      }
      unpack<T, V>(q, v[i]);
    }
    if (!EVEN && cols < V && t == 0) {
#pragma unroll
      for (int k = 0; k < V - 1; ++k)
        if (k < cols) v[0][k] = get1<T>(p, row0 + k);
    }
  }
  // PAST: not to stay in the L2 (a streaming store).
  template <bool PAST = false>
  static __device__ __forceinline__ void store(void* p, int64_t row0, int cols, int t,
                                               const float (&v)[R][V]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (t + TPR * i) * V;
      u32x4_2* const to = reinterpret_cast<u32x4_2*>(static_cast<uint8_t*>(p) + (row0 + c) * S);
      if (EVEN ? c < cols : c + V <= cols) {
        if constexpr (PAST)
          __builtin_nontemporal_store(pack<T, V>(v[i]), to);
        else
          *to = pack<T, V>(v[i]);
      }
    }
    if (!EVEN && t == cols / V % TPR) {
      const int c = cols / V * V;
      float e[V];
      tail(v, cols, e);
#pragma unroll
      for (int k = 0; k < V - 1; ++k)
        if (c + k < cols) put1<T>(p, row0 + c + k, e[k]);
    }
  }
  // The chunk in which the row ends, of the thread that has it.
  static __device__ __forceinline__ void tail(const float (&v)[R][V], int cols, float (&e)[V]) {
    const int at = cols / V / TPR;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      e[k] = v[0][k];
#pragma unroll
      for (int i = 1; i < R; ++i) e[k] = i == at ? v[i][k] : e[k];
    }
  }
};

// The weight's values of a thread's columns; its type is T or fp32 (wide).
template <int T, bool EVEN, int TPR, int R, int V>
__device__ __forceinline__ void load_weight(const void* w, bool wide, int cols, int t,
                                            float (&v)[R][V]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) v[i][k] = 1.f;
  } else if (T == kF32 || !wide) {
    Row<T, EVEN, TPR, R>::load(w, 0, cols, t, v);
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        const int c = (t + TPR * i) * V + k;
        const float* f = static_cast<const float*>(w);
        u32x4 q = {0, 0, 0, 0};
        if (c + 4 <= cols)
          q = *reinterpret_cast<const u32x4_2*>(f + c);
        else if (!EVEN)
#pragma unroll
          for (int e = 0; e < 3; ++e) q[e] = c + e < cols ? __float_as_uint(f[c + e]) : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][k + e] = __uint_as_float(q[e]);
      }
  }
}

// A value of another lane by a data-parallel move of its dwords (no LDS):
// P = 0, 1: lanes ^ 1, ^ 2; 2, 3: mirrored within 8 and within 16 lanes, which
// is as good as ^ 4 and ^ 8 once the smaller groups hold equal values.
template <int P, class X>
__device__ __forceinline__ X near_lane(X v) {
  constexpr int ctrl = P == 0 ? 0xb1 : P == 1 ? 0x4e : P == 2 ? 0x141 : 0x140;
  if constexpr (sizeof(X) == 8) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)b, ctrl, 0xf, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), ctrl, 0xf, 0xf, false);
    return __builtin_bit_cast(X, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(X, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), ctrl, 0xf, 0xf, false));
  }
}

// The two values of lanes l and l ^ 16 (W = 16) or l ^ 32 (W = 32), the same
// pair in both.
template <int W>
__device__ __forceinline__ void pair32(uint32_t v, uint32_t& a, uint32_t& b) {
  if constexpr (W == 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    a = s[0];
    b = s[1];
  } else {
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = s[0];
    b = s[1];
  }
}
template <int W, class X, class F>
__device__ __forceinline__ X far_lane(X v, F f) {
  uint32_t a, b;
  if constexpr (sizeof(X) == 8) {
    const uint64_t q = __builtin_bit_cast(uint64_t, v);
    uint32_t c, d;
    pair32<W>((uint32_t)q, a, b);
    pair32<W>((uint32_t)(q >> 32), c, d);
    return f(__builtin_bit_cast(X, (uint64_t)c << 32 | a), __builtin_bit_cast(X, (uint64_t)d << 32 | b));
  } else {
    pair32<W>(__builtin_bit_cast(uint32_t, v), a, b);
    return f(__builtin_bit_cast(X, a), __builtin_bit_cast(X, b));
  }
}

// Sum (or integer max) over the TPR threads of a row; every thread gets it.
// `red` holds one slot per wave; each call uses slots of its own, so one
// barrier is enough. The order is fixed.
template <int TPR, class X, class F>
__device__ __forceinline__ X reduce_row(X v, X* red, int t, F f) {
  v = f(v, near_lane<0>(v));
  v = f(v, near_lane<1>(v));
  v = f(v, near_lane<2>(v));
  if constexpr (TPR >= 16) v = f(v, near_lane<3>(v));
  if constexpr (TPR >= 32) v = far_lane<16>(v, f);
  if constexpr (TPR >= 64) v = far_lane<32>(v, f);
  if constexpr (TPR > 64) {
    if ((t & 63) == 0) red[t >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v = f(v, red[w]);
  }
  return v;
}

// 1 / sqrt(x) for x >= 0 in fp64 to about 2^-52: the hardware's estimate and two
// Newton steps, because every row waits for it. With the lane moves above, in
// place of a division, a root and shuffles through LDS, a call takes 2.8 us
// instead of 3.1 at 1 x 4096, 6.4 instead of 7.2 at 1541 x 1111 and 40.4 instead
// of 41.3 at 8192 x 4096 (in a graph, bf16 with a residual), the bits unchanged.
// 0, infinity and NaN as the estimate has them (inf, 0, NaN).
__device__ __forceinline__ double rsqrt64(double x) {
  double r = __builtin_amdgcn_rsq(x);
  if (x > 0.0 && x < __builtin_inf()) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const double e = fma(-x * r, r, 1.0);
      r = fma(r * 0.5, e, r);
    }
  }
  return r;
}

__device__ __forceinline__ double add64(double a, double b) { return a + b; }
__device__ __forceinline__ float add32(float a, float b) { return a + b; }
__device__ __forceinline__ uint32_t max32(uint32_t a, uint32_t b) { return max(a, b); }

// Codes and scale of a row of values. 127 / a overflows for a below 2^-120,
// so a row of small values is first scaled by 2^64, which is exact.
template <int T, bool EVEN, int TPR, int R, int V>
__device__ __forceinline__ void write_codes(const float (&v)[R][V], uint32_t* red, uint8_t* q,
                                            int64_t ld, float* scale, int cols, int t) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) m = max(m, __float_as_uint(v[i][k]) & 0x7fffffffu);
  m = reduce_row<TPR>(m, red, t, max32);
  const bool bad = m >= 0x7f800000u;
  const float a = __uint_as_float(m);
  const float up = a < 0x1p-64f ? 0x1p64f : 1.f;
  const float inv = (bad || m == 0) ? 0.f : 127.f / (a * up);
  if (t == 0) *scale = bad ? __uint_as_float(0x7fc00000u) : a / 127.f;
  const auto code = [&](float x) { return bad ? 0u : (uint32_t)(int)rintf(x * up * inv) & 255u; };
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int c = (t + TPR * i) * V;
    uint32_t d[V / 4] = {};
#pragma unroll
    for (int k = 0; k < V; ++k) d[k / 4] |= code(v[i][k]) << (8 * (k & 3));
    if (EVEN ? c < cols : c + V <= cols) {
      if constexpr (V == 4)
        *reinterpret_cast<u32_1*>(q + c) = d[0];
      else
        *reinterpret_cast<u32x2_1*>(q + c) = u32x2{d[0], d[1]};
    }
  }
  if (!EVEN && t == cols / V % TPR) {
    const int c = cols / V * V;
    float e[V];
    Row<T, EVEN, TPR, R>::tail(v, cols, e);
#pragma unroll
    for (int k = 0; k < V - 1; ++k)
      if (c + k < cols) q[c + k] = (uint8_t)code(e[k]);
  }
  // zero codes up to a multiple of 128 columns, as far as the pitch has them
  const int end = (int)min((int64_t)(cols + 127) / 128 * 128, ld);
  for (int c = cols + t; c < end; c += TPR) q[c] = 0;
}

}  // namespace
}  // namespace mx
