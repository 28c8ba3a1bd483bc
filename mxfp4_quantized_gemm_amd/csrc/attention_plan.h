// How paged attention's work is cut and where its tokens lie: integer arithmetic
// that the kernels (attention.hip) and a test on the CPU share.
#pragma once
#include <stdint.h>

#if defined(__HIPCC__)
#define MX_HD __host__ __device__ __forceinline__
#else
#define MX_HD inline
#endif

namespace mx {

constexpr int kTile = 32;        // tokens that a wave takes at a time
constexpr int kUnitWaves = 4;    // waves of a work-group
constexpr int kUnit = kTile * kUnitWaves;

// Tokens of a sequence that count, [first, n); units begin at `start`, a multiple of 16.
struct Span {
  int first, start, n, units;
};
// length: as given; most: what the table has room for (up to 2^31 - 16384);
// window: 0 for none.
MX_HD Span span_of(int length, int most, int window) {
  Span s;
  s.n = length < 0 ? 0 : length < most ? length : most;
  s.first = window > 0 && s.n > window ? s.n - window : 0;
  s.start = s.first & ~15;
  s.units = (s.n - s.start + kUnit - 1) / kUnit;
  return s;
}

// a / b of numbers that are not negative: 64 bits take the GPU five times as long.
MX_HD int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Of U units in a row, work-group w of W (W <= U) has [share(w), share(w + 1)).
MX_HD int64_t share(int64_t w, int64_t U, int64_t W) { return quotient(w * U, W); }
// The work-group that has unit u: the largest w with share(w) <= u, that is with w U
// / W < u + 1.
MX_HD int64_t owner(int64_t u, int64_t U, int64_t W) { return quotient((u + 1) * W - 1, U); }

// floor(x / d) = (x magic) >> shift for x < 2^27 and 1 <= d < 2^27: with d <= 2^s
// and d magic = 2^(27 + s) + e, e < d, the excess x e / (d 2^(27 + s)) is below
// 1 / d.
struct Divisor {
  uint32_t magic, shift;
};
MX_HD Divisor divisor_of(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return {(uint32_t)(((uint64_t(1) << (27 + s)) + d - 1) / d), 27 + s};
}
MX_HD uint32_t divided(uint32_t x, Divisor d) { return (uint32_t)(((uint64_t)x * d.magic) >> d.shift); }

}  // namespace mx
