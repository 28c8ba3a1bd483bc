// Operators on attention's heads for gfx950 (MI355X): the norm of each head of
// queries and keys with their rotation, its gradient, the same with keys and
// values written to an int8 cache, and the cache read back.
//
//   u = x r, r = 1 / sqrt(mean(x^2) + eps)    over a head's dim values
//   z = u w                                   (x itself without a norm)
//   y = z_i cos t - z_j sin t at i, z_j cos t + z_i sin t at j, for each
//       rotated pair (i, j); t = position * frequency; z past the pairs
//   gradient: dz is dy turned by -t, g = dz w,
//       dx = r (g - u mean(g u)),  dw = sum over tokens and heads of dz u
//   cache: codes and scale of y (keys) and of x (values) as int8 rows
//
// One pass over HBM: a head's values stay in the registers of 8, 16 or 32
// threads (8 values each), several heads a wave. The cosines and sines of a
// token are computed once by its work-group, and serve all its heads from
// LDS. Results leave by streaming stores: what reads them next runs on all XCDs, and
// finds little in this one's L2 (2048 tokens of 32 + 8 heads of 128, bf16: 11.1 us, 12.7
// by ordinary stores; read back, 32768 tokens: 34.3, 37.9). Angles are taken in fp64,
// where position * frequency and the whole turns are exact to 2^-53 of the angle; the
// rest of at most an eighth of a turn goes to fp32 and a Taylor series. Squares are
// summed in fp64 as in the norm of whole rows (norm.hip), everything else is in fp32,
// rounded once at the end.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "rows.h"

namespace mx {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kE = 8;  // values a thread

struct Angles {
  const int64_t* pos;  // [axes][tokens]
  const double* freq;
  int64_t tokens;
  int pairs, half;     // half: distance of a pair's values (1 or pairs)
  int ends[4];         // first pair behind each axis
};

// cos and sin of a * f, a whole number times radians. The product is brought
// to quarter turns; what is left of at most an eighth of a turn, x in
// [-pi/4, pi/4], has a relative error of 2^-24 and its series end at x^9 and
// x^10 (the next terms are below 2^-28 of the sum). A factor is then within 1.2 2^-24 of
// the exact one (at 4 million angles), where one rounded from fp64 is within 2^-25.
__device__ __forceinline__ void cos_sin(int64_t a, double f, float& c, float& s) {
  const double q = (double)a * f * 0.63661977236758134308;  // quarter turns
  const double n = rint(q);
  const float x = (float)((q - n) * 1.57079632679489661923);
  const float v = x * x;
  float ps = fmaf(v, 2.7557319224e-6f, -1.9841269841e-4f);
  ps = fmaf(v, ps, 8.3333333333e-3f);
  ps = fmaf(v, ps, -1.6666666667e-1f);
  ps = fmaf(x * v, ps, x);
  float pc = fmaf(v, -2.7557319224e-7f, 2.4801587302e-5f);
  pc = fmaf(v, pc, -1.3888888889e-3f);
  pc = fmaf(v, pc, 4.1666666667e-2f);
  pc = fmaf(v, pc, -0.5f);
  pc = fmaf(v, pc, 1.f);
  // n modulo 4 in fp64 (n may be past 2^63): sin turns into cos every quarter
  const int k = (int)(n - 4.0 * floor(n * 0.25));
  const float so = k & 1 ? pc : ps, co = k & 1 ? ps : pc;
  s = k & 2 ? -so : so;
  c = (k == 1 || k == 2) ? -co : co;
}

// For each of a token's dim columns the factors of y_i = z_i cs[i] + z_j sn[i];
// `n` tokens from `token` on, [n][256] each. All threads of the work-group.
__device__ __forceinline__ void turn_table(const Angles& A, int64_t token, int n, float* cs, float* sn) {
  for (int i = threadIdx.x; i < n * A.pairs; i += kThreads) {
    const int k = i / A.pairs, p = i - k * A.pairs;
    const int axis = (p >= A.ends[0]) + (p >= A.ends[1]) + (p >= A.ends[2]);
    float c, s;
    cos_sin(A.pos[axis * A.tokens + token + k], A.freq[p], c, s);
    const int at = k * (int)kHeadMax + (A.half == 1 ? 2 * p : p);
    cs[at] = cs[at + A.half] = c;
    sn[at] = -s;
    sn[at + A.half] = s;
  }
}

// The two weights as fp32 in LDS ([2][256], 1 where there is none), from where each row
// takes its columns': kept in registers they cost 16 of each thread's. Zeros past the
// head, for the threads whose columns those are: what lies in the LDS may be NaN, and
// its product with their zeros would be. All threads.
__device__ __forceinline__ void weight_table(const void* qw, const void* kw, int dim, int type, float* w) {
  for (int c = threadIdx.x; c < (int)kHeadMax; c += kThreads) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const void* p = k ? kw : qw;
      w[k * (int)kHeadMax + c] = c >= dim        ? 0.f
                                 : p == nullptr  ? 1.f
                                 : type == kF32  ? get1<kF32>(p, c)
                                 : type == kBF16 ? get1<kBF16>(p, c)
                                                 : get1<kF16>(p, c);
    }
  }
}

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The columns of a thread: chunk i holds V from (t + TPR i) V on, as Row has them.
template <int T, bool EVEN, int TPR>
struct Lanes {
  static constexpr int S = Type<T>::S, V = 16 / S, R = kE / V;
  typedef Row<T, EVEN, TPR, R> X;
  float c[R][V], s[R][V];  // the token's factors for these columns

  // sign 1 to turn, -1 to turn back; columns past the pairs keep their value: factors 1 and 0
  __device__ __forceinline__ void factors(const float* cs, const float* sn, int rot, float sign, int t) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int at = (t + TPR * i) * V + k;
        c[i][k] = at < rot ? cs[at] : 1.f;
        s[i][k] = at < rot ? sign * sn[at] : 0.f;
      }
  }

  // A table's values of the columns, up to its 256.
  static __device__ __forceinline__ void columns(const float* w, int t, float (&v)[R][V]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        const float4 f = *reinterpret_cast<const float4*>(w + (t + TPR * i) * V + k);
        v[i][k] = f.x;
        v[i][k + 1] = f.y;
        v[i][k + 2] = f.z;
        v[i][k + 3] = f.w;
      }
  }

  // The value of the thread TPR / 2 away.
  static __device__ __forceinline__ float opposite(float v, int t) {
    const int b = __builtin_bit_cast(int, v);
    if constexpr (TPR == 8) {  // from 4 above in the even fours, 4 below in the odd ones
      const int a = __builtin_amdgcn_update_dpp(0, b, 0x104, 0xf, 0x5, false);
      return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(a, b, 0x114, 0xf, 0xa, false));
    } else if constexpr (TPR == 16) {  // rotated by 8
      return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(b, 0x128, 0xf, 0xf, false));
    } else {
      uint32_t lo, hi;
      pair32<16>((uint32_t)b, lo, hi);
      return __uint_as_float(t < 16 ? hi : lo);
    }
  }

  // z turned. A pair's other value comes from
  // the same thread (neighbours; fp32 halves of a whole row), from the thread opposite
  // (16-bit halves of a whole row), or through `meet`, which holds this row of the wave.
  __device__ __forceinline__ void turn(float (&z)[R][V], float* meet, int half, int rot, int t) const {
    float o[R][V];
    // (a value, not a place: else the compiler chooses between z and LDS by address,
    // and z goes to memory)
    const auto value = [](float v) {
      asm("" : "+v"(v));
      return v;
    };
    if (half == 1) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) o[i][k] = value(z[i][k ^ 1]);
    } else if (half == TPR * kE / 2) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) o[i][k] = R == 2 ? value(z[R - 1 - i][k]) : opposite(z[i][k], t);
    } else {
      wave_sync();  // the last row's reads are done
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; k += 4)
          *reinterpret_cast<float4*>(meet + (t + TPR * i) * V + k) =
              float4{z[i][k], z[i][k + 1], z[i][k + 2], z[i][k + 3]};
      wave_sync();
      if (half % V == 0) {  // a chunk's other values lie side by side
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int at = (t + TPR * i) * V, to = at < half ? at + half : at < rot ? at - half : at;
#pragma unroll
          for (int k = 0; k < V; k += 4) {
            const float4 f = *reinterpret_cast<const float4*>(meet + to + k);
            o[i][k] = f.x;
            o[i][k + 1] = f.y;
            o[i][k + 2] = f.z;
            o[i][k + 3] = f.w;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const int at = (t + TPR * i) * V + k;
            o[i][k] = meet[at < half ? at + half : at < rot ? at - half : at];
          }
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        // an infinity behind the pairs is not multiplied by zero
        const int at = (t + TPR * i) * V + k;
        z[i][k] = at < rot ? fmaf(z[i][k], c[i][k], s[i][k] * o[i][k]) : z[i][k];
      }
  }
};

// 1 / sqrt(mean(x^2) + eps) of the row.
template <int TPR, int R, int V>
__device__ __forceinline__ float factor(const float (&v)[R][V], double inv, float eps) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) s = fma((double)v[i][k], (double)v[i][k], s);
  s = reduce_row<TPR>(s, (double*)nullptr, 0, add64);
  return (float)rsqrt64(s * inv + (double)eps);
}

// -------------------------------------------------------------- forward
struct HeadsArgs {
  Heads q, k, v;  // v.heads is 0 without a cache
  void *qo, *ko;
  float* rstd;  // [tokens][q heads + k heads], or NULL
  const void *qw, *kw;
  Angles a;
  double inv_dim;
  int64_t first, tokens;  // of this launch: [first, tokens)
  int dim, rot;
  int tpg, parts;         // tokens a work-group: 4, 2, or 1 and it has one of `parts` of its heads
  float eps;
  bool norm, wide;
  // the cache: codes [pages][heads][page][pitch]
  uint8_t *kc, *vc;
  float *ks, *vs;
  const int64_t* slots;
  int64_t capacity;
  int page, pitch;
};

// A wave's rows at a time are of one kind (queries, keys or values): item i is
// one of the queries', then of the keys', then of the values'.
template <int RPW>
struct Items {
  int q, k, all;
  __device__ __forceinline__ Items(const Heads& hq, const Heads& hk, int64_t v) {
    q = ((int)hq.heads + RPW - 1) / RPW;
    k = q + ((int)hk.heads + RPW - 1) / RPW;
    all = k + ((int)v + RPW - 1) / RPW;
  }
  __device__ __forceinline__ int kind(int i) const { return i < q ? 0 : i < k ? 1 : 2; }
  // head of the wave's row `sub`, which may be past the last
  __device__ __forceinline__ int head(int i, int sub) const {
    return (i - (i < q ? 0 : i < k ? q : k)) * RPW + sub;
  }
};

// Loads first, what waits for them last: the first rows, the weights and the
// slots are on their way while the token's cosines and sines are made, and a row's
// loads while the one before is worked on. (8192 tokens of 32 + 8 heads of 128,
// bf16: 32 us for 168 MB; without the latter, and with a pair's other value through LDS, 48.
// Waves a SIMD, with the cache: 8 instead of 6 take 46.8 us, not 49, for 8192 tokens, but 7.4,
// not 6.9, for 256.)
template <int T, bool EVEN, int TPR, bool CACHE>
__global__ __launch_bounds__(kThreads, CACHE ? 6 : T == kF32 ? 7 : 8) void heads_kernel(HeadsArgs A) {
  typedef Lanes<T, EVEN, TPR> L;
  constexpr int R = L::R, V = L::V, RPW = 64 / TPR;
  __shared__ float cs[kWaves * kHeadMax], sn[kWaves * kHeadMax];
  alignas(16) __shared__ float meet_all[kWaves * 64 * kE];
  alignas(16) __shared__ float weights[2 * kHeadMax];
  __shared__ int again[kWaves];
  static_assert(__alignof__(meet_all) >= 16 && __alignof__(weights) >= 16, "they are accessed 16 bytes at a time");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, t = lane % TPR, sub = lane / TPR;
  const int64_t group = blockIdx.x / A.parts;
  const int part = blockIdx.x - (int)group * A.parts;
  const int64_t token0 = A.first + group * A.tpg;
  const int n = (int)min((int64_t)A.tpg, A.tokens - token0);
  const int wpt = kWaves / A.tpg, mine = wave / wpt;  // waves a token; this wave's token of the work-group's
  const int64_t token = token0 + (mine < n ? mine : 0);
  const Items<RPW> items(A.q, A.k, A.v.heads);
  int item = part * wpt + wave % wpt;
  const int stride = wpt * A.parts;
  // rows past the last of their kind are the last one's again, and not stored
  const auto at = [&](int i) {
    const int kind = items.kind(i);
    const Heads& x = kind == 0 ? A.q : kind == 1 ? A.k : A.v;
    return token * x.ts + min(items.head(i, sub), (int)x.heads - 1) * x.hs;
  };
  const auto from = [&](int i) { return i < items.q ? A.q.p : i < items.k ? A.k.p : A.v.p; };
  u32x4 rows[R];  // the next ones
  const auto load = [&](int i) {  // never under a condition, after which all loads would be waited for
    i = min(i, items.all - 1);
    if constexpr (EVEN) L::X::load_raw(from(i), at(i), A.dim, t, rows);
  };
  load(item);
  if (A.norm) weight_table(A.qw, A.kw, A.dim, A.wide ? kF32 : T, weights);
  int64_t cell = -1;  // the token's row of head 0 in the cache
  if constexpr (CACHE) {
    // of tokens with the same slot the last one is written: work-groups look at the
    // slots behind theirs (a launch has few tokens, see below), two a load, four loads at
    // once; what a token without a slot finds does not matter
    int64_t slot[kWaves];
#pragma unroll
    for (int k = 0; k < kWaves; ++k) slot[k] = A.slots[token0 + min(k, n - 1)];
    uint64_t same[kWaves] = {};
    typedef int64_t i64x2 __attribute__((ext_vector_type(2), aligned(8)));
    for (int64_t base = token0 + n; base < A.tokens; base += 8 * kThreads) {
      i64x2 s[4];
      bool both[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // past the end: the last token, with one before it that does not count
        const int64_t i = base + 2 * (kThreads * e + (int)threadIdx.x);
        both[e] = i < A.tokens - 1;
        s[e] = *reinterpret_cast<const i64x2*>(A.slots + min(i, A.tokens - 2));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int k = 0; k < kWaves; ++k)
          same[k] |= __ballot(s[e].y == slot[k]) | __ballot(both[e] && s[e].x == slot[k]);
    }
    int found = 0;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      found |= same[k] ? 1 << k : 0;
#pragma unroll
      for (int b = k + 1; b < kWaves; ++b) found |= b < n && slot[b] == slot[k] ? 1 << k : 0;
    }
    if (lane == 0) again[wave] = found;
    int64_t s = slot[0];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) s = mine == k ? slot[k] : s;
    if (s >= 0 && s < A.capacity) {
      const uint32_t u = (uint32_t)s, p = u / (uint32_t)A.page;
      cell = (int64_t)p * A.k.heads * A.page + (u - p * (uint32_t)A.page);
    }
  }
  turn_table(A.a, token0, n, cs, sn);
  __syncthreads();
  if (mine >= n) return;  // no barrier of the work-group follows
  if constexpr (CACHE) {
    if ((again[0] | again[1] | again[2] | again[3]) >> mine & 1) cell = -1;
  }
  L f;
  float* const meet = meet_all + (wave * 64 + sub * TPR) * kE;
  f.factors(cs + mine * kHeadMax, sn + mine * kHeadMax, A.rot, 1.f, t);
  for (; item < items.all; item += stride) {
    float v[R][V];
    if constexpr (EVEN) {
#pragma unroll
      for (int i = 0; i < R; ++i) unpack<T, V>(rows[i], v[i]);
      load(item + stride);
    } else {
      L::X::load(from(item), at(item), A.dim, t, v);
    }
    const int kind = items.kind(item), h = items.head(item, sub);
    const bool real = h < (int)(kind == 0 ? A.q.heads : A.k.heads);  // whole rows of threads
    if (kind < 2) {
      if (A.norm) {
        float w[R][V];
        L::columns(weights + kind * (int)kHeadMax, t, w);
        const float r = factor<TPR>(v, A.inv_dim, A.eps);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) v[i][k] = v[i][k] * r * w[i][k];
        if (!CACHE && A.rstd != nullptr && t == 0 && real)
          A.rstd[token * (A.q.heads + A.k.heads) + (kind == 0 ? 0 : A.q.heads) + h] = r;
      }
      if (A.rot > 0) f.turn(v, meet, A.a.half, A.rot, t);
    }
    if (!real) continue;
    if (kind == 0) {
      L::X::template store<true>(A.qo, (token * A.q.heads + h) * A.dim, A.dim, t, v);
    } else if constexpr (CACHE) {
      if (cell >= 0) {
        const int64_t to = cell + (int64_t)h * A.page;
        write_codes<T, EVEN, TPR, R>(v, nullptr, (kind == 1 ? A.kc : A.vc) + to * A.pitch, A.pitch,
                                     (kind == 1 ? A.ks : A.vs) + to, A.dim, t);
      }
    } else {
      L::X::template store<true>(A.ko, (token * A.k.heads + h) * A.dim, A.dim, t, v);
    }
  }
}

// ------------------------------------------------------------- gradient
struct HeadsBwdArgs {
  Heads q, k, dq, dk;
  void *qo, *ko;
  const float* rstd;  // as the forward pass wrote them; NULL: no norm
  const void *qw, *kw;
  float* part;  // [gridDim.x][2][dim] partial sums of the weights' gradients, or NULL
  Angles a;
  float inv_dim;
  int64_t tokens;
  int dim, rot, tpg, parts;
  bool norm, wide;
};

// Work-groups walk the tokens in turn; the weights' gradients are summed in
// registers, then over a work-group in LDS, then over work-groups by a second
// kernel: a fixed order, no atomics.
template <int T, bool EVEN, int TPR>
__global__ __launch_bounds__(kThreads, T == kF32 ? 3 : 4) void heads_bwd_kernel(HeadsBwdArgs A) {
  typedef Lanes<T, EVEN, TPR> L;
  constexpr int R = L::R, V = L::V, RPW = 64 / TPR;
  __shared__ float cs[kWaves * kHeadMax], sn[kWaves * kHeadMax];
  alignas(16) __shared__ float meet_all[kWaves * 64 * kE];
  alignas(16) __shared__ float weights[2 * kHeadMax];
  static_assert(__alignof__(meet_all) >= 16 && __alignof__(weights) >= 16, "they are accessed 16 bytes at a time");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, t = lane % TPR, sub = lane / TPR;
  const int wpt = kWaves / A.tpg, mine = wave / wpt;
  const Items<RPW> items(A.q, A.k, 0);
  const int stride = wpt * A.parts;
  float* const meet = meet_all + (wave * 64 + sub * TPR) * kE;
  float dqw[R][V] = {}, dkw[R][V] = {};
  if (A.norm) weight_table(A.qw, A.kw, A.dim, A.wide ? kF32 : T, weights);
  const int64_t groups = (A.tokens + A.tpg - 1) / A.tpg * A.parts;
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t token0 = g / A.parts * A.tpg;
    const int part = (int)(g % A.parts);
    const int n = (int)min((int64_t)A.tpg, A.tokens - token0);
    const int64_t token = token0 + (mine < n ? mine : 0);
    int item = mine >= n ? items.all : part * wpt + wave % wpt;
    const auto at = [&](const Heads& x, int i) {
      return token * x.ts + min(items.head(i, sub), (int)x.heads - 1) * x.hs;
    };
    struct Next {  // rows that are on their way
      u32x4 x[R], y[R];
      float r;
    } next[2];
    const auto load = [&](int i, Next& to) {
      i = min(i, items.all - 1);
      const bool isq = i < items.q;
      const Heads &x = isq ? A.q : A.k, &y = isq ? A.dq : A.dk;
      if constexpr (EVEN) {
        L::X::load_raw(y.p, at(y, i), A.dim, t, to.y);
        if (A.norm) L::X::load_raw(x.p, at(x, i), A.dim, t, to.x);
      }
      if (A.norm)
        to.r = A.rstd[token * (A.q.heads + A.k.heads) + (isq ? 0 : A.q.heads) +
                      min(items.head(i, sub), (int)x.heads - 1)];
    };
    if (item < items.all) {
      load(item, next[0]);
      load(item + stride, next[1]);
    }
    __syncthreads();  // the last tokens' factors are read
    turn_table(A.a, token0, n, cs, sn);
    __syncthreads();
    L f;
    f.factors(cs + mine * kHeadMax, sn + mine * kHeadMax, A.rot, -1.f, t);
    const auto work = [&](int item, Next& rows) {
      const bool isq = item < items.q;
      const int h = items.head(item, sub);
      const bool real = h < (int)(isq ? A.q.heads : A.k.heads);
      float u[R][V], d[R][V];
      const float r = rows.r;
      if constexpr (EVEN) {
#pragma unroll
        for (int i = 0; i < R; ++i) unpack<T, V>(rows.y[i], d[i]);
        if (A.norm) {
#pragma unroll
          for (int i = 0; i < R; ++i) unpack<T, V>(rows.x[i], u[i]);
        }
      } else {
        const Heads &x = isq ? A.q : A.k, &y = isq ? A.dq : A.dk;
        L::X::load(y.p, at(y, item), A.dim, t, d);
        if (A.norm) L::X::load(x.p, at(x, item), A.dim, t, u);
      }
      load(item + 2 * stride, rows);
      if (!real) {  // a row again: nothing for the weight
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) d[i][k] = 0.f;
      }
      if (A.rot > 0) f.turn(d, meet, A.a.half, A.rot, t);
      if (A.norm) {
        float s = 0.f, w[R][V];
        L::columns(weights + (isq ? 0 : (int)kHeadMax), t, w);
        const auto step = [&](float (&dw)[R][V]) {
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
              u[i][k] *= r;
              dw[i][k] = fmaf(d[i][k], u[i][k], dw[i][k]);
              d[i][k] *= w[i][k];
              s = fmaf(d[i][k], u[i][k], s);
            }
        };
        if (isq) {
          step(dqw);
        } else {
          step(dkw);
        }
        s = reduce_row<TPR>(s, (float*)nullptr, 0, add32) * A.inv_dim;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) d[i][k] = r * (d[i][k] - u[i][k] * s);
      }
      if (real)
        L::X::template store<true>(isq ? A.qo : A.ko, (token * (isq ? A.q.heads : A.k.heads) + h) * A.dim, A.dim,
                                   t, d);
    };
    for (; item < items.all; item += 2 * stride) {
      work(item, next[0]);
      if (item + stride >= items.all) break;
      work(item + stride, next[1]);
    }
  }
  if (A.part == nullptr) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) meet[(t + TPR * i) * V + k] = which ? dkw[i][k] : dqw[i][k];
    __syncthreads();
    for (int c = threadIdx.x; c < A.dim; c += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < kWaves * RPW; ++r) s += meet_all[r * TPR * kE + c];
      A.part[((int64_t)blockIdx.x * 2 + which) * A.dim + c] = s;
    }
  }
}

// dw[c] = sum over the parts p of part[p][c], c < 2 dim (queries' weight, then
// keys'): 64 quarter-waves of a work-group take every 64th part of 16 columns.
template <int T>
__global__ __launch_bounds__(1024) void heads_dw_kernel(const float* part, int parts, int dim, void* dq,
                                                        void* dk) {
  __shared__ float red[64][17];
  const int lane = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + lane;
  float s = 0.f;
  if (c < 2 * dim) {
#pragma unroll 16
    for (int p = q; p < parts; p += 64) s += part[(int64_t)p * 2 * dim + c];
  }
  red[q][lane] = s;
  __syncthreads();
  if (q < 4) {  // one wave: four sums of 16, then theirs
    s = red[q][lane];
#pragma unroll
    for (int k = 1; k < 16; ++k) s += red[q + 4 * k][lane];
    s = far_lane<16>(s, add32);
    s = far_lane<32>(s, add32);
    if (q == 0 && c < 2 * dim) {
      if (c < dim) {
        if (dq != nullptr) put1<T>(dq, c, s);
      } else if (dk != nullptr) {
        put1<T>(dk, c - dim, s);
      }
    }
  }
}

// ------------------------------------------------------------ read back
struct ReadArgs {
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int64_t* slots;
  void *k, *v;
  int64_t tokens, capacity;
  int dim, heads, page, pitch;
};

// y = code * scale, rounded once. A slot outside the cache reads as zeros. (A code
// is converted as the byte code + 128: a signed one's conversion takes three times as long.)
template <int T, bool EVEN, int TPR, int ROWS>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs A) {
  constexpr int V = 16 / Type<T>::S, R = kE / V;
  const int t = threadIdx.x % TPR;
  const uint32_t each = 2 * A.heads, rows = (uint32_t)A.tokens * each;  // below 2^31, see below
  const uint32_t row0 = blockIdx.x * (ROWS * (kThreads / TPR)) + threadIdx.x / TPR;
  // several rows a thread, all their slots and then all their codes on the way at once
  int64_t slot[ROWS], to[ROWS];
  uint32_t h[ROWS];
#pragma unroll
  for (int n = 0; n < ROWS; ++n) {
    const uint32_t row = min(row0 + n * (kThreads / TPR), rows - 1), token = row / each, at = row - token * each;
    slot[n] = A.slots[token];
    h[n] = at;
    to[n] = ((int64_t)token * A.heads + (at >> 1)) * A.dim;
  }
  uint32_t d[ROWS][R][V / 4];
  float scale[ROWS];
#pragma unroll
  for (int n = 0; n < ROWS; ++n) {
    const bool in = slot[n] >= 0 && slot[n] < A.capacity;
    const uint32_t s = in ? (uint32_t)slot[n] : 0, p = s / (uint32_t)A.page;
    const int64_t from = ((int64_t)p * A.heads + (h[n] >> 1)) * A.page + (s - p * (uint32_t)A.page);
    const uint8_t* q = (h[n] & 1 ? A.vc : A.kc) + from * A.pitch;
    scale[n] = (h[n] & 1 ? A.vs : A.ks)[from];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = min((t + TPR * i) * V, A.pitch - V);  // the pitch is a multiple of 64: whole words
      if constexpr (V == 4) {
        d[n][i][0] = *reinterpret_cast<const uint32_t*>(q + c);
      } else {
        const u32x2 e = *reinterpret_cast<const u32x2*>(q + c);
        d[n][i][0] = e.x;
        d[n][i][1] = e.y;
      }
    }
    if (!in) {  // zeros, whatever the scale
      scale[n] = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V / 4; ++k) d[n][i][k] = 0;
    }
  }
#pragma unroll
  for (int n = 0; n < ROWS; ++n) {
    if (row0 + n * (kThreads / TPR) >= rows) return;
    float v[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k)
        v[i][k] = ((float)((d[n][i][k / 4] ^ 0x80808080u) >> (8 * (k & 3)) & 255u) - 128.f) * scale[n];
    Row<T, EVEN, TPR, R>::template store<true>(h[n] & 1 ? A.v : A.k, to[n], A.dim, t, v);
  }
}

// -------------------------------------------------------------- launches
Angles angles(const mxfp4_rotation& r, int64_t tokens) {
  Angles a{r.positions, r.frequencies, tokens, (int)r.pairs, r.interleaved ? 1 : (int)r.pairs, {}};
  int64_t end = 0;
  for (int i = 0; i < 4; ++i) {
    end += i < r.axes ? r.axis_pairs[i] : 0;
    a.ends[i] = (int)end;
  }
  if (r.pairs == 1) a.half = 1;
  return a;
}

// Calls f with a kernel for the width: Kernel<T, EVEN, TPR>.
template <int T, bool EVEN, class F>
hipError_t by_width(int64_t dim, F f) {
  if (dim <= 64) return f.template go<T, EVEN, 8>();
  if (dim <= 128) return f.template go<T, EVEN, 16>();
  return f.template go<T, EVEN, 32>();
}
template <class F>
hipError_t by_type(int dtype, int64_t dim, F f) {
  switch (dtype) {
    case kBF16: return dim % 8 ? by_width<kBF16, false>(dim, f) : by_width<kBF16, true>(dim, f);
    case kF16: return dim % 8 ? by_width<kF16, false>(dim, f) : by_width<kF16, true>(dim, f);
    default: return dim % 4 ? by_width<kF32, false>(dim, f) : by_width<kF32, true>(dim, f);
  }
}

// Work-groups: of as many tokens as leave about 2048 of them, which is how many
// the GPU holds; below that one token each, or a part of its heads (a wave's rows at a
// time for each wave) for up to 512 work-groups. A cache's work-group compares all slots
// with its own whatever their number, and has four tokens earlier, with few heads
// earlier still. (32 + 8 heads of 128, bf16, one | two | four tokens each, us: 2048
// tokens 11.4 | 11.4 | 13.2, with gradient 34.3 | 31.3 | 34.3, with the cache 17.5 | 14.9
// | 17.2; 4096 tokens 19.6 | 16.7 | 18.0, with the cache 29.5 | 24.3 | 23.7; 8192 tokens
// 38.8 | 34.7 | 33.4, with the cache 66.5 | 51.0 | 48.6; 3001 tokens of 5 heads of 96
// written 15.1 | 10.9 | 9.4.)
struct Shape {
  int tpg, parts;
  int64_t groups;
};
Shape shape_of(int64_t tokens, int64_t heads, int64_t dim, bool cache = false) {
  const int64_t four = !cache ? 8192 : heads > 16 ? 4096 : 2048;
  const int tpg = tokens >= four ? 4 : tokens >= 2048 ? 2 : 1;
  if (tpg > 1) return {tpg, 1, (tokens + tpg - 1) / tpg};
  const int64_t rpw = dim <= 64 ? 8 : dim <= 128 ? 4 : 2, most = (heads + kWaves * rpw - 1) / (kWaves * rpw);
  int64_t parts = tokens > 0 ? 512 / tokens : 1;
  if (parts > most) parts = most;
  if (parts < 1) parts = 1;
  return {1, (int)parts, tokens * parts};
}

struct Forward {
  HeadsArgs A;
  hipStream_t st;
  template <int T, bool EVEN, int TPR>
  hipError_t go() const {
    const dim3 grid((unsigned)((A.tokens - A.first + A.tpg - 1) / A.tpg * A.parts));
    if (A.slots)
      hipLaunchKernelGGL((heads_kernel<T, EVEN, TPR, true>), grid, dim3(kThreads), 0, st, A);
    else
      hipLaunchKernelGGL((heads_kernel<T, EVEN, TPR, false>), grid, dim3(kThreads), 0, st, A);
    return hipGetLastError();
  }
};

struct Backward {
  HeadsBwdArgs A;
  unsigned groups;
  hipStream_t st;
  template <int T, bool EVEN, int TPR>
  hipError_t go() const {
    hipLaunchKernelGGL((heads_bwd_kernel<T, EVEN, TPR>), dim3(groups), dim3(kThreads), 0, st, A);
    return hipGetLastError();
  }
};

struct Read {
  ReadArgs A;
  hipStream_t st;
  template <int T, bool EVEN, int TPR>
  hipError_t go() const {
    // four rows a thread where that leaves work-groups for all CUs (32768 tokens of 8
    // heads of 128, bf16, in a graph: 33.7 us, 34.1 with one; 256 tokens: 3.4, 2.6 with one)
    const int64_t rows = A.tokens * 2 * A.heads, per = kThreads / TPR;
    if (rows >= 2048 * per)
      hipLaunchKernelGGL((read_kernel<T, EVEN, TPR, 4>), dim3((unsigned)((rows + 4 * per - 1) / (4 * per))),
                         dim3(kThreads), 0, st, A);
    else
      hipLaunchKernelGGL((read_kernel<T, EVEN, TPR, 1>), dim3((unsigned)((rows + per - 1) / per)), dim3(kThreads), 0,
                         st, A);
    return hipGetLastError();
  }
};

HeadsArgs forward_args(Heads q, Heads k, Heads v, int64_t tokens, int64_t dim, const mxfp4_rotation& rot,
                       const HeadNorm& n, void* qo, void* ko, const int64_t* slots) {
  HeadsArgs A{};
  A.q = q;
  A.k = k;
  A.v = v;
  A.qo = qo;
  A.ko = ko;
  A.qw = n.qw;
  A.kw = n.kw;
  A.a = angles(rot, tokens);
  A.inv_dim = 1.0 / (double)dim;
  A.tokens = tokens;
  A.dim = (int)dim;
  A.rot = 2 * (int)rot.pairs;
  A.slots = slots;
  const Shape sh = shape_of(tokens, q.heads + k.heads + v.heads, dim, slots != nullptr);
  A.tpg = sh.tpg;
  A.parts = sh.parts;
  A.eps = n.eps;
  A.norm = n.eps >= 0.f;
  A.wide = n.wide;
  return A;
}

// A grid holds below 2^32 threads, and a launch of the cache's form looks at
// the slots of all its tokens for each work-group's (64 KB at most, from the L2).
constexpr int64_t kLaunchTokens = int64_t(1) << 22, kLaunchSlots = 8192;

// Work-groups of the gradient: enough waves to keep the loads going, few
// partial sums.
int64_t bwd_groups(int64_t tokens, int64_t heads, int64_t dim) {
  const int64_t need = shape_of(tokens, heads, dim).groups;
  return need < 1024 ? need : 1024;
}

}  // namespace

hipError_t launch_qk_norm_rope(Heads q, Heads k, int64_t tokens, int64_t dim, int dtype,
                               const mxfp4_rotation& rot, HeadNorm n, void* qo, void* ko, float* rstd,
                               hipStream_t stream) {
  HeadsArgs A = forward_args(q, k, Heads{}, tokens, dim, rot, n, qo, ko, nullptr);
  A.rstd = rstd;
  for (A.first = 0; A.first < tokens; A.first += kLaunchTokens) {
    A.tokens = tokens - A.first < kLaunchTokens ? tokens : A.first + kLaunchTokens;
    const hipError_t e = by_type(dtype, dim, Forward{A, stream});
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_int8_kv_write(Heads q, Heads k, Heads v, int64_t tokens, int64_t dim, int dtype,
                                const mxfp4_rotation& rot, HeadNorm n, const mxfp4_int8_kv& cache,
                                const int64_t* slots, void* qo, hipStream_t stream) {
  HeadsArgs A = forward_args(q, k, v, tokens, dim, rot, n, qo, nullptr, slots);
  A.kc = static_cast<uint8_t*>(cache.k);
  A.vc = static_cast<uint8_t*>(cache.v);
  A.ks = cache.k_scales;
  A.vs = cache.v_scales;
  A.capacity = cache.pages * cache.page_size;
  A.page = (int)cache.page_size;
  A.pitch = (int)cache.pitch;
  // launch after launch, so that a later launch's tokens replace an earlier one's
  for (A.first = 0; A.first < tokens; A.first += kLaunchSlots) {
    A.tokens = tokens - A.first < kLaunchSlots ? tokens : A.first + kLaunchSlots;
    const hipError_t e = by_type(dtype, dim, Forward{A, stream});
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

size_t qk_norm_rope_bwd_ws(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim) {
  return (size_t)bwd_groups(tokens, q_heads + k_heads, dim) * 2 * (size_t)dim * sizeof(float);
}

hipError_t launch_qk_norm_rope_bwd(Heads dq, Heads dk, Heads q, Heads k, int64_t tokens, int64_t dim,
                                   int dtype, const mxfp4_rotation& rot, HeadNorm n, const float* rstd,
                                   void* dqx, void* dkx, void* dqw, void* dkw, void* ws, hipStream_t stream) {
  const bool weights = dqw != nullptr || dkw != nullptr;
  const int parts = (int)bwd_groups(tokens, q.heads + k.heads, dim);
  if (tokens > 0) {
    HeadsBwdArgs A{};
    A.q = q;
    A.k = k;
    A.dq = dq;
    A.dk = dk;
    A.qo = dqx;
    A.ko = dkx;
    A.rstd = rstd;
    A.qw = n.qw;
    A.kw = n.kw;
    A.part = weights ? static_cast<float*>(ws) : nullptr;
    A.a = angles(rot, tokens);
    A.inv_dim = 1.f / (float)dim;
    A.tokens = tokens;
    A.dim = (int)dim;
    A.rot = 2 * (int)rot.pairs;
    const Shape sh = shape_of(tokens, q.heads + k.heads, dim);
    A.tpg = sh.tpg;
    A.parts = sh.parts;
    A.norm = rstd != nullptr;
    A.wide = n.wide;
    const hipError_t e = by_type(dtype, dim, Backward{A, (unsigned)parts, stream});
    if (e != hipSuccess) return e;
  }
  if (!weights) return hipSuccess;
  const dim3 grid((unsigned)((2 * dim + 15) / 16)), blk(1024);
  const float* p = static_cast<const float*>(ws);
  const int wt = n.wide ? kF32 : dtype;
  if (wt == kBF16)
    hipLaunchKernelGGL((heads_dw_kernel<kBF16>), grid, blk, 0, stream, p, parts, (int)dim, dqw, dkw);
  else if (wt == kF16)
    hipLaunchKernelGGL((heads_dw_kernel<kF16>), grid, blk, 0, stream, p, parts, (int)dim, dqw, dkw);
  else
    hipLaunchKernelGGL((heads_dw_kernel<kF32>), grid, blk, 0, stream, p, parts, (int)dim, dqw, dkw);
  return hipGetLastError();
}

hipError_t launch_int8_kv_read(const mxfp4_int8_kv& cache, const int64_t* slots, int64_t tokens,
                               int64_t dim, int dtype, void* k, void* v, hipStream_t stream) {
  // launches of below 2^27 rows, whose 32 threads each fit a grid
  const int64_t most = (int64_t(1) << 27) / (2 * cache.heads), row = cache.heads * dim * (dtype == kF32 ? 4 : 2);
  for (int64_t first = 0; first < tokens; first += most) {
    const int64_t n = tokens - first < most ? tokens - first : most;
    const ReadArgs A{static_cast<const uint8_t*>(cache.k), static_cast<const uint8_t*>(cache.v),
                     cache.k_scales, cache.v_scales, slots + first, static_cast<uint8_t*>(k) + first * row,
                     static_cast<uint8_t*>(v) + first * row, n, cache.pages * cache.page_size,
                     (int)dim, (int)cache.heads, (int)cache.page_size, (int)cache.pitch};
    const hipError_t e = by_type(dtype, dim, Read{A, stream});
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mx
