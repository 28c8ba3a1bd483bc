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
// LDS. Angles are taken in fp64, where position * frequency and the whole
// turns are exact to 2^-53 of the angle; the rest of at most an eighth of a turn goes to
// fp32 and a Taylor series. Squares are summed in fp64 as in the norm of whole
// rows (norm.hip), everything else is in fp32, rounded once at the end.
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
// x^10 (the next terms are below 2^-29 of the sum).
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

  // columns past the pairs keep their value: factors 1 and 0
  __device__ __forceinline__ void factors(const float* cs, const float* sn, int rot, int t) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int at = (t + TPR * i) * V + k;
        c[i][k] = at < rot ? cs[at] : 1.f;
        s[i][k] = at < rot ? sn[at] : 0.f;
      }
  }

  // z turned (sign 1) or turned back (sign -1). A pair's other value comes from
  // the same thread (half 1), or through `meet`, which holds this row of the wave.
  __device__ __forceinline__ void turn(float (&z)[R][V], float* meet, int half, int rot, float sign,
                                       int t) const {
    float o[R][V];
    if (half == 1) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) o[i][k] = z[i][k ^ 1];
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
        z[i][k] = at < rot ? fmaf(z[i][k], c[i][k], sign * s[i][k] * o[i][k]) : z[i][k];
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
  const void *qw, *kw;
  Angles a;
  double inv_dim;
  int64_t first, tokens;  // of this launch: [first, tokens)
  int dim, rot;
  int wpt;                // waves a token: 4, or 1
  float eps;
  bool norm, wide;
  // the cache: codes [pages][heads][page][pitch]
  uint8_t *kc, *vc;
  float *ks, *vs;
  const int64_t* slots;
  int64_t capacity;
  int page, pitch;
};

template <int T, bool EVEN, int TPR, bool CACHE>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsArgs A) {
  typedef Lanes<T, EVEN, TPR> L;
  constexpr int R = L::R, V = L::V, RPW = 64 / TPR;
  __shared__ float cs[kWaves * kHeadMax], sn[kWaves * kHeadMax];
  __shared__ float meet_all[kWaves * 64 * kE];
  __shared__ int64_t cell[kWaves];  // a token's row of head 0 in the cache, or -1
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, t = lane % TPR, sub = lane / TPR;
  const int tpg = kWaves / A.wpt;   // tokens a work-group
  const int64_t token0 = A.first + (int64_t)blockIdx.x * tpg;
  const int n = (int)min((int64_t)tpg, A.tokens - token0);
  turn_table(A.a, token0, n, cs, sn);
  const int mine = wave / A.wpt;    // this wave's token of the work-group's
  const int64_t token = token0 + mine;
  if constexpr (CACHE) {
    // of tokens with the same slot the last one is written: work-groups look
    // at the slots behind theirs (a launch has few tokens, see below)
    int64_t slot[kWaves];
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      slot[k] = k < n ? A.slots[token0 + k] : -1;
      if (slot[k] >= A.capacity) slot[k] = -1;
    }
    if (threadIdx.x < kWaves) {
      int64_t at = -1;
#pragma unroll
      for (int k = 0; k < kWaves; ++k)
        if ((int)threadIdx.x == k && slot[k] >= 0) {
          const uint32_t s = (uint32_t)slot[k], p = s / (uint32_t)A.page;
          at = (int64_t)p * A.k.heads * A.page + (s - p * (uint32_t)A.page);
        }
      cell[threadIdx.x] = at;
    }
    __syncthreads();
    for (int64_t i = token0 + 1 + threadIdx.x; i < A.tokens; i += kThreads) {
      const int64_t s = A.slots[i];
#pragma unroll
      for (int k = 0; k < kWaves; ++k)
        if (s == slot[k] && i > token0 + k && s >= 0) cell[k] = -1;
    }
  }
  __syncthreads();
  if (mine >= n) return;  // no barrier of the work-group follows
  L f;
  float* const meet = meet_all + (wave * 64 + sub * TPR) * kE;
  f.factors(cs + mine * kHeadMax, sn + mine * kHeadMax, A.rot, t);
  float qw[R][V], kw[R][V];
  load_weight<T, EVEN, TPR, R>(A.qw, A.wide, A.dim, t, qw);
  load_weight<T, EVEN, TPR, R>(A.kw, A.wide, A.dim, t, kw);
  const int H = (int)A.q.heads, K = (int)A.k.heads, rows = H + K + (int)A.v.heads;
  for (int g = (wave % A.wpt) * RPW; g < rows; g += A.wpt * RPW) {
    // rows past the last are done again, and not stored
    const int row = min(g + sub, rows - 1), kind = row < H ? 0 : row < H + K ? 1 : 2;
    const int h = kind == 0 ? row : kind == 1 ? row - H : row - H - K;
    const Heads& x = kind == 0 ? A.q : kind == 1 ? A.k : A.v;
    float v[R][V];
    L::X::load(x.p, token * x.ts + h * x.hs, A.dim, t, v);
    if (A.norm) {
      const float r = factor<TPR>(v, A.inv_dim, A.eps);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k)
          v[i][k] = kind == 2 ? v[i][k] : v[i][k] * r * (kind == 0 ? qw[i][k] : kw[i][k]);
    }
    if (A.rot > 0) {
      float y[R][V];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) y[i][k] = v[i][k];
      f.turn(y, meet, A.a.half, A.rot, 1.f, t);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] = kind == 2 ? v[i][k] : y[i][k];
    }
    if (g + sub >= rows) continue;  // whole rows of threads
    if (kind == 0) {
      L::X::store(A.qo, (token * H + h) * A.dim, A.dim, t, v);
    } else if constexpr (CACHE) {
      const int64_t at = cell[mine];
      if (at >= 0) {
        const int64_t to = at + (int64_t)h * A.page;
        write_codes<T, EVEN, TPR, R>(v, nullptr, (kind == 1 ? A.kc : A.vc) + to * A.pitch, A.pitch,
                                     (kind == 1 ? A.ks : A.vs) + to, A.dim, t);
      }
    } else {
      L::X::store(A.ko, (token * K + h) * A.dim, A.dim, t, v);
    }
  }
}

// ------------------------------------------------------------- gradient
struct HeadsBwdArgs {
  Heads q, k, dq, dk;
  void *qo, *ko;
  const void *qw, *kw;
  float* part;  // [gridDim.x][2][dim] partial sums of the weights' gradients, or NULL
  Angles a;
  double inv_dim;
  int64_t tokens;
  int dim, rot, wpt;
  float eps;
  bool norm, wide;
};

// Work-groups walk the tokens in turn; the weights' gradients are summed in
// registers, then over a work-group in LDS, then over work-groups by a second
// kernel: a fixed order, no atomics.
template <int T, bool EVEN, int TPR>
__global__ __launch_bounds__(kThreads) void heads_bwd_kernel(HeadsBwdArgs A) {
  typedef Lanes<T, EVEN, TPR> L;
  constexpr int R = L::R, V = L::V, RPW = 64 / TPR;
  __shared__ float cs[kWaves * kHeadMax], sn[kWaves * kHeadMax];
  __shared__ float meet_all[kWaves * 64 * kE];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, t = lane % TPR, sub = lane / TPR;
  const int tpg = kWaves / A.wpt, mine = wave / A.wpt;
  const int H = (int)A.q.heads, rows = H + (int)A.k.heads;
  float* const meet = meet_all + (wave * 64 + sub * TPR) * kE;
  float qw[R][V], kw[R][V], dqw[R][V] = {}, dkw[R][V] = {};
  load_weight<T, EVEN, TPR, R>(A.qw, A.wide, A.dim, t, qw);
  load_weight<T, EVEN, TPR, R>(A.kw, A.wide, A.dim, t, kw);
  for (int64_t token0 = (int64_t)blockIdx.x * tpg; token0 < A.tokens; token0 += (int64_t)gridDim.x * tpg) {
    const int n = (int)min((int64_t)tpg, A.tokens - token0);
    __syncthreads();  // the last tokens' factors are read
    turn_table(A.a, token0, n, cs, sn);
    __syncthreads();
    if (mine >= n) continue;
    const int64_t token = token0 + mine;
    L f;
    f.factors(cs + mine * kHeadMax, sn + mine * kHeadMax, A.rot, t);
    for (int g = (wave % A.wpt) * RPW; g < rows; g += A.wpt * RPW) {
      const bool real = g + sub < rows;
      const int row = min(g + sub, rows - 1);
      const bool isq = row < H;
      const int h = isq ? row : row - H;
      const Heads &x = isq ? A.q : A.k, &y = isq ? A.dq : A.dk;
      float u[R][V], d[R][V];
      L::X::load(y.p, token * y.ts + h * y.hs, A.dim, t, d);
      if (A.norm) L::X::load(x.p, token * x.ts + h * x.hs, A.dim, t, u);
      if (A.rot > 0) f.turn(d, meet, A.a.half, A.rot, -1.f, t);
      if (A.norm) {
        const float r = factor<TPR>(u, A.inv_dim, A.eps);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            u[i][k] *= r;
            const float e = d[i][k] * u[i][k];
            dqw[i][k] += real && isq ? e : 0.f;
            dkw[i][k] += real && !isq ? e : 0.f;
            d[i][k] *= isq ? qw[i][k] : kw[i][k];
            s = fmaf(d[i][k], u[i][k], s);
          }
        s = reduce_row<TPR>(s, (float*)nullptr, 0, add32) / (float)A.dim;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) d[i][k] = r * (d[i][k] - u[i][k] * s);
      }
      if (real) L::X::store(isq ? A.qo : A.ko, (token * (isq ? A.q.heads : A.k.heads) + h) * A.dim, A.dim, t, d);
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
// keys'): 32 half-waves of a work-group take every 32nd part of 32 columns.
template <int T>
__global__ __launch_bounds__(1024) void heads_dw_kernel(const float* part, int parts, int dim, void* dq,
                                                        void* dk) {
  __shared__ float red[32][32];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * dim) {
#pragma unroll 8
    for (int p = q; p < parts; p += 32) s += part[(int64_t)p * 2 * dim + c];
  }
  red[q][lane] = s;
  __syncthreads();
  if (q == 0 && c < 2 * dim) {
#pragma unroll
    for (int k = 1; k < 32; ++k) s += red[k][lane];
    if (c < dim) {
      if (dq != nullptr) put1<T>(dq, c, s);
    } else if (dk != nullptr) {
      put1<T>(dk, c - dim, s);
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

// y = code * scale, rounded once. A slot outside the cache reads as zeros.
template <int T, bool EVEN, int TPR>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs A) {
  constexpr int V = 16 / Type<T>::S, R = kE / V;
  const int t = threadIdx.x % TPR;
  const int64_t rows = A.tokens * 2 * A.heads;
  for (int64_t row = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR; row < rows;
       row += (int64_t)gridDim.x * (kThreads / TPR)) {
    const int64_t token = row / (2 * A.heads);
    const int at = (int)(row - token * 2 * A.heads), h = at >> 1;
    const bool isv = at & 1;
    const int64_t slot = A.slots[token];
    float v[R][V] = {};
    if (slot >= 0 && slot < A.capacity) {
      const uint32_t s = (uint32_t)slot, p = s / (uint32_t)A.page;
      const int64_t from = ((int64_t)p * A.heads + h) * A.page + (s - p * (uint32_t)A.page);
      const float scale = (isv ? A.vs : A.ks)[from];
      const uint8_t* q = (isv ? A.vc : A.kc) + from * A.pitch;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = (t + TPR * i) * V;
        if (c < A.pitch) {  // the pitch is a multiple of 64: whole words
          uint32_t d[V / 4];
          if constexpr (V == 4) {
            d[0] = *reinterpret_cast<const uint32_t*>(q + c);
          } else {
            const u32x2 e = *reinterpret_cast<const u32x2*>(q + c);
            d[0] = e.x;
            d[1] = e.y;
          }
#pragma unroll
          for (int k = 0; k < V; ++k) v[i][k] = (float)(int8_t)(d[k / 4] >> (8 * (k & 3))) * scale;
        }
      }
    }
    Row<T, EVEN, TPR, R>::store(isv ? A.v : A.k, (token * A.heads + h) * A.dim, A.dim, t, v);
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

// Waves a token: one where there are tokens enough to fill the GPU with a wave
// each, else four share a token's heads.
int waves_a_token(int64_t tokens) { return tokens >= 4096 ? 1 : 4; }

struct Forward {
  HeadsArgs A;
  hipStream_t st;
  template <int T, bool EVEN, int TPR>
  hipError_t go() const {
    const int64_t tpg = kWaves / A.wpt;
    const dim3 grid((unsigned)((A.tokens - A.first + tpg - 1) / tpg));
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
    const int64_t rows = A.tokens * 2 * A.heads, per = kThreads / TPR;
    const int64_t groups = (rows + per - 1) / per;
    hipLaunchKernelGGL((read_kernel<T, EVEN, TPR>), dim3((unsigned)(groups < 16384 ? groups : 16384)),
                       dim3(kThreads), 0, st, A);
    return hipGetLastError();
  }
};

HeadsArgs forward_args(Heads q, Heads k, Heads v, int64_t tokens, int64_t dim, const mxfp4_rotation& rot,
                       const HeadNorm& n, void* qo, void* ko) {
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
  A.wpt = waves_a_token(tokens);
  A.eps = n.eps;
  A.norm = n.eps >= 0.f;
  A.wide = n.wide;
  return A;
}

// A grid holds below 2^32 threads, and a launch of the cache's form looks at
// the slots of all its tokens for each work-group's (32 KB, from the L2).
constexpr int64_t kLaunchTokens = int64_t(1) << 22, kLaunchSlots = 4096;

// Work-groups of the gradient: enough waves to keep the loads going, few
// partial sums.
int64_t bwd_groups(int64_t tokens) {
  const int64_t tpg = kWaves / waves_a_token(tokens), need = (tokens + tpg - 1) / tpg;
  return need < 1024 ? need : 1024;
}

}  // namespace

hipError_t launch_qk_norm_rope(Heads q, Heads k, int64_t tokens, int64_t dim, int dtype,
                               const mxfp4_rotation& rot, HeadNorm n, void* qo, void* ko,
                               hipStream_t stream) {
  HeadsArgs A = forward_args(q, k, Heads{}, tokens, dim, rot, n, qo, ko);
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
  HeadsArgs A = forward_args(q, k, v, tokens, dim, rot, n, qo, nullptr);
  A.kc = static_cast<uint8_t*>(cache.k);
  A.vc = static_cast<uint8_t*>(cache.v);
  A.ks = cache.k_scales;
  A.vs = cache.v_scales;
  A.slots = slots;
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
  (void)q_heads;
  (void)k_heads;
  return (size_t)bwd_groups(tokens) * 2 * (size_t)dim * sizeof(float);
}

hipError_t launch_qk_norm_rope_bwd(Heads dq, Heads dk, Heads q, Heads k, int64_t tokens, int64_t dim,
                                   int dtype, const mxfp4_rotation& rot, HeadNorm n, void* dqx, void* dkx,
                                   void* dqw, void* dkw, void* ws, hipStream_t stream) {
  const bool weights = dqw != nullptr || dkw != nullptr;
  const int parts = (int)bwd_groups(tokens);
  if (tokens > 0) {
    HeadsBwdArgs A{};
    A.q = q;
    A.k = k;
    A.dq = dq;
    A.dk = dk;
    A.qo = dqx;
    A.ko = dkx;
    A.qw = n.qw;
    A.kw = n.kw;
    A.part = weights ? static_cast<float*>(ws) : nullptr;
    A.a = angles(rot, tokens);
    A.inv_dim = 1.0 / (double)dim;
    A.tokens = tokens;
    A.dim = (int)dim;
    A.rot = 2 * (int)rot.pairs;
    A.wpt = waves_a_token(tokens);
    A.eps = n.eps;
    A.norm = n.eps >= 0.f;
    A.wide = n.wide;
    const hipError_t e = by_type(dtype, dim, Backward{A, (unsigned)parts, stream});
    if (e != hipSuccess) return e;
  }
  if (!weights) return hipSuccess;
  const dim3 grid((unsigned)((2 * dim + 31) / 32)), blk(1024);
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
  const ReadArgs A{static_cast<const uint8_t*>(cache.k), static_cast<const uint8_t*>(cache.v),
                   cache.k_scales, cache.v_scales, slots, k, v, tokens, cache.pages * cache.page_size,
                   (int)dim, (int)cache.heads, (int)cache.page_size, (int)cache.pitch};
  return by_type(dtype, dim, Read{A, stream});
}

}  // namespace mx
