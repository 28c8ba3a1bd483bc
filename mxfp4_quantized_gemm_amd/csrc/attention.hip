// Attention of one new token a sequence over an int8 key-value cache in pages,
// for gfx950 (MI355X).
//
//   s_t = scale ks_t (q . kc_t),   t in [max(0, n - window), n)
//   p_t = exp(s_t - max s),  o = sum_t p_t vs_t vc_t / sum_t p_t
//
// with codes kc, vc and scales ks, vs of the cache's rows. One pass: every wave
// keeps the running maximum, sum and output of its tokens, and they are joined
// at the end.
//
// Work. A line is a key head of a sequence with up to 16 of its query heads; its
// tokens are cut into units of 128, and the work-groups share the units of all
// lines evenly, whatever the sequences' lengths: work-group w takes units [w U /
// W, (w + 1) U / W) of all U, in order of sequence, line and token. A line that
// one work-group has whole is written by it; of the others every work-group
// leaves maximum, sum and output in the workspace (at most two lines a
// work-group, its first and its last), and a second kernel joins them. The
// lengths stay on the GPU: a captured graph serves them as they grow.
//
// A wave takes 32 tokens at a time, without LDS: the codes go from memory to
// registers in the layout in which the matrix instructions (16x16x32, bf16,
// fp32 sums) take them. Scores: rows are tokens, columns query heads; a lane
// then has one head's scores of 4 tokens (twice), which is the layout that the
// second product takes its probabilities in, if its k runs over the tokens in
// the order (lane / 16) 4 + r of the first 16 and then of the last. Its rows
// are the head's columns: a lane holds the values of 8 tokens in dim / 16
// columns, so that bytes become bf16 pairs of two tokens without a move between
// lanes. Outputs have one head a lane, as the scores have.
//
// Precision. Codes are whole numbers below 2^7, exact in bf16. Queries enter as
// the sum of one (bf16), two (fp16) or three (fp32) bf16 numbers, exact but for
// fp32's values below 2^-110; p vs as the sum of two (error 2^-16 of each) for
// 16-bit outputs, three (2^-24) for fp32. All sums are in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "attention_plan.h"
#include "rows.h"

namespace mx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = kUnitWaves, kThreads = 64 * kWaves;
constexpr int kGroup = 16;       // query heads of a line
constexpr int kBatch = 1024;     // sequences of a launch
constexpr int kMaxGroups = 512;  // work-groups: two on each of the 256 CUs
constexpr float kNone = -__builtin_inff();

struct Args {
  Heads q;  // [batch][heads][dim]
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int32_t *table, *lengths;
  void* out;
  float* lse;
  float* ws;
  int64_t table_ld;
  int64_t cache_pages;
  int batch, dim, kv, tiles, group;  // group: query heads a key head; tiles: lines a key head
  int page, most;                    // tokens of a page, and of a table's row
  int window;                        // 0: none
  int rows;                          // heads of a line at most: min(group, 16)
  Divisor page16;                    // by page / 16
  float scale;                       // times log2(e)
};

// A value that is the same in all lanes, for the compiler to know.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// prefix[b] = units a line of the sequences before b, for b <= batch.
__device__ __forceinline__ void prefix_units(const Args& A, int64_t* prefix) {
  __shared__ int64_t sums[kWaves];
  constexpr int PER = kBatch / kThreads;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int64_t own[PER], s = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = threadIdx.x * PER + i;
    s += b < A.batch ? span_of(A.lengths[b], A.most, A.window).units : 0;
    own[i] = s;
  }
  int64_t up = s;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t o = __shfl_up(up, d);
    up += lane >= d ? o : 0;
  }
  if (lane == 63) sums[wave] = up;
  __syncthreads();
  int64_t base = up - s;
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w) base += w < wave ? sums[w] : 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = threadIdx.x * PER + i;
    if (b < A.batch) prefix[b + 1] = base + own[i];
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
}

// Codes and scales of 32 tokens, as a lane holds them.
template <int DP>
struct Raw {
  uint32_t k[2][DP / 16];  // token lane % 16 (+ 16): bytes [lane / 16 * DP / 4, + DP / 4)
  uint32_t v[8][DP / 64];  // token (lane / 16) 4 + j (+ 16): bytes [lane % 16 * DP / 16, + DP / 16)
  f32x4 ks[2], vs[2];      // tokens (lane / 16) 4 + r (+ 16)
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&d)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 q = *reinterpret_cast<const u32x4*>(p + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i + e] = q[e];
    }
  } else if constexpr (N == 3) {
    typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
    typedef u32x3 u32x3_4 __attribute__((aligned(4)));
    const u32x3 q = *reinterpret_cast<const u32x3_4*>(p);
#pragma unroll
    for (int e = 0; e < 3; ++e) d[e] = q[e];
  } else if constexpr (N == 2) {
    const u32x2 q = *reinterpret_cast<const u32x2*>(p);
    d[0] = q.x;
    d[1] = q.y;
  } else {
    d[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Whether tokens [t, t + 16) lie in a page of the cache, and its row (uniform).
struct Place {
  bool ok;
  int64_t row;  // of token t, in rows of all heads
};
__device__ __forceinline__ Place place(const Args& A, const int32_t* table, int head, int t, int n) {
  const int col = (int)divided((uint32_t)t >> 4, A.page16), off = t - col * A.page;
  int id = t < n ? uniform(table[col]) : -1;
  Place p;
  p.ok = id >= 0 && id < A.cache_pages;
  id = p.ok ? id : 0;
  p.row = ((int64_t)id * A.kv + head) * A.page + off;
  return p;
}

template <int DP>
__device__ __forceinline__ void load_tile(const Args& A, const Place& a, const Place& b, int lane,
                                          Raw<DP>& r) {
  const int c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = h ? b.row : a.row;
    load_words<DP / 16>(A.kc + row * DP + (c * DP + g * (DP / 4)), r.k[h]);
    const uint8_t* v = A.vc + row * DP + (g * 4 * DP + c * (DP / 16));
#pragma unroll
    for (int j = 0; j < 4; ++j) load_words<DP / 64>(v + j * DP, r.v[4 * h + j]);
    r.ks[h] = *reinterpret_cast<const f32x4*>(A.ks + row + g * 4);
    r.vs[h] = *reinterpret_cast<const f32x4*>(A.vs + row + g * 4);
  }
}

__device__ __forceinline__ float byte_of(uint32_t q, int b) { return (float)(int8_t)(q >> (8 * b)); }
// The upper halves of two floats, a in the low half: bf16 by truncation.
__device__ __forceinline__ uint32_t upper(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float truncated(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

struct Frag {
  uint32_t w[4];
  __device__ __forceinline__ bf16x8 v() const {
    const u32x4 q = {w[0], w[1], w[2], w[3]};
    return __builtin_bit_cast(bf16x8, q);
  }
};

// v as the sum of N bf16 numbers, each the rest's upper 8 bits (the last one
// rounded); not finite: the first one alone.
template <int N>
__device__ __forceinline__ void split(const float (&v)[8], Frag (&f)[N]) {
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = v[j];
#pragma unroll
  for (int p = 0; p < N; ++p) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      if (p + 1 < N || N == 1) {
        f[p].w[j / 2] = upper(r[j], r[j + 1]);
      } else {
        const bf16x2 h = {(__bf16)r[j], (__bf16)r[j + 1]};
        f[p].w[j / 2] = __builtin_bit_cast(uint32_t, h);
      }
    }
    if (p + 1 < N) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] -= truncated(r[j]);
    }
  }
}

template <int X>
__device__ __forceinline__ float max_groups(float v) {
  return far_lane<X>(v, [](float a, float b) { return fmaxf(a, b); });
}

template <int T, int DP, int QP, int PP>
struct Wave {
  static constexpr int KS = DP / 32, NB = DP / 16;
  Frag q[KS][QP];
  f32x4 acc[NB];
  float m, l;

  __device__ __forceinline__ void start(const Args& A, int b, int head0, int heads, int lane) {
    const int c = lane & 15, g = lane >> 4;
    const int64_t at = b * A.q.ts + (head0 + min(c, heads - 1)) * A.q.hs;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float v[8];
      const int d = g * (DP / 4) + 8 * s;
      constexpr int S = Type<T>::S, V = 16 / S;
      if (A.dim % 8 == 0) {
#pragma unroll
        for (int k = 0; k < 8; k += V) {
          float e[V] = {};
          if (c < heads && d < A.dim)
            unpack<T, V>(*reinterpret_cast<const u32x4_2*>(static_cast<const uint8_t*>(A.q.p) + (at + d + k) * S), e);
#pragma unroll
          for (int j = 0; j < V; ++j) v[k + j] = e[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c < heads && d + j < A.dim ? get1<T>(A.q.p, at + d + j) : 0.f;
      }
      split<QP>(v, q[s]);
      if constexpr (QP > 1) {
        // the rest of an infinity is no number: it stands alone, and so does a NaN,
        // whose upper half might be an infinity's
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!__builtin_isfinite(v[j])) {
            if (v[j] != v[j]) q[s][0].w[j / 2] |= j & 1 ? 0x400000u : 0x40u;
#pragma unroll
            for (int p = 1; p < QP; ++p) q[s][p].w[j / 2] &= j & 1 ? 0xffffu : 0xffff0000u;
          }
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    m = kNone;
    l = 0.f;
  }

  // 32 tokens from t on; `whole`: all of them count.
  __device__ __forceinline__ void tile(const Args& A, const Raw<DP>& r, bool whole, bool oka, bool okb,
                                       int t, const Span& sp, int lane) {
    const int g = lane >> 4;
    float s[8], vs[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 sc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        Frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = r.k[h][2 * k + j / 2];
          f.w[j] = upper(byte_of(w, 2 * (j & 1)), byte_of(w, 2 * (j & 1) + 1));
        }
#pragma unroll
        for (int p = 0; p < QP; ++p)
          sc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.v(), q[k][p].v(), sc, 0, 0, 0);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[4 * h + e] = sc[e] * (r.ks[h][e] * A.scale);
        vs[4 * h + e] = r.vs[h][e];
      }
    }
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = t + (e & 4) * 4 + g * 4 + (e & 3);
        const bool in = (e & 4 ? okb : oka) && at >= sp.first && at < sp.n;
        s[e] = in ? s[e] : kNone;
        vs[e] = in ? vs[e] : 0.f;
      }
    }
    float top = s[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
    if (__any(top > m)) {  // rare after the first tiles
      const float now = fmaxf(m, max_groups<32>(max_groups<16>(top)));
      const float a = now == m ? 1.f : __builtin_amdgcn_exp2f(m - now);
#pragma unroll
      for (int i = 0; i < NB; ++i) acc[i] *= a;
      l *= a;
      m = now;
    }
    const float ref = m == kNone ? 0.f : m;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = __builtin_amdgcn_exp2f(s[e] - ref);
      l += p;
      w[e] = p * vs[e];
    }
    Frag pf[PP];
    split<PP>(w, pf);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      Frag f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f.w[j] = upper(byte_of(r.v[2 * j][i / 4], i & 3), byte_of(r.v[2 * j + 1][i / 4], i & 3));
#pragma unroll
      for (int p = 0; p < PP; ++p)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.v(), pf[p].v(), acc[i], 0, 0, 0);
    }
  }
};

// A line's output and log-sum in its type, from sums relative to 2^m.
template <int T>
__device__ __forceinline__ void finish(const Args& A, int64_t row, int d, float v, float m, float l) {
  // no token, or none with a score above -infinity: zeros
  put1<T>(A.out, row * A.dim + d, l == 0.f ? 0.f : v / l);
  if (d == 0 && A.lse != nullptr) A.lse[row] = l == 0.f ? kNone : (m + __log2f(l)) * 0.69314718f;
}

template <int T, int DP, int QP, int PP>
__global__ __launch_bounds__(kThreads, DP > 128 ? 1 : 2) void attention_kernel(Args A) {
  __shared__ int64_t prefix[kBatch + 1];
  __shared__ float all[kWaves][kGroup][DP + 4];
  __shared__ float all_m[kWaves][kGroup], all_l[kWaves][kGroup];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  prefix_units(A, prefix);
  const int lines = A.kv * A.tiles;
  const int64_t U = prefix[A.batch] * lines;
  // sequences without a token
  for (int b = blockIdx.x; b < A.batch; b += gridDim.x)
    if (prefix[b + 1] == prefix[b])
      for (int i = threadIdx.x; i < (int)A.q.heads * A.dim; i += kThreads)
        finish<T>(A, (int64_t)b * A.q.heads + i / A.dim, i % A.dim, 0.f, 0.f, 0.f);
  if (U == 0) return;
  const int64_t W = min((int64_t)gridDim.x, U), w = blockIdx.x;
  if (w >= W) return;
  const int64_t lo = share(w, U, W), hi = share(w + 1, U, W);
  int b = 0;  // the last sequence that starts at or before lo and has a unit
  for (int at = A.batch, from = 0; from < at;) {
    const int mid = (from + at) / 2;
    if (prefix[mid + 1] * lines > lo) {
      at = mid;
    } else {
      from = mid + 1;
    }
    b = at;
  }
  for (int64_t u = lo; u < hi;) {
    while (prefix[b + 1] * lines <= u) ++b;
    b = uniform(b);
    const Span sp = span_of(uniform(A.lengths[b]), A.most, A.window);
    const int64_t in = u - prefix[b] * lines;
    const int line = uniform((int)(in / sp.units)), unit = uniform((int)(in - (int64_t)line * sp.units));
    const int count = uniform((int)min(hi - u, (int64_t)(sp.units - unit)));
    const int head = line / A.tiles, tile = line - head * A.tiles;
    const int head0 = head * A.group + tile * kGroup, heads = min(A.group - tile * kGroup, kGroup);
    const int32_t* table = A.table + b * A.table_ld;
    Wave<T, DP, QP, PP> W_;
    W_.start(A, b, head0, heads, lane);
    int t = uniform(sp.start + unit * kUnit + wave * kTile);
    const int end = min(sp.n, sp.start + (unit + count) * kUnit);
    Raw<DP> next;
    Place a{false, 0}, c{false, 0};
    if (t < end) {
      a = place(A, table, head, t, sp.n);
      c = place(A, table, head, t + 16, sp.n);
      load_tile<DP>(A, a, c, lane, next);
    }
    while (t < end) {
      const Raw<DP> now = next;
      const bool oka = a.ok, okc = c.ok;
      const int tn = t + kUnit;
      if (tn < end) {
        a = place(A, table, head, tn, sp.n);
        c = place(A, table, head, tn + 16, sp.n);
        load_tile<DP>(A, a, c, lane, next);
      }
      W_.tile(A, now, oka && okc && t >= sp.first && t + kTile <= sp.n, oka, okc, t, sp, lane);
      t = tn;
    }
    // the four waves' sums meet
    float l = W_.l;
    l = far_lane<16>(l, add32);
    l = far_lane<32>(l, add32);
    const int hh = lane & 15, g = lane >> 4;
    if (hh < heads) {
#pragma unroll
      for (int i = 0; i < DP / 16; i += 4)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<f32x4*>(&all[wave][hh][(g * 4 + r) * (DP / 16) + i]) =
              f32x4{W_.acc[i][r], W_.acc[i + 1][r], W_.acc[i + 2][r], W_.acc[i + 3][r]};
      if (g == 0) {
        all_m[wave][hh] = W_.m;
        all_l[wave][hh] = l;
      }
    }
    __syncthreads();
    const bool complete = count == sp.units;
    // a work-group's first line has its first slot, its last line the second
    float* part = A.ws + (2 * w + (u == lo ? 0 : 1)) * (int64_t)A.rows * (DP + 2);
    for (int i = threadIdx.x; i < heads * DP; i += kThreads) {
      const int h = i / DP, d = i % DP;
      float M = all_m[0][h];
#pragma unroll
      for (int k = 1; k < kWaves; ++k) M = fmaxf(M, all_m[k][h]);
      float L = 0.f, v = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        const float f = all_m[k][h] == M ? 1.f : __builtin_amdgcn_exp2f(all_m[k][h] - M);
        L = fmaf(f, all_l[k][h], L);
        v = fmaf(f, all[k][h][d], v);
      }
      if (complete) {
        if (d < A.dim) finish<T>(A, (int64_t)b * A.q.heads + head0 + h, d, v, M, L);
      } else {
        part[h * (DP + 2) + d] = v;
        if (d == 0) part[h * (DP + 2) + DP] = M;
        if (d == 0) part[h * (DP + 2) + DP + 1] = L;
      }
    }
    __syncthreads();
    u += count;
  }
}

// Joins the lines that several work-groups have: one work-group a query head,
// 8 parts at a time, each by 32 threads.
template <int T, int DP>
__global__ __launch_bounds__(kThreads) void join_kernel(Args A, int64_t groups) {
  __shared__ int64_t prefix[kBatch + 1];
  __shared__ float all[8][DP], all_m[8], all_l[8];
  prefix_units(A, prefix);
  const int b = blockIdx.x / (int)A.q.heads, head = blockIdx.x % (int)A.q.heads;
  const int lines = A.kv * A.tiles;
  const int64_t U = prefix[A.batch] * lines, units = prefix[b + 1] - prefix[b];
  if (units == 0) return;
  const int64_t W = min(groups, U);
  const int tile = head % A.group / kGroup, row = head % A.group % kGroup;
  const int64_t L0 = prefix[b] * lines + (head / A.group * A.tiles + tile) * units;
  const int64_t first = owner(L0, U, W), last = owner(L0 + units - 1, U, W);
  if (first == last) return;  // written already
  const int q = threadIdx.x >> 5, t = threadIdx.x & 31;
  constexpr int C = DP / 32;
  float v[C] = {}, m = kNone, l = 0.f;
  for (int64_t w = first + q; w <= last; w += 8) {
    const int slot = w == first && share(w, U, W) < L0 ? 1 : 0;
    const float* part = A.ws + ((2 * w + slot) * A.rows + row) * (int64_t)(DP + 2);
    const float pm = part[DP], pl = part[DP + 1], now = fmaxf(m, pm);
    const float a = m == now ? 1.f : __builtin_amdgcn_exp2f(m - now);
    const float f = pm == now ? 1.f : __builtin_amdgcn_exp2f(pm - now);
    l = l * a + pl * f;
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = v[i] * a + part[t + 32 * i] * f;
    m = now;
  }
#pragma unroll
  for (int i = 0; i < C; ++i) all[q][t + 32 * i] = v[i];
  if (t == 0) {
    all_m[q] = m;
    all_l[q] = l;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < A.dim; d += kThreads) {
    float M = all_m[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) M = fmaxf(M, all_m[k]);
    float L = 0.f, o = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float f = all_m[k] == M ? 1.f : __builtin_amdgcn_exp2f(all_m[k] - M);
      L = fmaf(f, all_l[k], L);
      o = fmaf(f, all[k][d], o);
    }
    finish<T>(A, (int64_t)b * A.q.heads + head, d, o, M, L);
  }
}

int pitch_of(int64_t dim) { return (int)((dim + 63) / 64 * 64); }
int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

// Work-groups of a launch: no more than there can be units.
int64_t groups_of(int64_t batch, int64_t lines, int64_t most) {
  return min64(kMaxGroups, batch * lines * ((most + kUnit - 1) / kUnit));
}

template <int T, int DP, int QP, int PP>
hipError_t go(const Args& A, int64_t groups, hipStream_t st) {
  hipLaunchKernelGGL((attention_kernel<T, DP, QP, PP>), dim3((unsigned)(groups > 0 ? groups : 1)), dim3(kThreads),
                     0, st, A);
  hipError_t e = hipGetLastError();
  // a line of one unit is never cut
  if (e != hipSuccess || A.most <= kUnit) return e;
  hipLaunchKernelGGL((join_kernel<T, DP>), dim3((unsigned)(A.batch * A.q.heads)), dim3(kThreads), 0, st, A,
                     groups);
  return hipGetLastError();
}

template <int T, int QP, int PP>
hipError_t go_dim(const Args& A, int64_t groups, hipStream_t st) {
  switch (pitch_of(A.dim)) {
    case 64: return go<T, 64, QP, PP>(A, groups, st);
    case 128: return go<T, 128, QP, PP>(A, groups, st);
    case 192: return go<T, 192, QP, PP>(A, groups, st);
    default: return go<T, 256, QP, PP>(A, groups, st);
  }
}

}  // namespace

size_t paged_attention_ws(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t table,
                          int64_t page_size) {
  if (table * page_size <= kUnit) return 0;  // nothing to join
  const int64_t group = q_heads / kv_heads, tiles = (group + kGroup - 1) / kGroup;
  const int64_t groups = groups_of(min64(batch, kBatch), kv_heads * tiles, table * page_size);
  return (size_t)groups * 2 * (size_t)min64(group, kGroup) * (size_t)(pitch_of(dim) + 2) * sizeof(float);
}

hipError_t launch_paged_attention(Heads q, int64_t batch, int64_t dim, int dtype, const mxfp4_int8_kv& cache,
                                  const int32_t* pages, int64_t pages_ld, int64_t table,
                                  const int32_t* lengths, float scale, int64_t window, void* out,
                                  float* lse, void* ws, hipStream_t stream) {
  Args A{};
  A.q = q;
  A.kc = static_cast<const uint8_t*>(cache.k);
  A.vc = static_cast<const uint8_t*>(cache.v);
  A.ks = cache.k_scales;
  A.vs = cache.v_scales;
  A.ws = static_cast<float*>(ws);
  A.table_ld = pages_ld;
  A.cache_pages = cache.pages;
  A.dim = (int)dim;
  A.kv = (int)cache.heads;
  A.group = (int)(q.heads / cache.heads);
  A.tiles = (A.group + kGroup - 1) / kGroup;
  A.rows = A.group < kGroup ? A.group : kGroup;
  A.page = (int)cache.page_size;
  A.most = (int)(table * cache.page_size);
  A.page16 = divisor_of((uint32_t)(cache.page_size / kPageUnit));
  A.window = window > 0 && window < A.most ? (int)window : 0;
  A.scale = scale * 1.44269504f;
  for (int64_t b = 0; b < batch; b += kBatch) {
    A.batch = (int)min64(kBatch, batch - b);
    A.q.p = static_cast<const uint8_t*>(q.p) + b * q.ts * (dtype == kF32 ? 4 : 2);
    A.out = static_cast<uint8_t*>(out) + b * q.heads * dim * (dtype == kF32 ? 4 : 2);
    A.lse = lse ? lse + b * q.heads : nullptr;
    A.table = pages + b * pages_ld;
    A.lengths = lengths + b;
    const int64_t groups = groups_of(A.batch, A.kv * A.tiles, A.most);
    const hipError_t e = dtype == kBF16  ? go_dim<kBF16, 1, 2>(A, groups, stream)
                         : dtype == kF16 ? go_dim<kF16, 2, 2>(A, groups, stream)
                                         : go_dim<kF32, 3, 3>(A, groups, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mx
