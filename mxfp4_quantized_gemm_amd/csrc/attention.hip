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
// Work. A line is a key head of a sequence with up to 16 of its query heads. A
// work-group takes a line, or a part of it of the same number of tokens for all
// lines (line_kernel). Where parts would be longer than 4096 tokens, and one long
// sequence among short ones would be waited for, lines are cut into units of 128
// tokens and the work-groups share the units of all lines evenly, whatever the
// sequences' lengths (attention_kernel): work-group w takes units [w U / W, (w + 1) U
// / W) of all U, in order of sequence, line and token. A line that one work-group has
// whole is written by it; of the others every work-group leaves maximum, sum and
// output in the workspace, and a second kernel joins them. The lengths stay on the
// GPU: a captured graph serves them as they grow.
//
// A wave takes 32 tokens at a time. Matrix instructions are 16x16x32, f16, with fp32
// sums. Scores: rows are tokens, columns query heads; the keys' codes and both scales
// reach the instructions' layout through a part of the LDS that is the wave's own (see
// kPitch). A lane then has one head's scores of 4 tokens (twice), which is the layout
// that the second product takes its probabilities in, if its k runs over the tokens in
// the order (lane / 16) 4 + r of the first 16 and then of the last. Its rows are the
// head's columns: the values' codes go from memory to registers in its layout, without
// LDS, a lane holding those of 8 tokens in dim / 16 columns, so that bytes become f16
// pairs of two tokens without a move between lanes. Outputs have one head a lane, as
// the scores have.
//
// Codes to f16, two at a time: with the sign flipped a code c is the byte c + 128;
// a permutation puts two of them into the low bytes of f16 words, where they are
// the subnormals (c + 128) 2^-24, and a packed multiply-add with 2^15 and -2^-2
// makes c 2^-9 of them, exact. (The conversion of a signed byte takes three times as
// long as other instructions here: 7.0 against 2.2 to 2.5 ns a wave.)
//
// Precision. Queries are scaled by a power of two for each head, to a largest
// value in [2^14, 2^15), and enter as one f16 number (bf16, fp16: exact but
// for what lies 2^-39 below the largest) or as the sum of two (fp32: within 2^-24
// of each, or 2^-39 of the largest). p vs is scaled by a power of two for the
// largest vs so far, to below 2^14, and enters as the sum of two (2^-24). One is enough
// for bf16 outputs themselves (2^-12, and calls take up to 4 % less: 64 x 8192 tokens of
// 32 over 8 heads of 128 175.7 us, not 178.2), but the 8-bit product behind them rounds
// again: its result was twice as far from 64 bits as with fp32 probabilities. All sums,
// the maximum and p are in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "attention_plan.h"
#include "rows.h"

namespace mx {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = kUnitWaves, kThreads = 64 * kWaves;
constexpr int kGroup = 16;       // query heads of a line
constexpr int kBatch = 1024;     // sequences of a launch
// Work-groups that share the units evenly: two on each of the 256 CUs at once, of heads
// of more than 128 columns one (their registers leave a SIMD one wave, or two).
constexpr int kMaxGroups = 512;
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
  int splits, chunk;                 // line_kernel's parts of a line, and their tokens
  int rows;                          // heads of a line at most: min(group, 16)
  Divisor page16;                    // by page / 16
  float scale;                       // times log2(e)
};

// A value that is the same in all lanes, for the compiler to know.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Sum over the lanes up to and with this one.
__device__ __forceinline__ int scan_lanes(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // within 16 lanes: shifted by 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 to the next 16, of each 32
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to the upper 32
  return v;
}

// Units a line of the sequences before each: up to 64 sequences in the lanes of
// every wave (their units sum to below 2^31), without a barrier, more in LDS.
struct Plan {
  int64_t* all;  // LDS: [batch + 1], or NULL
  int length;    // this lane's sequence's,
  int upto;      // its units and those before it
  int64_t total;
  __device__ __forceinline__ int length_of(const Args& A, int b) const {
    return all != nullptr ? uniform(A.lengths[b]) : __builtin_amdgcn_readlane(length, b);
  }
  __device__ __forceinline__ int64_t before(int b) const {
    if (all != nullptr) return all[b];
    const int v = __builtin_amdgcn_readlane(upto, uniform(b > 0 ? b - 1 : 0));
    return b > 0 ? v : 0;
  }
};
__device__ __forceinline__ Plan plan_of(const Args& A, int64_t* prefix) {
  __shared__ int64_t sums[kWaves];
  constexpr int PER = kBatch / kThreads;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  Plan p{nullptr, 0, 0, 0};
  if (A.batch <= 64) {
    p.length = lane < A.batch ? A.lengths[lane] : 0;
    p.upto = scan_lanes(span_of(p.length, A.most, A.window).units);
    p.total = __builtin_amdgcn_readlane(p.upto, 63);
    return p;
  }
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
  p.all = prefix;
  p.total = prefix[A.batch];
  return p;
}

// Codes and scales of 32 tokens, as a lane holds them.
template <int DP>
struct Raw {
  u32x4 k[2][DP / 64];     // the first (last) 16 tokens' codes: 16 bytes a lane, 1 KiB a load
  uint32_t v[8][DP / 64];  // token (lane / 16) 4 + j (+ 16): bytes [lane % 16 * DP / 16, + DP / 16)
  float scale;             // of token lane % 32: ks in lanes below 32, vs in the others
  bool ok[2];              // whether the 16 tokens' page is in the cache
};

// The cache is read once: past the caches (64 x 8000 tokens, with one number for p vs:
// 169 us; 189 through them; with two 172 now). Not so the values of heads of 129 to 192
// columns, whose three words a lane are one ordinary load.
template <class X>
__device__ __forceinline__ X load_once(const void* p) {
  return __builtin_nontemporal_load(static_cast<const X*>(p));
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&d)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 q = load_once<u32x4>(p + 4 * i);
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
    const u32x2 q = load_once<u32x2>(p);
    d[0] = q.x;
    d[1] = q.y;
  } else {
    d[0] = load_once<uint32_t>(p);
  }
}

// Where a wave's next 32 tiles lie: lane 2 i + h has the page (as the table has
// it) and the row in it of the 16 tokens from t + i step + 16 h on. Looked up
// for 32 tiles at once, so that no tile's loads wait for a page's number.
struct Places {
  int id, off;
};
__device__ __forceinline__ Places places(const Args& A, const int32_t* table, uint32_t t, int step, int lane) {
  const uint32_t at = t + (uint32_t)(lane >> 1) * step + (lane & 1) * 16;  // may be past 2^31
  const uint32_t col = divided(at >> 4, A.page16);                         // read where it is below
  Places p;
  p.off = (int)(at - col * A.page);
  p.id = -1;
  if (at < (uint32_t)A.most) p.id = table[col];
  return p;
}

// The same as rows of the cache (of all heads), with a bit of `ok` for each 16
// tokens whose page is in it; those of the others are in page 0.
struct Rows16 {
  int64_t row;
  uint64_t ok;
};
__device__ __forceinline__ Rows16 rows_of_pages(const Args& A, Places p, int head) {
  const bool ok = p.id >= 0 && p.id < A.cache_pages;
  return {((int64_t)(ok ? p.id : 0) * A.kv + head) * A.page + p.off, __ballot(ok)};
}
__device__ __forceinline__ int64_t lane_of(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)v, lane), hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

template <int DP>
__device__ __forceinline__ void load_tile(const Args& A, const Rows16& p, int tile, int lane, Raw<DP>& r) {
  const int c = lane & 15, g = lane >> 4;
  int64_t row[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    row[h] = lane_of(p.row, 2 * tile + h);
    r.ok[h] = p.ok >> (2 * tile + h) & 1;
#pragma unroll
    for (int i = 0; i < DP / 64; ++i) r.k[h][i] = load_once<u32x4>(A.kc + row[h] * DP + (1024 * i + 16 * lane));
    const uint8_t* v = A.vc + row[h] * DP + (g * 4 * DP + c * (DP / 16));
#pragma unroll
    for (int j = 0; j < 4; ++j) load_words<DP / 64>(v + j * DP, r.v[4 * h + j]);
  }
  r.scale = load_once<float>((lane & 32 ? A.vs : A.ks) + (lane & 16 ? row[1] : row[0]) + c);
  __builtin_amdgcn_sched_barrier(0);  // all loads before what waits for the last tile's
}

constexpr uint32_t kFlip = 0x80808080u;  // codes to bytes code + 128
// c 2^-9 of byte b of p and byte e of q (of flipped words), as an f16 pair.
__device__ __forceinline__ uint32_t pair_of(uint32_t p, int b, uint32_t q, int e) {
  const f16x2 up = {(_Float16)0x1p15f, (_Float16)0x1p15f}, off = {(_Float16)-0.25f, (_Float16)-0.25f};
  const uint32_t u = __builtin_amdgcn_perm(q, p, 0x0c000c00u | (uint32_t)(4 + e) << 16 | (uint32_t)b);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, u), up, off));
}

struct Frag {
  uint32_t w[4];
  __device__ __forceinline__ f16x8 v() const {
    const u32x4 q = {w[0], w[1], w[2], w[3]};
    return __builtin_bit_cast(f16x8, q);
  }
};
__device__ __forceinline__ f32x4 mfma(const Frag& a, const Frag& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v(), b.v(), c, 0, 0, 0);
}

// v as the sum of N f16 numbers, each the rest rounded to nearest. (The values are hidden
// from the compiler: it fuses a product that made one into its conversion, which can
// then round otherwise than the fp32 number that the rest is taken from.)
template <int N>
__device__ __forceinline__ void split(float (&v)[8], Frag (&f)[N]) {
  if constexpr (N > 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) asm("" : "+v"(v[j]));
  }
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const f16x2 h = {(_Float16)v[j], (_Float16)v[j + 1]};
    f[0].w[j / 2] = __builtin_bit_cast(uint32_t, h);
    if constexpr (N > 1) {
      const f16x2 r = {(_Float16)(v[j] - (float)h.x), (_Float16)(v[j + 1] - (float)h.y)};
      f[1].w[j / 2] = __builtin_bit_cast(uint32_t, r);
    }
  }
}

template <int X>
__device__ __forceinline__ float max_groups(float v) {
  return far_lane<X>(v, [](float a, float b) { return fmaxf(a, b); });
}

// K's codes pass through LDS, a wave's tile through 2 to 9 KiB of its own: the
// matrix instruction's lanes hold 16 tokens side by side, whose rows, loaded so,
// are 16 cache lines for every 16 lanes; loaded row after row a 16th of that (64 x 8000
// tokens, with one number for p vs: 174 us and 169). Rows have 16 bytes more there, so
// that 16 tokens' reads meet in no bank.
template <int DP>
constexpr int kPitch = DP + 16;

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A work-group's LDS: what its waves stage, then their sums.
template <int DP, int NW>
union alignas(16) Shared {
  uint8_t stage[NW][kTile * kPitch<DP> + 256];
  float all[NW][kGroup][DP + 4];
};

static_assert(alignof(Shared<64, 4>) >= 16, "it is accessed 16 bytes at a time");

constexpr float kSmallest = 0x1p-112f;  // so that 2^14 over it is in fp32's range

template <int T, int DP, int QP>
struct Wave {
  static constexpr int KS = DP / 32, NB = DP / 16, PP = 2;  // PP, QP: f16 numbers for p vs and a query
  Frag q[KS][QP];
  f32x4 acc[NB];  // sum of p vs c, times 2^14 / top_vs and 2^-9
  float hs;       // scores are sums of codes times this and ks
  float m, l;     // scores' maximum, sum of p (of this lane's tokens)
  float top_vs;   // a power of two above the scales so far,
  float unit;     // 2^14 over it
  uint8_t* stage; // this wave's LDS: 32 rows of K's codes, their ks and vs

  // The first of 8 columns that lanes of group g have in k-step s of the scores.
  static __device__ __forceinline__ int column(int s, int g) { return (g + 4 * (s / 2)) * 16 + 8 * (s & 1); }

  // The queries of a lane's head (of the last one in the lanes past it, whose
  // results nobody reads), loaded early and converted when the first codes are
  // on their way.
  static constexpr int V = 16 / Type<T>::S;  // values of a load
  __device__ __forceinline__ void load_queries(const Args& A, int b, int head0, int heads, int lane,
                                               float (&v)[KS][8]) {
    const int64_t at = b * A.q.ts + (head0 + min(lane & 15, heads - 1)) * A.q.hs;
    if (A.dim % 8 == 0) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        // columns past the head: the first ones' values, replaced below
        const int d = column(s, lane >> 4), from = d < A.dim ? d : 0;
#pragma unroll
        for (int k = 0; k < 8; k += V) {
          float e[V];
          const uint8_t* p = static_cast<const uint8_t*>(A.q.p) + (at + from + k) * Type<T>::S;
          unpack<T, V>(*reinterpret_cast<const u32x4_2*>(p), e);
#pragma unroll
          for (int j = 0; j < V; ++j) v[s][k + j] = e[j];
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[s][j] = get1<T>(A.q.p, at + min(column(s, lane >> 4) + j, A.dim - 1));
    }
  }

  __device__ __forceinline__ void start(const Args& A, float (&v)[KS][8], int lane) {
    if (A.dim < DP) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[s][j] = column(s, lane >> 4) + j < A.dim ? v[s][j] : 0.f;
    }
    float big = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(v[s][j]));  // (a NaN is passed over)
    if (__any(big == __builtin_inff())) {
      big = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(v[s][j]) < __builtin_inff() ? fabsf(v[s][j]) : 0.f);
    }
    big = max_groups<32>(max_groups<16>(big));
    const int up = big > 0.f ? 15 - __builtin_amdgcn_frexp_expf(big) : 0;  // big 2^up in [2^14, 2^15)
    hs = __builtin_amdgcn_ldexpf(A.scale, 9 - up);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[s][j] = __builtin_amdgcn_ldexpf(v[s][j], up);
      split<QP>(v[s], q[s]);
      if constexpr (QP > 1) {
        // the rest of an infinity is no number: it stands alone
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!__builtin_isfinite(v[s][j])) q[s][1].w[j / 2] &= j & 1 ? 0xffffu : 0xffff0000u;
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    m = kNone;
    l = 0.f;
    top_vs = kSmallest;
    unit = 0x1p14f / kSmallest;
  }

  // 32 tokens from t on.
  __device__ __forceinline__ void tile(const Args& A, const Raw<DP>& r, int t, const Span& sp, int lane) {
    const int g = lane >> 4;
    f32x4 sc[2] = {};
    wave_sync();  // the last tile's reads are done
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) {
        const int at = 64 * i + lane;
        uint8_t* const to = stage + (16 * h + at / (DP / 16)) * kPitch<DP> + at % (DP / 16) * 16;
        *reinterpret_cast<u32x4*>(to) = r.k[h][i] ^ kFlip;
      }
    float* const scales = reinterpret_cast<float*>(stage + kTile * kPitch<DP>);
    scales[lane] = r.scale;
    wave_sync();
    f32x4 kss[2], vss[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      kss[h] = *reinterpret_cast<const f32x4*>(scales + 16 * h + 4 * g);
      vss[h] = *reinterpret_cast<const f32x4*>(scales + 32 + 16 * h + 4 * g);
    }
    u32x4 codes[2][DP / 64];
#pragma unroll
    for (int i = 0; i < DP / 64; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        codes[h][i] =
            *reinterpret_cast<const u32x4*>(stage + (16 * h + (lane & 15)) * kPitch<DP> + (g + 4 * i) * 16);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      Frag f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = codes[h][k / 2][2 * (k & 1) + j / 2];
          f[h].w[j] = pair_of(w, 2 * (j & 1), w, 2 * (j & 1) + 1);
        }
#pragma unroll
      for (int p = 0; p < QP; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[h] = mfma(f[h], q[k][p], sc[h]);
    }
    float s[8], vs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s[e] = sc[e / 4][e & 3] * (kss[e / 4][e & 3] * hs);
      vs[e] = vss[e / 4][e & 3];
    }
    if (!(r.ok[0] && r.ok[1] && t >= sp.first && t + kTile <= sp.n)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = t + (e & 4) * 4 + g * 4 + (e & 3);
        const bool in = r.ok[e / 4] && at >= sp.first && at < sp.n;
        s[e] = in ? s[e] : kNone;
        vs[e] = in ? vs[e] : 0.f;
      }
    }
    float top = s[0], big = fabsf(vs[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      top = fmaxf(top, s[e]);
      big = fmaxf(big, fabsf(vs[e]));
    }
    if (__any(top > m || big >= top_vs)) {  // rare after the first tiles
      const float now = fmaxf(m, max_groups<32>(max_groups<16>(top)));
      big = max_groups<32>(max_groups<16>(big));
      // the power of two above (2^127 at most: a scale past it is as good as infinite)
      const float above = __uint_as_float(min((__float_as_uint(big) & 0x7f800000u) + 0x800000u, 0x7f000000u));
      const float vs_now = fmaxf(top_vs, above);
      const float a = now == m ? 1.f : __builtin_amdgcn_exp2f(m - now);
      const float o = a * (top_vs / vs_now);
#pragma unroll
      for (int i = 0; i < NB; ++i) acc[i] *= o;
      l *= a;
      m = now;
      top_vs = vs_now;
      unit = 0x1p14f / vs_now;
    }
    const float ref = m == kNone ? 0.f : m;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = __builtin_amdgcn_exp2f(s[e] - ref);
      w[e] = p * (vs[e] * unit);
      s[e] = p;
    }
    l += ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    Frag pf[PP];
    split<PP>(w, pf);
    uint32_t v[8][DP / 64];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) v[j][i] = r.v[j][i] ^ kFlip;
#pragma unroll
    for (int i = 0; i < NB; i += 2) {
      Frag f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f[h].w[j] = pair_of(v[2 * j][i / 4], (i + h) & 3, v[2 * j + 1][i / 4], (i + h) & 3);
#pragma unroll
      for (int p = 0; p < PP; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[i + h] = mfma(f[h], pf[p], acc[i + h]);
    }
  }

  // Tiles at t, t + step, ... below `end`; p: where the first ones lie; v: the
  // queries. With AHEAD > 0 that many tiles' loads are on their way during one's
  // products. They are made in any case then (behind the last tile: the last one's again),
  // because what waits for a tile's loads counts those behind them: with loads under a
  // condition it waited for the next tile's too.
  template <int AHEAD>
  __device__ __forceinline__ void run(const Args& A, const int32_t* table, Places p, int head, int t, int step,
                                      int end, const Span& sp, float (&v)[KS][8], int lane) {
    constexpr int BUFS = AHEAD + 1, BATCH = 32 / BUFS * BUFS;
    Raw<DP> r[BUFS];
    // tiles from the batch's first on
    int left = t < end ? uniform((int)((uint32_t)(end - t + step - 1) / (uint32_t)step)) : 0;
    Places then = p;
    Rows16 now = rows_of_pages(A, p, head);
#pragma unroll
    for (int j = 0; j < (AHEAD > 0 ? AHEAD : 1); ++j) load_tile<DP>(A, now, max(min(j, left - 1), 0), lane, r[j]);
    start(A, v, lane);
    if (left == 0) return;
    for (int i = 0;;) {
      if (i == 0) then = places(A, table, (uint32_t)t + (uint32_t)(BATCH * step), step, lane);
      const Rows16 next = i + BUFS == BATCH ? rows_of_pages(A, then, head) : now;  // needed from here on
#pragma unroll
      for (int j = 0; j < BUFS; ++j) {
        const int k = min(i + j + (AHEAD > 0 ? AHEAD : 1), left - 1);
        const auto ahead = [&]() {
          load_tile<DP>(A, k < BATCH ? now : next, k < BATCH ? k : k - BATCH, lane, r[(j + AHEAD) % BUFS]);
        };
        if (AHEAD > 0) ahead();
        tile(A, r[j], t, sp, lane);
        t += step;
        if (t >= end) return;
        if (AHEAD == 0) ahead();
      }
      i += BUFS;
      if (i == BATCH) {
        i = 0;
        left -= BATCH;
        now = next;
      }
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

// The waves' sums of a line meet in LDS: its output, or (part not NULL) the sums
// for another kernel to join. `u` is in a wave's registers until here.
template <int T, int DP, int NW, class W>
__device__ __forceinline__ void meet(const Args& A, Shared<DP, NW>& lds, const W& u, int wave, int lane, int b,
                                     int head0, int heads, float* part) {
  auto& all = lds.all;
  __syncthreads();  // the waves are done with what they staged
  __shared__ float all_m[NW][kGroup], all_l[NW][kGroup];
  const int hh = lane & 15, g = lane >> 4, thread = wave * 64 + lane;
  float l = u.l;
  l = far_lane<16>(l, add32);
  l = far_lane<32>(l, add32);
  const float unit = u.top_vs * 0x1p-5f;  // of acc: 2^9 top_vs / 2^14
  if (hh < heads) {
#pragma unroll
    for (int i = 0; i < DP / 16; i += 4)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<f32x4*>(&all[wave][hh][(g * 4 + r) * (DP / 16) + i]) =
            f32x4{u.acc[i][r], u.acc[i + 1][r], u.acc[i + 2][r], u.acc[i + 3][r]} * unit;
    if (g == 0) {
      all_m[wave][hh] = u.m;
      all_l[wave][hh] = l;
    }
  }
  __syncthreads();
  for (int i = thread; i < heads * DP; i += 64 * NW) {
    const int h = i / DP, d = i % DP;
    float M = all_m[0][h];
#pragma unroll
    for (int k = 1; k < NW; ++k) M = fmaxf(M, all_m[k][h]);
    float L = 0.f, v = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float f = all_m[k][h] == M ? 1.f : __builtin_amdgcn_exp2f(all_m[k][h] - M);
      L = fmaf(f, all_l[k][h], L);
      v = fmaf(f, all[k][h][d], v);
    }
    if (part == nullptr) {
      if (d < A.dim) finish<T>(A, (int64_t)b * A.q.heads + head0 + h, d, v, M, L);
    } else {
      part[h * (DP + 2) + d] = v;
      if (d == 0) part[h * (DP + 2) + DP] = M;
      if (d == 0) part[h * (DP + 2) + DP + 1] = L;
    }
  }
  __syncthreads();
}

// Lines shared evenly by the work-groups.
template <int T, int DP, int QP>
__global__ __launch_bounds__(kThreads, DP > 128 ? 1 : 2) void attention_kernel(Args A) {
  __shared__ int64_t prefix[kBatch + 1];
  __shared__ Shared<DP, kWaves> lds;
  const int wave = threadIdx.x >> 6;
  int lane = threadIdx.x & 63;
  const Plan plan = plan_of(A, prefix);
  const int lines = A.kv * A.tiles;
  const int64_t U = plan.total * lines;
  // sequences without a token
  for (int b = blockIdx.x; b < A.batch; b += gridDim.x)
    if (plan.before(b + 1) == plan.before(b))
      for (int i = threadIdx.x; i < (int)A.q.heads * A.dim; i += kThreads)
        finish<T>(A, (int64_t)b * A.q.heads + i / A.dim, i % A.dim, 0.f, 0.f, 0.f);
  if (U == 0) return;
  const int64_t W = min((int64_t)gridDim.x, U), w = blockIdx.x;
  if (w >= W) return;
  const int64_t lo = share(w, U, W), hi = share(w + 1, U, W);
  int b = 0;  // the last sequence that starts at or before lo and has a unit
  if (plan.all == nullptr) {
    b = __popcll(__ballot(lane < A.batch && (int64_t)plan.upto * lines <= lo));
  } else {
    for (int at = A.batch, from = 0; from < at;) {
      const int mid = (from + at) / 2;
      if (prefix[mid + 1] * lines > lo) {
        at = mid;
      } else {
        from = mid + 1;
      }
      b = at;
    }
  }
  for (int64_t u = lo; u < hi;) {
    asm volatile("" : "+v"(lane));  // else what a line needs of it is kept over all lines, and spills
    while (plan.before(b + 1) * lines <= u) ++b;
    b = uniform(b);
    const Span sp = span_of(plan.length_of(A, b), A.most, A.window);
    const int64_t in = u - plan.before(b) * lines;
    const int line = uniform((int)quotient(in, sp.units)), unit = uniform((int)(in - (int64_t)line * sp.units));
    const int count = uniform((int)min(hi - u, (int64_t)(sp.units - unit)));
    const int head = line / A.tiles, tile = line - head * A.tiles;
    const int head0 = head * A.group + tile * kGroup, heads = min(A.group - tile * kGroup, kGroup);
    const int32_t* table = A.table + b * A.table_ld;
    const int t = uniform(sp.start + unit * kUnit + wave * kTile);
    const int end = uniform(min(sp.n, sp.start + (unit + count) * kUnit));
    const Places p = places(A, table, t, kUnit, lane);
    typedef Wave<T, DP, QP> Sums;
    Sums sums;
    sums.stage = lds.stage[wave];
    float q[Sums::KS][8];
    sums.load_queries(A, b, head0, heads, lane, q);
    sums.template run<1>(A, table, p, head, t, kUnit, end, sp, q, lane);
    // a work-group's first line has its first slot, its last line the second
    meet<T, DP, kWaves>(A, lds, sums, wave, lane, b, head0, heads,
                        count == sp.units ? nullptr : A.ws + (2 * w + (u == lo ? 0 : 1)) * (int64_t)A.rows * (DP + 2));
    u += count;
  }
}

// A work-group a line, or one of A.splits parts of it, each of A.chunk tokens.
template <int T, int DP, int QP, int NW>
__global__ __launch_bounds__(64 * NW, DP > 128 ? 1 : T == kF32 ? 2 : 4) void line_kernel(Args A) {
  __shared__ Shared<DP, NW> lds;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int lines = A.kv * A.tiles;
  const int part = blockIdx.x % A.splits, of = blockIdx.x / A.splits, b = of / lines, line = of - b * lines;
  const int head = line / A.tiles, tile = line - head * A.tiles;
  const int head0 = head * A.group + tile * kGroup, heads = min(A.group - tile * kGroup, kGroup);
  const int32_t* table = A.table + b * A.table_ld;
  const int length = A.lengths[b];
  typedef Wave<T, DP, QP> Sums;
  Sums sums;
  sums.stage = lds.stage[wave];
  float q[Sums::KS][8];
  sums.load_queries(A, b, head0, heads, lane, q);
  Places p{-1, 0};
  // without a window the pages are looked up before the length is there
  const int from = part * A.chunk + wave * kTile;
  if (A.window == 0) p = places(A, table, uniform(from), NW * kTile, lane);
  const Span sp = span_of(uniform(length), A.most, A.window);
  if (part > 0 && sp.start + part * A.chunk >= sp.n) return;
  const int t = uniform(sp.start + from);
  if (A.window != 0) p = places(A, table, t, NW * kTile, lane);
  sums.template run<0>(A, table, p, head, t, NW * kTile, min(sp.n, sp.start + (part + 1) * A.chunk), sp, q,
                       lane);
  meet<T, DP, NW>(A, lds, sums, wave, lane, b, head0, heads,
                  sp.n - sp.start <= A.chunk ? nullptr : A.ws + (int64_t)blockIdx.x * A.rows * (DP + 2));
}

// Joins the lines that several work-groups have: one work-group a query head, 8
// parts at a time, each by 32 threads. CUT: as line_kernel cuts them, else as
// attention_kernel does.
template <int T, int DP, bool CUT>
__global__ __launch_bounds__(kThreads) void join_kernel(Args A, int64_t groups) {
  __shared__ int64_t prefix[CUT ? 1 : kBatch + 1];
  __shared__ float all[8][DP], all_m[8], all_l[8];
  const int b = blockIdx.x / (int)A.q.heads, head = blockIdx.x % (int)A.q.heads;
  const int lines = A.kv * A.tiles, tile = head % A.group / kGroup, row = head % A.group % kGroup;
  const int line = head / A.group * A.tiles + tile;
  int64_t first, last, slot;  // parts; the slot of the first one
  int step;                   // slots from part to part
  if constexpr (CUT) {
    const Span sp = span_of(A.lengths[b], A.most, A.window);
    first = 0;
    last = (sp.n - sp.start - 1) / A.chunk;
    slot = ((int64_t)b * lines + line) * A.splits;
    step = 1;
  } else {
    const Plan plan = plan_of(A, prefix);
    const int64_t U = plan.total * lines, units = plan.before(b + 1) - plan.before(b);
    if (units == 0) return;
    const int64_t W = min(groups, U), L0 = plan.before(b) * lines + line * units;
    first = owner(L0, U, W);
    last = owner(L0 + units - 1, U, W);
    slot = 2 * first;
    step = 2;
    // of the first one's two slots the line has the second if another line begins in it
    if (share(first, U, W) < L0) slot |= int64_t(1) << 62;
  }
  if (first >= last) return;  // written already
  const bool second = slot >> 62 & 1;
  slot &= ~(int64_t(1) << 62);
  const int q = threadIdx.x >> 5, t = threadIdx.x & 31;
  constexpr int C = DP / 32;
  float v[C] = {}, m = kNone, l = 0.f;
  for (int64_t w = first + q; w <= last; w += 8) {
    const int64_t at = slot + (w - first) * step + (w == first && second ? 1 : 0);
    const float* part = A.ws + (at * A.rows + row) * (int64_t)(DP + 2);
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

// How a launch is cut: 160 lines or more are left whole, and those of at most two
// steps of a work-group's waves; others go into about 512 parts. Where work-groups would
// have more than kChunk tokens, the units are shared evenly. (32 query and 8 key heads
// of 128, bf16, in a graph, tables as wide as the longest sequence. 16 sequences of up to
// 2048 tokens: all of them full 18.0 to 19.2 us, spread evenly from 1 on 16.2, one full
// and the others of 100 tokens 11.6; in 256 parts 16.9, 15.7, 14.0; shared evenly 22.7,
// 18.6, 10.1. Whole | in parts: 20 x 1000 tokens 13.4 | 16.0, 30 x 4000 42.4 | 48.5, but
// 16 x 4000 35.8 | 28.8; 1 x 500 8.2 | 8.8, but 1 x 1000 11.6 | 8.9.)
//
// The host knows a table's room, not the lengths, and does not wait for these: the room
// sets the cut. Parts of short sequences are without work then, and few work-groups have
// it all where the tables have room for far more than the sequences hold: one sequence of
// 1000 tokens takes 8.8 us by its own table, 20.3 by one of 131072 tokens; 4096 tokens 9.3
// and 35.5; two of 4096 9.5 and 58.2; four (shared evenly then) 12.7 and 14.9. So do one
// long line among many short ones that are left whole: 24 sequences, one of 4096 tokens
// and the others of 100, 32 us; all of 4096 tokens 37.9 (shared evenly 12.5 and 43.5).
struct Cut {
  int64_t splits, chunk;  // splits 0: shared evenly
  int64_t groups;
};
constexpr int64_t kEnough = 160, kParts = 512, kChunk = 4096;
// Tokens that line_kernel's waves take at a time.
int64_t step_of(int64_t dim) { return pitch_of(dim) > 128 ? 4 * kTile : 8 * kTile; }
// most: tokens that a line may have. Fewer than 160 lines are cut, into fewer than
// 512 + 160 parts: below kMaxSlots, twice the even shares.
constexpr int64_t kMaxSlots = 2 * kMaxGroups;
Cut cut_of(int64_t batch, int64_t lines, int64_t dim, int64_t most) {
  const int64_t step = step_of(dim), steps = (most + step - 1) / step;
  if (steps <= 2) return {1, steps * step, batch * lines};
  int64_t splits = batch * lines >= kEnough ? 1 : min64(steps, (kParts + batch * lines - 1) / (batch * lines));
  const int64_t chunk = (steps + splits - 1) / splits * step;
  splits = (most + chunk - 1) / chunk;
  if (chunk <= kChunk) return {splits, chunk, batch * lines * splits};
  return {0, 0, min64(kMaxGroups, batch * lines * ((most + kUnit - 1) / kUnit))};
}

template <int T, int DP, int QP>
hipError_t go(Args A, hipStream_t st) {
  const Cut c = cut_of(A.batch, A.kv * A.tiles, A.dim, A.window > 0 ? min64(A.most, (int64_t)A.window + 15) : A.most);
  const dim3 heads((unsigned)(A.batch * A.q.heads));
  hipError_t e;
  if (c.splits > 0) {
    A.splits = (int)c.splits;
    A.chunk = (int)c.chunk;
    constexpr int NW = DP > 128 ? 4 : 8;
    hipLaunchKernelGGL((line_kernel<T, DP, QP, NW>), dim3((unsigned)c.groups), dim3(64 * NW), 0, st, A);
    e = hipGetLastError();
    if (e != hipSuccess || c.splits == 1) return e;
    hipLaunchKernelGGL((join_kernel<T, DP, true>), heads, dim3(kThreads), 0, st, A, c.groups);
  } else {
    hipLaunchKernelGGL((attention_kernel<T, DP, QP>), dim3((unsigned)c.groups), dim3(kThreads), 0, st, A);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((join_kernel<T, DP, false>), heads, dim3(kThreads), 0, st, A, c.groups);
  }
  return hipGetLastError();
}

template <int T, int QP>
hipError_t go_dim(const Args& A, hipStream_t st) {
  switch (pitch_of(A.dim)) {
    case 64: return go<T, 64, QP>(A, st);
    case 128: return go<T, 128, QP>(A, st);
    case 192: return go<T, 192, QP>(A, st);
    default: return go<T, 256, QP>(A, st);
  }
}

}  // namespace

size_t paged_attention_ws(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t table,
                          int64_t page_size) {
  (void)batch;
  if (table * page_size <= 2 * step_of(dim)) return 0;
  return (size_t)kMaxSlots * (size_t)min64(q_heads / kv_heads, kGroup) * (size_t)(pitch_of(dim) + 2) * sizeof(float);
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
    const hipError_t e = dtype == kBF16  ? go_dim<kBF16, 1>(A, stream)
                         : dtype == kF16 ? go_dim<kF16, 1>(A, stream)
                                         : go_dim<kF32, 2>(A, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mx
