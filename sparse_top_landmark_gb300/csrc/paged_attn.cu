// Attention of one new token per sequence over a paged key-value cache.
//
//   z_j = cap(scale * q . k_j) + slope * (j - (len - 1)),   cap(x) = softcap * tanh(x / softcap)
//   out = sum_j e^{z_j} v_j / sum_j e^{z_j}   over the keys j < len (the last `window` of them)
//
// One pass over keys and values with a running maximum and sum.  The G query heads of a key
// head read it together: they are the rows of the score tile.  Bound by HBM: 4 G D flops
// on 4 D bytes (bf16) for each key, far below the tensor cores' rate for any G this takes.
//
// Work is dealt out on the device, since lengths live there (a replayed graph sees new ones):
// every (sequence, key head, block of query rows) is a segment of tiles of kTile keys, the
// segments stand in one row, and each CTA takes an equal share of that row, whatever the lengths
// are.  Ending a segment takes a tile's time or two, so it counts as kSegmentCost tiles more.  A
// CTA finishes the segments that lie wholly in its share; of a segment that is cut it leaves a
// partial (maximum, sum, weighted values) in its first or its last slot of the workspace, and the
// CTA that is the last one to do so (a counter says which) joins the segment's partials in their
// order.  No sum is atomic: the result depends on the inputs alone.  (A second kernel for the joins
// took as long on the GPU and a launch more: 3.5 us of the host's time in each call.)
//
// A warp works on its own keys of each tile (kKeys) through its own ring of shared-memory stages,
// filled by 16-byte asynchronous copies some stages ahead, across the ends of segments; warps
// meet only where a segment ends.  Rows that are not to be seen (beyond the length, before the
// window, on an invalid page) are filled with zeros and never read: what the cache holds there,
// NaN included, reaches nothing.
//
// Measured (bf16): 128 sequences of up to 8192 keys, 32 query and 8 key heads of 128, in 311 us,
// 6.7 TB/s; one sequence of 1,048,575 keys, 8 and 2 heads of 64, in 88 us, 6.1 TB/s (loading alone
// takes 85 us); 200 of up to 900 keys, 32 and 8 heads of 128, in 72 us; one of 333 keys in 9.1 to 9.4 us,
// some 2.5 thousand cycles to find the share, as many to the first keys, 3.5 thousand for a first
// tile, 1.5 for its end, 2.5 for the count and 3 for a join.
#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mita.h"

namespace mita {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum before the first key: below every finite score, and finite, so that
// differences with it need no special case (a score of -inf weighs nothing against it).
constexpr float kLowest = -FLT_MAX;
constexpr int kMaxPagedCtas = 255;     // CTAs of a call, and counters in its workspace
// Counters carry the number of the call that counts, above the count's kCountBits bits: whatever an
// earlier call left in them is below this one's zero.  (Were a caller to change lengths while they are
// read, CTAs would disagree on how many parts a segment has, and a counter that a segment's join puts
// back to zero would stay where it is, for every later call.)  Behind the counters one word gives the
// calls their numbers: each call adds kCallStep to it, all of its CTAs 1 but the first one, which adds the
// rest; so whichever comes first, each finds the same multiple of kCallStep there.  Nothing has to
// be waited for or put back at the end of a call (333 keys 9.4 us; with a word that counts the CTAs that are
// done, the last of which clears the counters, 10.4 us, and 9.6 where no fence orders the two).
constexpr int kCallNumber = kMaxPagedCtas;
constexpr int kCallStep = 256;
constexpr int kCountBits = 16;
static_assert(kCallStep > kMaxPagedCtas, "a call's CTAs stay within its step");

// A cut segment whose parts are to be joined: the row of its first query, the CTA that begins it,
// its parts (0: nothing to do) and its query rows.
struct Join {
  long long row;
  int c, n, rows, unused;
};

// Shared memory and shape of one instantiation.  RT: query rows of a CTA.  A warp's stage is 8 KB
// (less for small heads: 32 keys are as many as a mask has bits): enough work behind each wait, and
// stages for 128 KB on the way to each SM (fp32, 64 sequences of up to 20000 keys of 32: 49 us with
// 16 keys, 38.5 us with 32).  Small heads leave registers for 16 warps (bf16, 67 sequences of up to
// 30515 keys of 32: 35 us with 8, 32 us with 16; fp32, the 64 with heads of 16: 32.5 and 29.4 us).
// (These choices of shape were measured before fp32 factors were rounded, which takes 5 % more.)
template <typename T, int D, int RT>
struct Shape {
  static constexpr bool kTensor = std::is_same<T, bf16>::value;
  static constexpr int kWarps = RT == 8 && D <= (kTensor ? 32 : 16) ? 16 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRowBytes = D * (int)sizeof(T);
  static constexpr int kKeys = (kTensor || D <= 32 ? 32 : 16) / (D == 128 ? 2 : 1);  // of a warp
  static constexpr int kTile = kWarps * kKeys;
  static constexpr int kSegmentCost = kTensor ? 2 : 1;         // tiles that ending a segment is worth
  static constexpr int kChunks = kRowBytes / 16;               // 16-byte chunks of a row
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;    // K then V
  static constexpr int kStages =
      196608 / (kStageBytes * kWarps) > 8 ? 8 : 196608 / (kStageBytes * kWarps);
  static constexpr int kRing = kStages * kStageBytes;          // of one warp
  // byte offsets
  static constexpr int kOffMl = kWarps * kRing;                           // [warps][RT][2]
  static constexpr int kOffMask = kOffMl + kWarps * RT * 8;               // [warps][stages]
  static constexpr int kOffJoins = kOffMask + (kWarps * kStages * 4 + 15) / 16 * 16;   // [2]
  static constexpr int kOffBase = kOffJoins + 2 * (int)sizeof(Join);     // of this call's counts
  static constexpr int kBytes = kOffBase + 16;
  static_assert(kBytes <= 232448 && kStages >= 3, "shared memory");
  static_assert(RT * D * 4 <= kStageBytes, "a warp's sums in one of its stages");
};

// Chunk c of row r lies at chunk c ^ f(r) of it, so that eight rows' equal chunks lie in
// eight different groups of banks.
template <int kRowBytes>
__device__ __forceinline__ int swizzle(int r, int c) {
  if constexpr (kRowBytes >= 128) return c ^ (r & 7);
  else if constexpr (kRowBytes == 64) return c ^ ((r >> 1) & 3);
  else return c ^ ((r >> 2) & 1);
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes, or zeros where `valid` is not set (src is then not read)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// An 8 x 8 matrix of 16-bit values, two of a row in a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 products summed in fp32
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// The row of tiles
// ---------------------------------------------------------------------------
// A sequence's seen keys [first, len), in tiles that start at multiples of `tile`.
struct Span {
  int first, len, base, tiles;
};
__device__ __forceinline__ Span span_of(const PagedLayout& pg, int window, int tile, int s) {
  Span r;
  const long long room = (long long)pg.width << pg.page_log2;
  r.len = (int)min((long long)max(pg.lengths[s], 0), room);
  r.first = window > 0 ? max(r.len - window, 0) : 0;
  r.base = r.first / tile * tile;
  r.tiles = (r.len - r.base + tile - 1) / tile;
  return r;
}

// A place in the row: tile `t` of segment (s, hr), hr = key head * row blocks + block; the segment
// begins at position `segment` of the row, and ends kSegmentCost positions after its last tile's.
struct Cursor {
  int s, hr, t;
  long long segment;
  Span span;
};

template <typename S>
__device__ __forceinline__ void advance(Cursor& c, const PagedLayout& pg, int window, int HR) {
  if (++c.t < c.span.tiles) return;
  c.t = 0;
  c.segment += c.span.tiles + S::kSegmentCost;
  if (++c.hr < HR) return;
  c.hr = 0;
  do {
    if (++c.s >= pg.S) {            // behind the last segment: behind every share
      c.segment = LLONG_MAX / 2;
      return;
    }
    c.span = span_of(pg, window, S::kTile, c.s);
  } while (c.span.tiles == 0);
}

__device__ __forceinline__ long long warp_incl_scan64(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// a / b, which are not negative: 64-bit division is some hundred instructions, and seldom needed.
__device__ __forceinline__ long long quotient(long long a, int b) {
  return a >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

__device__ __forceinline__ long long share_begin(long long row, int n, int c) {
  const long long q = quotient(row, n), r = row - q * n;
  return q * c + min((long long)c, r);
}
// The index of the CTA whose share of a row of that length has position x (one of the n, even where
// a caller changes lengths while they are read, and x lies anywhere).
__device__ __forceinline__ int share_of(long long x, long long row, int n) {
  const long long q = quotient(row, n), r = row - q * n;
  const long long large = r * (q + 1);       // the length of the r shares that are one longer
  if (q == 0) return (int)min(x, (long long)n - 1);
  return (int)min(x < large ? quotient(x, (int)q + 1) : r + quotient(x - large, (int)q),
                  (long long)n - 1);
}

// The length of the row, the place of this CTA's first tile, and the position where its share
// ends (a share may be empty, or hold ends of segments only: the first tile then lies behind).
// Each warp finds them for itself: a running sum over the sequences, of which those behind the
// first batch are summed ahead.
struct Share {
  long long row, end;
  Cursor at;
};
template <typename S>
__device__ __forceinline__ Share my_share(const PagedLayout& pg, int window, int HR) {
  const int lane = threadIdx.x & 31;
  constexpr int kEach = 4, kBatch = 32 * kEach;     // sequences of a lane, and of a warp, at a time
  auto cost_of = [&](int tiles) {
    return tiles > 0 ? (long long)(tiles + S::kSegmentCost) * HR : 0;
  };
  const int each = pg.S <= 32 ? 1 : kEach;
  int tiles[kEach];
  auto load = [&](int s0) {                         // its lane's tiles, and what they cost
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int s = s0 + lane * each + i;
      tiles[i] = i < each && s < pg.S ? span_of(pg, window, S::kTile, s).tiles : 0;
      sum += tiles[i] > 0 ? tiles[i] + S::kSegmentCost : 0;
    }
    return (long long)sum * HR;
  };
  long long rest = 0;                               // behind the first batch: mostly there is none
  for (int s0 = kBatch; s0 < pg.S; s0 += kBatch) rest += load(s0);
  if (pg.S > kBatch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
  }
  long long cost = load(0), incl = warp_incl_scan64(cost);
  Share sh;
  sh.row = __shfl_sync(0xffffffffu, incl, 31) + rest;
  const long long x = share_begin(sh.row, gridDim.x, blockIdx.x);
  sh.end = share_begin(sh.row, gridDim.x, blockIdx.x + 1);
  sh.at.segment = sh.row;
  sh.at.t = 0;
  if (x >= sh.end) return sh;
  int s0 = 0;
  unsigned hit;
  while ((hit = __ballot_sync(0xffffffffu, x < incl)) == 0) {
    const long long run = __shfl_sync(0xffffffffu, incl, 31);
    s0 += kBatch;
    if (s0 >= pg.S) return sh;
    cost = load(s0);
    incl = run + warp_incl_scan64(cost);
  }
  const int src = __ffs(hit) - 1;
  long long start = __shfl_sync(0xffffffffu, incl - cost, src);
  int n = __shfl_sync(0xffffffffu, tiles[0], src);
  sh.at.s = s0 + src * each;
  if (each > 1) {
#pragma unroll
    for (int i = 1; i < kEach; ++i) {
      const int next = __shfl_sync(0xffffffffu, tiles[i], src);
      if (sh.at.s == s0 + src * kEach + i - 1 && x - start >= cost_of(n)) {
        start += cost_of(n);
        n = next;
        ++sh.at.s;
      }
    }
  }
  const int seg = (int)quotient(x - start, n + S::kSegmentCost);
  sh.at.segment = start + (long long)seg * (n + S::kSegmentCost);
  const int in = (int)(x - sh.at.segment);
  sh.at.hr = seg;
  sh.at.t = min(in, n - 1);
  sh.at.span = span_of(pg, window, S::kTile, sh.at.s);
  if (in >= n) advance<S>(sh.at, pg, window, HR);   // it begins behind a segment's last tile
  return sh;
}

// What a tile's scores need besides q and k.
struct ScoreRule {
  float scale2;          // scale * log2(e): the scores of the running softmax are in log2 units
  float cap, rcap;       // softcap (0: none), scale / softcap
  int last;              // len - 1
  bool plain;            // scores are just scale2 * dot, with scale2 >= 0
};
// Below kSeries a capped score is its uncapped one times tanh(x) / x, x = score / softcap, by that
// function's Taylor series in x^2 (up to x^10: what is left out is below 2^-24 there).  So small scores
// under a large cap keep fp32's relative accuracy, and caps up to the largest number, where x itself
// underflows, leave the score as it is.
constexpr float kSeries = 0.4f;
__device__ __forceinline__ float tanh_ratio(float xx) {
  float p = fmaf(xx, -8.8632355e-3f, 2.1869489e-2f);      // -1382/155925, 62/2835
  p = fmaf(xx, p, -5.3968254e-2f);                        // -17/315
  p = fmaf(xx, p, 1.3333333e-1f);                         // 2/15
  p = fmaf(xx, p, -3.3333333e-1f);                        // -1/3
  return fmaf(xx, p, 1.f);
}
// tanh from one exponential and one reciprocal, to 2^-22 absolute: for |x| >= kSeries that is 2^-20 of
// the value, in a quarter of tanhf's instructions.
__device__ __forceinline__ float tanh_fast(float x) {
  const float e = exp2_fast(fabsf(x) * (2.f * kLog2e));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return copysignf(fmaf(-2.f, r, 1.f), x);
}
// The score where the cap's series does (the last 2092 keys of 53 sequences in bf16, cap 30: 37.1 us
// where every score computes both forms, 34.1 where a warp's tile takes this one if all its scores allow it;
// in fp32, 192 of up to 3783, 85.3 and 82.0).
__device__ __forceinline__ float score_near_zero(const ScoreRule& r, float dot, float slope2, int key) {
  const float x = dot * r.rcap;
  return dot * r.scale2 * tanh_ratio(x * x) + slope2 * (float)(key - r.last);
}
template <bool FAST>
__device__ __forceinline__ float score_of(const ScoreRule& r, float dot, float slope2, int key) {
  float z = dot * r.scale2;
  if (r.cap > 0.f) {
    const float x = dot * r.rcap;
    z = fabsf(x) < kSeries ? z * tanh_ratio(x * x)
                           : r.cap * (FAST ? tanh_fast(x) : tanhf(x)) * kLog2e;
  }
  return z + slope2 * (float)(key - r.last);
}

// ---------------------------------------------------------------------------
// One warp's running softmax, bf16 on the tensor cores.  Both products are taken transposed, keys
// and value columns on the matrix instruction's 16 rows and the query heads on its 8 columns: the
// group of a key head seldom has more than 8, and half of a 16-row tile would be padding.  (The
// queries on the 16 rows measured 334.9 us where this takes 330.9, 128 sequences of up to 8192 keys.)
// A lane has columns (lane % 4) * 2, + 1 of each eight query heads (those behind the last are
// zeros), and rows lane / 4, + 8 of every 16 keys or value columns.
// ---------------------------------------------------------------------------
template <int D, int RT>
struct TensorState {
  using S = Shape<bf16, D, RT>;
  static constexpr int kN = RT / 8;  // tiles of eight query heads
  uint32_t q[D / 16][kN][2];
  float o[D / 16][kN][4];
  float m[kN][2], l[kN][2];          // l: of this lane's keys
  float slope2[kN][2];

  __device__ __forceinline__ void start(const PagedAttnArgs<bf16>& a, int s, int head, int rows) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int r = 8 * n + lane / 4;
      const uint32_t* p = reinterpret_cast<const uint32_t*>(a.q + s * a.q_s +
                                                            (long long)(head + r) * a.q_h);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][n][0] = r < rows ? p[k * 8 + lane % 4] : 0u;
        q[k][n][1] = r < rows ? p[k * 8 + 4 + lane % 4] : 0u;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 8 * n + lane % 4 * 2 + i;
        slope2[n][i] = a.slopes && c < rows ? a.slopes[head + c] * kLog2e : 0.f;
        m[n][i] = kLowest;
        l[n][i] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][n][i] = 0.f;
    }
  }

  // kt, vt: the warp's key and value rows; key0 the first one's position; `mask` the seen ones
  __device__ __forceinline__ void tile(const ScoreRule& rule, uint32_t kt, uint32_t vt, int key0,
                                       unsigned mask) {
    constexpr int kT = S::kKeys / 16;
    const int lane = threadIdx.x & 31;
    float z[kT][kN][4] = {};
    {
      const int row = (lane & 7) + ((lane >> 3) & 1) * 8, c = lane >> 4;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          uint32_t x[4];
          ldsm4(kt + (row + 16 * t) * S::kRowBytes +
                    swizzle<S::kRowBytes>(row + 16 * t, 2 * k + c) * 16, x);
#pragma unroll
          for (int n = 0; n < kN; ++n) mma16816(z[t][n], x, q[k][n][0], q[k][n][1]);
        }
    }
    // z becomes the scores, or stays the dot products where a factor is all that is missing
    float factor = rule.scale2;
    if (!rule.plain || mask != (unsigned)((1ull << S::kKeys) - 1)) {
      factor = 1.f;
      bool small = rule.cap > 0.f;
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) small &= fabsf(z[t][n][i] * rule.rcap) < kSeries;
      if (__all_sync(0xffffffffu, small)) {
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 16 * t + lane / 4 + 8 * (i >> 1);
              z[t][n][i] = (mask >> j) & 1 ? score_near_zero(rule, z[t][n][i], slope2[n][i & 1], key0 + j)
                                           : -INFINITY;
            }
      } else {
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 16 * t + lane / 4 + 8 * (i >> 1);
              z[t][n][i] = (mask >> j) & 1 ? score_of<true>(rule, z[t][n][i], slope2[n][i & 1], key0 + j)
                                           : -INFINITY;
            }
      }
    }
    // The running maxima are looked for again only where a score is above them: most tiles
    // bring none, and need no exchange between lanes.
    bool above = false;
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) above |= fmaf(z[t][n][i], factor, -m[n][i & 1]) > 0.f;
    if (__any_sync(0xffffffffu, above)) {
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = fmaxf(z[0][n][i], z[0][n][i + 2]);
#pragma unroll
          for (int t = 1; t < kT; ++t) top = fmaxf(top, fmaxf(z[t][n][i], z[t][n][i + 2]));
#pragma unroll
          for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          top = fmaxf(m[n][i], top * factor);
          f[i] = exp2_fast(m[n][i] - top);
          l[n][i] *= f[i];
          m[n][i] = top;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][n][i] *= f[i & 1];
      }
    }
    // The weights go to the value product as a sum of two bf16 values, 16 bits in all: one alone
    // would add an error of the size of the output's own rounding, and the second product
    // is free where HBM is the bound.
    uint32_t hi[kT][kN][2], lo[kT][kN][2];
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = exp2_fast(fmaf(z[t][n][2 * i], factor, -m[n][0]));
          const float p1 = exp2_fast(fmaf(z[t][n][2 * i + 1], factor, -m[n][1]));
          l[n][0] += p0;
          l[n][1] += p1;
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
          const uint32_t h = *reinterpret_cast<const uint32_t*>(&h2);
          const __nv_bfloat162 e2 = __floats2bfloat162_rn(p0 - __uint_as_float(h << 16),
                                                          p1 - __uint_as_float(h & 0xffff0000u));
          hi[t][n][i] = transpose8(h);
          lo[t][n][i] = transpose8(*reinterpret_cast<const uint32_t*>(&e2));
        }
    {
      const int row = (lane & 7) + (lane >> 4) * 8, c = (lane >> 3) & 1;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        // The tensor cores cut sums instead of rounding them: over a long chain the values would lean
        // towards zero (100 thousand keys a warp: by 8e-4), so a tile's are added to the running ones
        // outside (128 sequences of up to 8192 keys: 307 us in one chain, 308 so).
        float sum[kN][4] = {};
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          uint32_t x[4];
          ldsm4_t(vt + (row + 16 * t) * S::kRowBytes +
                      swizzle<S::kRowBytes>(row + 16 * t, 2 * j + c) * 16, x);
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            mma16816(sum[n], x, hi[t][n][0], hi[t][n][1]);
            mma16816(sum[n], x, lo[t][n][0], lo[t][n][1]);
          }
        }
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][n][i] += sum[n][i];
      }
    }
  }

  // this warp's (maximum, sum) of every row
  __device__ __forceinline__ void put_ml(float2* ml) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], x);
        if (lane < 4) ml[8 * n + lane * 2 + i] = make_float2(m[n][i], l[n][i]);
      }
  }
  // column c of a row of sums lies at c ^ spread(row): put_o's four rows lie in different banks
  __device__ __forceinline__ static int spread(int r) { return ((r >> 1 & 3) * 8) & (D - 1); }
  // the rows below `rows`, moved to the maxima top(row), to dst[row][..]
  template <typename Top>
  __device__ __forceinline__ void put_o(float* dst, int rows, Top top) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * n + lane % 4 * 2 + i;
        if (r >= rows) continue;
        const float f = exp2_fast(m[n][i] - top(r));
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          dst[r * D + ((8 * j + lane / 4) ^ spread(r))] = o[j / 2][n][(j & 1) * 2 + i] * f;
      }
  }
};

// ---------------------------------------------------------------------------
// One warp's running softmax, fp32 on the tensor cores in tf32 (11 bits of a value).  Every value
// goes in as a sum of two, hi its upper 11 bits and lo = x - hi, of which the instruction uses the
// upper 11 of at most 13 bits.  It cuts the rest off, 3 units of x's last place at most and always
// towards zero, which leaned every score and every value; so lo is rounded, or hi is, so that lo
// has a bit less (below): 2 units at most, and none on average.  The error against fp64 is then that of
// fp32 arithmetic or less (4 x 8192 keys of 64, 3 heads, root mean square: 3.0e-7, cut 6.1e-7, products
// and sums in fp32 3.8e-7), for 2.5 % of the time where the tensor cores bound it (192 sequences of up
// to 3783 keys: 72.1 -> 73.9 us).  The 16 rows of the instruction hold
// the hi parts of eight query heads (or their weights) and below them the lo parts, so that two
// products with the hi and the lo part of the other side give all four terms, and a row and the
// one eight below it add up to the sum.
// The tensor cores cut sums instead of rounding them, so that long chains lose a little each time:
// a score is summed in four chains, and a tile's values are added to the running ones outside.
// A lane has query head lane / 4, and keys (lane % 4) * 2, + 1 of every eight.
// ---------------------------------------------------------------------------
template <int D>
struct SplitState {
  using S = Shape<float, D, 8>;
  static constexpr int kV = D >= 32 ? 4 : 2;   // value columns a lane reads at once
  static constexpr int kChains = D >= 64 ? 4 : 2;
  uint32_t q[D / 8][4];
  float o[D / 8][2];
  float m, l;            // l: of this lane's keys
  float slope2;
  const float* q_row;    // null behind the last query head

  // hi cut, lo rounded: q and the weights (of which there are few)
  __device__ __forceinline__ static void split(float x, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(x) & 0xffffe000u;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
  }
  // hi rounded, which leaves lo a sign and 12 bits, of which one is cut: keys.  (From 2^-12 below the
  // largest number on hi is infinite, the score NaN, and so done again below.)
  __device__ __forceinline__ static void split_key(float x, uint32_t& hi, uint32_t& lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
  }
  // hi cut, lo made larger by 3/8 to 3/4 of a unit of its eleventh bit, so that the cut rounds it: values.
  // (An infinite hi could not be done again; a rounding instruction takes 1 us more in 74.)
  __device__ __forceinline__ static void split_value(float x, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint((x - __uint_as_float(hi)) * 1.0003662109375f);    // 1 + 3 / 2^13
  }
  // c[16 x 8] += a[16 x 8] b[8 x 8], tf32 products
  __device__ __forceinline__ static void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }

  __device__ __forceinline__ void start(const PagedAttnArgs<float>& a, int s, int head, int rows) {
    const int lane = threadIdx.x & 31, r = lane / 4;
    const float* p = a.q + s * a.q_s + (long long)(head + r) * a.q_h;
#pragma unroll
    for (int k = 0; k < D / 8; ++k) {
      split(r < rows ? p[k * 8 + lane % 4] : 0.f, q[k][0], q[k][1]);
      split(r < rows ? p[k * 8 + 4 + lane % 4] : 0.f, q[k][2], q[k][3]);
    }
    q_row = r < rows ? p : nullptr;
    slope2 = a.slopes && r < rows ? a.slopes[head + r] * kLog2e : 0.f;
    m = kLowest;
    l = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = 0.f;
  }

  static __device__ __noinline__ float plain_dot(const float* q_row, uint32_t kt, int row) {
    float sum = 0.f;
    if (q_row == nullptr) return sum;
    for (int c = 0; c < D; ++c) {
      float k;
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(k)
                   : "r"(kt + row * S::kRowBytes + swizzle<S::kRowBytes>(row, c / 4) * 16 + c % 4 * 4)
                   : "memory");
      sum = fmaf(q_row[c], k, sum);
    }
    return sum;
  }

  __device__ __forceinline__ void tile(const ScoreRule& rule, uint32_t kt, uint32_t vt, int key0,
                                       unsigned mask) {
    constexpr int kT = S::kKeys / 8;
    const int lane = threadIdx.x & 31;
    float z[kT][2];
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float c[kChains][4] = {};
      const int row = 8 * t + (lane & 7);
#pragma unroll
      for (int k = 0; k < D / 8; k += 2) {
        uint32_t b[4], lo[4];
        ldsm4(kt + row * S::kRowBytes + swizzle<S::kRowBytes>(row, 2 * k + (lane >> 3)) * 16, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) split_key(__uint_as_float(b[i]), b[i], lo[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma(c[(k + i) % kChains], q[k + i], b[2 * i], b[2 * i + 1]);
          mma(c[(k + i) % kChains], q[k + i], lo[2 * i], lo[2 * i + 1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        z[t][i] = 0.f;
#pragma unroll
        for (int x = 0; x < kChains; ++x) z[t][i] += c[x][i] + c[x][i + 2];
      }
    }
    // An infinite key or query value has no parts: where a sum came out NaN it is done again in
    // plain fp32.
    bool odd = false;
#pragma unroll
    for (int t = 0; t < kT; ++t) odd |= isnan(z[t][0]) || isnan(z[t][1]);
    if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (isnan(z[t][i])) z[t][i] = plain_dot(q_row, kt, 8 * t + lane % 4 * 2 + i);
    }
    bool small = rule.cap > 0.f;
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) small &= fabsf(z[t][i] * rule.rcap) < kSeries;
    const bool series = __all_sync(0xffffffffu, small);
    bool above = false;
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = 8 * t + lane % 4 * 2 + i;
        z[t][i] = rule.plain ? z[t][i] * rule.scale2
                  : series   ? score_near_zero(rule, z[t][i], slope2, key0 + j)
                             : score_of<false>(rule, z[t][i], slope2, key0 + j);
        if (!((mask >> j) & 1)) z[t][i] = -INFINITY;
        above |= z[t][i] > m;
      }
    if (__any_sync(0xffffffffu, above)) {
      float top = m;
#pragma unroll
      for (int t = 0; t < kT; ++t) top = fmaxf(top, fmaxf(z[t][0], z[t][1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float f = exp2_fast(m - top);
      m = top;
      l *= f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][0] *= f;
        o[j][1] *= f;
      }
    }
    // The weights are the left operand as they lie if its eight keys are taken in the order 0, 2,
    // 4, 6, 1, 3, 5, 7, and so are the value rows: lane % 4 reads rows 2 (lane % 4) and + 1.
    uint32_t p[kT][4];
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float w = exp2_fast(z[t][i] - m);
        l += w;
        split(w, p[t][2 * i], p[t][2 * i + 1]);
      }
    // columns of the values in the order that lets a lane read kV at once: column n of product
    // kV * g + x is column 8 kV g + kV n + x of the row
#pragma unroll
    for (int g = 0; g < D / 8 / kV; ++g) {
      float c[kV][4] = {};
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        float v[2][kV];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 8 * t + lane % 4 * 2 + i, col = 8 * kV * g + kV * (lane / 4);
          const uint32_t at = vt + row * S::kRowBytes +
                              swizzle<S::kRowBytes>(row, col / 4) * 16 + col % 4 * 4;
          if constexpr (kV == 4)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[i][0]), "=f"(v[i][1]), "=f"(v[i][2]), "=f"(v[i][3])
                         : "r"(at)
                         : "memory");
          else
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                         : "=f"(v[i][0]), "=f"(v[i][1])
                         : "r"(at)
                         : "memory");
        }
#pragma unroll
        for (int x = 0; x < kV; ++x) {
          uint32_t h0, h1, l0, l1;
          split_value(v[0][x], h0, l0);
          split_value(v[1][x], h1, l1);
          mma(c[x], p[t], h0, h1);
          mma(c[x], p[t], l0, l1);
        }
      }
#pragma unroll
      for (int x = 0; x < kV; ++x) {
        o[kV * g + x][0] += c[x][0] + c[x][2];
        o[kV * g + x][1] += c[x][1] + c[x][3];
      }
    }
  }

  __device__ __forceinline__ void put_ml(float2* ml) {
    const int lane = threadIdx.x & 31;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (lane % 4 == 0) ml[lane / 4] = make_float2(m, l);
  }
  __device__ __forceinline__ static int spread(int r) { return r & 7; }   // eight rows
  template <typename Top>
  __device__ __forceinline__ void put_o(float* dst, int rows, Top top) const {
    const int lane = threadIdx.x & 31, r = lane / 4;
    if (r >= rows) return;
    const float f = exp2_fast(m - top(r));
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = 8 * kV * (j / kV) + kV * (lane % 4 * 2 + i) + j % kV;
        dst[r * D + (col ^ spread(r))] = o[j][i] * f;
      }
  }
};

// ln of a sum that is kept relative to 2^base; -inf of an empty one
__device__ __forceinline__ float lse_of(float base, float sum) {
  return sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
}
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }

// ---------------------------------------------------------------------------
// The warp's loader: page numbers one tile ahead of the copies, copies kStages - 1 tiles
// ahead of the arithmetic.  Where a page holds all of a warp's keys of a tile (they then lie one
// behind the other) one page number does for all; smaller pages are looked up row by row.
// ---------------------------------------------------------------------------
template <typename T, int D, int RT>
struct Loader {
  using S = Shape<T, D, RT>;
  Cursor at;
  long long end;           // of the share
  struct Rows {            // a warp's keys of a tile
    int page, key0, head;  // page: of this lane's key
    unsigned mask;         // those to be seen
  };

  __device__ __forceinline__ Rows look_up(const PagedAttnArgs<T>& a, int HR) {
    int page = 0, key0 = 0, head = 0;
    unsigned mask = 0;
    if (at.segment + at.t >= end) return {0, 0, 0, 0};
    const int warp = threadIdx.x >> 5;
    key0 = at.span.base + at.t * S::kTile + warp * S::kKeys;
    const int lo = max(at.span.first - key0, 0), hi = min(at.span.len - key0, S::kKeys);
    if (lo < hi) {
      constexpr unsigned kAll = (unsigned)((1ull << S::kKeys) - 1);
      mask = (kAll << lo) & (kAll >> (S::kKeys - hi));
      head = a.row_blocks == 1 ? at.hr : at.hr / a.row_blocks;
      // lanes whose key is not to be seen read the first one's page
      const int mine = (threadIdx.x & 31) % S::kKeys;
      const int key = key0 + ((mask >> mine) & 1 ? mine : lo);
      page = a.paged.table[(long long)at.s * a.paged.width + (key >> a.paged.page_log2)];
    }
    advance<S>(at, a.paged, a.window, HR);
    return {page, key0, head, mask};
  }

  // copies looked-up rows to `stage`, notes which of them are seen, and commits
  __device__ __forceinline__ void issue(const PagedAttnArgs<T>& a, const Rows& r, uint32_t stage,
                                        unsigned* mask_out) const {
    const int lane = threadIdx.x & 31;
    const int page = r.page, key0 = r.key0, head = r.head;
    unsigned mask = r.mask;
    if (mask) {
      const bool bad = page < 0 || page >= a.paged.num_pages;
      const unsigned wrong = __ballot_sync(0xffffffffu, bad);
      if (wrong) {
        if (lane == 0) flag_error(a.status, kDevErrBadIndex);
        mask &= ~wrong;
      }
    }
    if (lane == 0) *mask_out = mask;
    if (mask) {
      constexpr int kPerPass = 32 / S::kChunks;      // rows a warp copies at once
      constexpr int kPasses = S::kKeys / kPerPass;
      const int c = lane % S::kChunks, r0 = lane / S::kChunks;
      const int log2 = a.paged.page_log2, in_page = (1 << log2) - 1;
      if ((1 << log2) >= S::kKeys) {
        const long long first = ((((long long)page * a.Hkv + head) << log2) + (key0 & in_page)) * D;
        const long long off = first + r0 * D + c * (16 / (int)sizeof(T));
        const T *k = a.k_cache + off, *v = a.v_cache + off;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int row = i * kPerPass + r0;
          const uint32_t dst = stage + row * S::kRowBytes + swizzle<S::kRowBytes>(row, c) * 16;
          const bool live = (mask >> row) & 1;
          copy16(dst, k + i * kPerPass * D, live);
          copy16(dst + S::kKeys * S::kRowBytes, v + i * kPerPass * D, live);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int row = i * kPerPass + r0;
          const int pg = __shfl_sync(0xffffffffu, page, row);
          const bool live = (mask >> row) & 1;
          const long long at_row = (((long long)pg * a.Hkv + head) << log2) +
                                   ((key0 + row) & in_page);
          const long long off = live ? at_row * D + c * (16 / (int)sizeof(T)) : 0;
          const uint32_t dst = stage + row * S::kRowBytes + swizzle<S::kRowBytes>(row, c) * 16;
          copy16(dst, a.k_cache + off, live);
          copy16(dst + S::kKeys * S::kRowBytes, a.v_cache + off, live);
        }
      }
    }
    copy_commit();
  }
};

// Adds this CTA's part to the word that numbers the calls; returns what it was.
__device__ __forceinline__ unsigned long long count_call(unsigned long long* number) {
  const unsigned long long mine = blockIdx.x == 0 ? kCallStep - (gridDim.x - 1) : 1;
  unsigned long long old;
  asm volatile("atom.relaxed.gpu.global.add.u64 %0, [%1], %2;"
               : "=l"(old)
               : "l"(number), "l"(mine)
               : "memory");
  return old;
}
// Counts one up from `base`, this call's zero, after what this CTA's threads wrote before their last
// barrier, and before what they read after the next one; returns the count before.
__device__ __forceinline__ int count_up(unsigned long long* counter, unsigned long long base) {
  unsigned long long old;
  asm volatile("red.relaxed.gpu.global.max.u64 [%0], %1;" ::"l"(counter), "l"(base) : "memory");
  asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], 1;"
               : "=l"(old)
               : "l"(counter)
               : "memory");
  return (int)(old - base);
}

// Joins the partials of a cut segment, all of them written: the beginning is CTA c's last part, the
// rest the first parts of CTAs c + 1 .. c + n - 1; out and lse: the segment's rows.  Called by a
// whole CTA (out of line: it should not cost the tile loop registers); `mem`: shared, of
// kThreads * 4 + kGroups * 2 floats.
// D / 4 threads take four columns of a row's parts, kAhead of them on their way at a time, with a
// running maximum; where there are fewer rows than such groups of threads, a row's parts are dealt
// to several groups, which are then joined in their order.
template <typename T, int D, int RT, int kThreads>
__device__ __noinline__ void join_parts(const float* part_ml, const float* part_o, T* out,
                                        float* lse, int c, int n, int rows, float* mem) {
  constexpr int kLanes = D / 4, kGroups = kThreads / kLanes, kAhead = RT == 16 ? 16 : 6;
  float4* sums = reinterpret_cast<float4*>(mem);               // [groups][D / 4]
  float2* totals = reinterpret_cast<float2*>(mem + kThreads * 4);   // [groups] (maximum, sum)
  static_assert((kThreads * 4 + kGroups * 2) * 4 <= Shape<T, D, RT>::kOffMl, "shared memory");
  const int group = threadIdx.x / kLanes, col = threadIdx.x % kLanes;
  for (int r0 = 0; r0 < rows; r0 += kGroups) {
    const int now = min(rows - r0, kGroups), share = kGroups / now;
    const int row = group / share, first = group - row * share;
    if (row < now) {
      float base = kLowest, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = first; i0 < n; i0 += share * kAhead) {
        float2 x[kAhead];
        float4 v[kAhead];
        float top = base;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + k * share;
          // written by other CTAs while this one ran: read past the L1
          const long long at = (long long)(i == 0 ? c * 2 + 1 : (c + i) * 2) * RT + r0 + row;
          x[k] = make_float2(kLowest, 0.f);
          v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < n) {
            x[k] = __ldcg(reinterpret_cast<const float2*>(part_ml) + at);
            v[k] = __ldcg(reinterpret_cast<const float4*>(part_o) + at * kLanes + col);
          }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) top = fmaxf(top, x[k].x);
        const float f = exp2_fast(base - top);
        base = top;
        sum *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float w = exp2_fast(x[k].x - top);
          sum = fmaf(w, x[k].y, sum);
          acc.x = fmaf(w, v[k].x, acc.x);
          acc.y = fmaf(w, v[k].y, acc.y);
          acc.z = fmaf(w, v[k].z, acc.z);
          acc.w = fmaf(w, v[k].w, acc.w);
        }
      }
      sums[threadIdx.x] = acc;
      if (col == 0) totals[group] = make_float2(base, sum);
    }
    __syncthreads();
    if (row < now && first == 0) {
      float base = kLowest, sum = 0.f;
      for (int g = 0; g < share; ++g) base = fmaxf(base, totals[group + g].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int g = 0; g < share; ++g) {
        const float2 x = totals[group + g];
        const float4 v = sums[threadIdx.x + g * kLanes];
        const float w = exp2_fast(x.x - base);
        sum = fmaf(w, x.y, sum);
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      T* to = out + (long long)(r0 + row) * D + col * 4;
      to[0] = from_f<T>(acc.x * inv);
      to[1] = from_f<T>(acc.y * inv);
      to[2] = from_f<T>(acc.z * inv);
      to[3] = from_f<T>(acc.w * inv);
      if (lse && col == 0) lse[r0 + row] = lse_of(base, sum);
    }
    __syncthreads();
  }
}

template <typename T, int D, int RT> struct StateOf;
template <int D, int RT> struct StateOf<bf16, D, RT> { using type = TensorState<D, RT>; };
template <int D> struct StateOf<float, D, 8> { using type = SplitState<D>; };

// Brings a segment's query rows near, ahead of State::start.
template <typename T, int D, int RT>
__device__ __forceinline__ void prefetch_q(const PagedAttnArgs<T>& a, const Cursor& at) {
  const int kv = a.row_blocks == 1 ? at.hr : at.hr / a.row_blocks;
  const int rb = at.hr - kv * a.row_blocks;
  constexpr int kLines = (D * (int)sizeof(T) + 127) / 128;      // of a row
  const int r = (int)threadIdx.x / kLines;
  if (r < min(RT, a.G - rb * RT)) {
    const char* p = reinterpret_cast<const char*>(
        a.q + at.s * a.q_s + (long long)(kv * a.G + rb * RT + r) * a.q_h);
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p + threadIdx.x % kLines * 128));
  }
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(Shape<T, D, RT>::kThreads, 1)
paged_attn_kernel(const __grid_constant__ PagedAttnArgs<T> a) {
  using S = Shape<T, D, RT>;
  using State = typename StateOf<T, D, RT>::type;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int HR = a.Hkv * a.row_blocks, Hq = a.Hkv * a.G;
  uint8_t* ring = smem + warp * S::kRing;
  float2* ml = reinterpret_cast<float2*>(smem + S::kOffMl);
  unsigned* masks = reinterpret_cast<unsigned*>(smem + S::kOffMask) + warp * S::kStages;
  // of the segment that another CTA begins, and of the one that another CTA ends
  Join* joins = reinterpret_cast<Join*>(smem + S::kOffJoins);

  griddep_wait();
  griddep_launch();
  unsigned long long call = 0;
  if (threadIdx.x == 0) call = count_call(a.counters + kCallNumber);     // looked at further below
  const Share share = my_share<S>(a.paged, a.window, HR);
  Cursor at = share.at;
  if (threadIdx.x < 2) joins[threadIdx.x] = {};        // read behind the barriers of the share's end
  if (at.segment + at.t < share.end) {
    prefetch_q<T, D, RT>(a, at);
    using Ld = Loader<T, D, RT>;
    Ld ld;
    ld.at = at;
    ld.end = share.end;
    typename Ld::Rows rows_of[S::kStages];
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) rows_of[i] = ld.look_up(a, HR);   // their loads together
    // Not unrolled in bf16: a short call waits for its instructions (333 keys: 9.3 us unrolled, 9.1 us
    // so; fp32 loses as much in long ones).
#pragma unroll(S::kTensor ? 1 : S::kStages)
    for (int i = 0; i < S::kStages - 1; ++i) {
      ld.issue(a, rows_of[0], smem_addr(ring) + i * S::kStageBytes, masks + i);
#pragma unroll
      for (int j = 1; j < S::kStages; ++j) rows_of[j - 1] = rows_of[j];
    }
    typename Ld::Rows coming = rows_of[0];
    // thread 0's alone, kept where it takes no registers
    auto* const base = reinterpret_cast<unsigned long long*>(smem + S::kOffBase);
    if (threadIdx.x == 0) *base = call / kCallStep << kCountBits;
    State st;
    ScoreRule rule;
    rule.scale2 = a.scale * kLog2e;
    rule.cap = a.softcap;
    // finite, so that a score of zero stays one under the smallest caps too
    rule.rcap = a.softcap > 0.f ? fminf(fmaxf(a.scale / a.softcap, -FLT_MAX), FLT_MAX) : 0.f;
    rule.plain = a.softcap == 0.f && a.slopes == nullptr && a.scale >= 0.f;
    int slot = 0, next = S::kStages - 1;     // stages: of this tile, of the next one to issue
    int from = at.t, head = 0, rows = 0;
    bool begin = true;
    do {
      if (begin) {
        const int kv = a.row_blocks == 1 ? at.hr : at.hr / a.row_blocks;
        const int rb = at.hr - kv * a.row_blocks;
        head = kv * a.G + rb * RT;
        rows = min(RT, a.G - rb * RT);
        rule.last = at.span.len - 1;
        from = at.t;
        st.start(a, at.s, head, rows);
        begin = false;
      }
      copy_wait<S::kStages - 2>();
      __syncwarp();
      ld.issue(a, coming, smem_addr(ring) + next * S::kStageBytes, masks + next);
      coming = ld.look_up(a, HR);
      const unsigned mask = masks[slot];
      if (mask) {
        const uint32_t stage = smem_addr(ring) + slot * S::kStageBytes;
        st.tile(rule, stage, stage + S::kKeys * S::kRowBytes,
                at.span.base + at.t * S::kTile + warp * S::kKeys, mask);
      }

      const bool ends = at.t + 1 == at.span.tiles;
      if (ends || at.segment + at.t + 1 == share.end) {
        // join the warps' parts: every row's sums are added by one warp
        Cursor then = at;
        advance<S>(then, a.paged, a.window, HR);
        if (ends && then.segment < share.end) prefetch_q<T, D, RT>(a, then);
        st.put_ml(ml + warp * RT);
        __syncthreads();
        const bool whole = ends && from == 0;
        const int part = blockIdx.x * 2 + (from == 0 ? 1 : 0);
        auto top = [&](int r) {
          float t = ml[r].x;
#pragma unroll
          for (int w = 1; w < S::kWarps; ++w) t = fmaxf(t, ml[w * RT + r].x);
          return t;
        };
        // Every warp's sums go to the stage that it has just read: no copy goes there until its
        // next tile.
        float* const sums = reinterpret_cast<float*>(smem + slot * S::kStageBytes);
        st.put_o(sums + warp * (S::kRing / 4), rows, top);
        __syncthreads();
        for (int r = warp; r < rows; r += S::kWarps) {
          const float base = top(r);
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < S::kWarps; ++w) {
            const float2 x = ml[w * RT + r];
            sum = fmaf(x.y, exp2_fast(x.x - base), sum);
          }
          if (lane == 0) {
            if (!whole)
              reinterpret_cast<float2*>(a.part_ml)[(long long)part * RT + r] =
                  make_float2(base, sum);
            else if (a.lse)
              a.lse[(long long)at.s * Hq + head + r] = lse_of(base, sum);
          }
          const float inv = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
          T* out = a.out + ((long long)at.s * Hq + head + r) * D;
          float* part_o = a.part_o + ((long long)part * RT + r) * D;
#pragma unroll
          for (int c = lane; c < D; c += 32) {
            const float* from_w = sums + r * D + (c ^ State::spread(r));
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) x += from_w[w * (S::kRing / 4)];
            if (whole) out[c] = from_f<T>(x * inv);
            else part_o[c] = x;
          }
        }
        __syncthreads();
        if (!whole && threadIdx.x == 0) {
          // Whoever leaves a segment's last part joins them all, when its own share is done (the
          // others go on meanwhile): the count is asked for now, and looked at then.
          const int c0 = from == 0 ? (int)blockIdx.x : share_of(at.segment, share.row, gridDim.x);
          const int n = share_of(at.segment + at.span.tiles - 1, share.row, gridDim.x) - c0 + 1;
          const bool last = count_up(a.counters + c0, *base) == n - 1;
          joins[from == 0] = {(long long)at.s * Hq + head, c0, last ? n : 0, rows, 0};
        }
        begin = true;
      }
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
      next = next + 1 == S::kStages ? 0 : next + 1;
      advance<S>(at, a.paged, a.window, HR);
    } while (at.segment + at.t < share.end);
    copy_wait<0>();
    __syncthreads();
    for (int i = 0; i < 2; ++i) {
      const Join x = joins[i];
      if (x.n == 0) continue;
      join_parts<T, D, RT, S::kThreads>(a.part_ml, a.part_o, a.out + x.row * D,
                                        a.lse ? a.lse + x.row : nullptr, x.c, x.n, x.rows,
                                        reinterpret_cast<float*>(smem));
    }
  }
  // sequences without a key: zeros, and the logarithm of an empty sum
  for (int s = blockIdx.x; s < a.paged.S; s += gridDim.x) {
    const int len = a.paged.lengths[s];
    if (threadIdx.x == 0 && (len < 0 || len > (long long)a.paged.width << a.paged.page_log2))
      flag_error(a.status, kDevErrBadIndex);
    if (len > 0 && a.paged.width > 0) continue;
    for (int e = threadIdx.x; e < Hq * D; e += S::kThreads)
      a.out[(long long)s * Hq * D + e] = from_f<T>(0.f);
    if (a.lse)
      for (int e = threadIdx.x; e < Hq; e += S::kThreads) a.lse[(long long)s * Hq + e] = -INFINITY;
  }
}

// CTAs for this call: one on each SM, but no more than there can be tiles.
template <typename T, int D, int RT>
int grid_of(int S, int width, int page_log2, int HR, int sms) {
  using Sh = Shape<T, D, RT>;
  const long long keys = (long long)width << page_log2;
  const long long tiles = (keys + Sh::kTile - 1) / Sh::kTile * HR * (long long)S;
  return (int)std::max<long long>(1, std::min<long long>({(long long)sms, tiles, kMaxPagedCtas}));
}

// The counters come first and in the same place for every shape: calls of different shapes can
// have one workspace.
struct Carve {
  size_t ml, o, total;
};
Carve carve(int ctas, int RT, int D) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  Carve c{};
  static_assert((kCallNumber + 1) * sizeof(long long) == MITA_PAGED_COUNTERS, "counters");
  c.ml = MITA_PAGED_COUNTERS;
  c.o = c.ml + up((size_t)ctas * 2 * RT * 2 * sizeof(float));
  c.total = c.o + up((size_t)ctas * 2 * RT * D * sizeof(float));
  return c;
}

template <typename T, int D, int RT>
struct Run {
  static size_t bytes(int Hkv, int G, int S, int width, int page_log2, int sms) {
    const int HR = Hkv * ((G + RT - 1) / RT);
    return carve(grid_of<T, D, RT>(S, width, page_log2, HR, sms), RT, D).total;
  }
  // the kernel's shared memory, allowed once for each device
  static cudaError_t allow_shared() {
    static std::atomic<unsigned long long> allowed{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (allowed.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(paged_attn_kernel<T, D, RT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Shape<T, D, RT>::kBytes);
    if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
  static cudaError_t launch(PagedAttnArgs<T> a, void* ws, int sms, cudaStream_t st) {
    using Sh = Shape<T, D, RT>;
    a.row_blocks = (a.G + RT - 1) / RT;
    const int grid = grid_of<T, D, RT>(a.paged.S, a.paged.width, a.paged.page_log2,
                                       a.Hkv * a.row_blocks, sms);
    const Carve c = carve(grid, RT, D);
    a.counters = static_cast<unsigned long long*>(ws);
    a.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + c.ml);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + c.o);
    cudaError_t e = allow_shared();
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_pdl(paged_attn_kernel<T, D, RT>, dim3(grid), dim3(Sh::kThreads), Sh::kBytes, st,
                      a);
  }
};

// The instantiation for a head dim, type and group: a CTA takes 8 query rows, in bf16 16 where the
// group has more; larger groups take several CTAs.
template <typename T, int RT, typename F>
auto with_dim(int d, F f) {
  switch (d) {
    case 16: return f(Run<T, 16, RT>{});
    case 32: return f(Run<T, 32, RT>{});
    case 64: return f(Run<T, 64, RT>{});
    default: return f(Run<T, 128, RT>{});
  }
}
template <typename T, typename F>
auto with_shape(int d, int G, F f) {
  if constexpr (std::is_same<T, bf16>::value) {
    if (G > 8) return with_dim<T, 16>(d, f);
  }
  return with_dim<T, 8>(d, f);
}

}  // namespace

size_t paged_attn_ws_bytes(int d, int Hkv, int G, int S, int width, int page_log2, int is_f32,
                           int sms) {
  auto bytes = [&](auto run) { return run.bytes(Hkv, G, S, width, page_log2, sms); };
  return is_f32 ? with_shape<float>(d, G, bytes) : with_shape<bf16>(d, G, bytes);
}

template <typename T>
cudaError_t launch_paged_attn(PagedAttnArgs<T> a, int d, void* ws, int sms, cudaStream_t st) {
  return with_shape<T>(d, a.G, [&](auto run) { return run.launch(a, ws, sms, st); });
}

template cudaError_t launch_paged_attn<float>(PagedAttnArgs<float>, int, void*, int, cudaStream_t);
template cudaError_t launch_paged_attn<bf16>(PagedAttnArgs<bf16>, int, void*, int, cudaStream_t);

}  // namespace mita
