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
#include "paged_row.cuh"

namespace mita {
namespace {

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
  static constexpr int kThreads = kWarps * 32, kTeams = 1, kTeamThreads = kThreads;
  static constexpr int kRowBytes = D * (int)sizeof(T);
  static constexpr int kKeys = (kTensor || D <= 32 ? 32 : 16) / (D == 128 ? 2 : 1);  // of a warp
  using Mask = unsigned;
  static constexpr int kTile = kWarps * kKeys;
  static constexpr int kSegmentCost = kTensor ? 2 : 1;         // tiles that ending a segment is worth
  static constexpr int kChunks = kRowBytes / 16;               // 16-byte chunks of a row
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;    // K then V
  static constexpr int kStages =
      196608 / (kStageBytes * kWarps) > 8 ? 8 : 196608 / (kStageBytes * kWarps);
  static constexpr int kRing = kStages * kStageBytes;          // of one warp
  __device__ __forceinline__ static int warp() { return threadIdx.x >> 5; }
  static constexpr int kUnrollStart = kTensor ? 1 : kStages;
  // byte offsets
  static constexpr int kJoinBytes = kWarps * kRing;
  static constexpr int kOffMl = kJoinBytes;                               // [warps][RT][2]
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

// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 products summed in fp32
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
  bool plain;                        // the rule's, until a maximum is beyond kFar

  __device__ __forceinline__ void start(const PagedAttnArgs<bf16>& a, int s, int head, int rows,
                                        const ScoreRule& rule) {
    const int lane = threadIdx.x & 31;
    plain = rule.plain;
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

  // stage: the warp's key rows, then its value rows; key0 the first one's position; `mask` the seen ones
  __device__ __forceinline__ void tile(const ScoreRule& rule, uint32_t stage, int key0,
                                       unsigned mask) {
    const uint32_t kt = stage, vt = stage + S::kKeys * S::kRowBytes;
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
    if (!plain || mask != (unsigned)((1ull << S::kKeys) - 1)) {
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
        bool far = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = fmaxf(z[0][n][i], z[0][n][i + 2]);
#pragma unroll
          for (int t = 1; t < kT; ++t) top = fmaxf(top, fmaxf(z[t][n][i], z[t][n][i + 2]));
#pragma unroll
          for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          top = fmaxf(m[n][i], __fmul_rn(top, factor));
          f[i] = exp2_fast(m[n][i] - top);
          l[n][i] *= f[i];
          m[n][i] = top;
          far |= fabsf(top) > kFar && top > kLowest;
        }
        plain &= !__any_sync(0xffffffffu, far);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][n][i] *= f[i & 1];
      }
      if (!plain) {                  // (scores that are rounded already have a factor of one)
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[t][n][i] = __fmul_rn(z[t][n][i], factor);
        factor = 1.f;
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

  __device__ __forceinline__ void start(const PagedAttnArgs<float>& a, int s, int head, int rows,
                                        const ScoreRule&) {
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

  __device__ __forceinline__ void tile(const ScoreRule& rule, uint32_t stage, int key0,
                                       unsigned mask) {
    const uint32_t kt = stage, vt = stage + S::kKeys * S::kRowBytes;
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

// ---------------------------------------------------------------------------
// The warp's loader.  Where a page holds all of a warp's keys of a tile (they then lie one behind the
// other) one page number does for all; smaller pages are looked up row by row.
// ---------------------------------------------------------------------------
template <typename T, int D, int RT>
struct Loader : RowLoader<Shape<T, D, RT>, PagedAttnArgs<T>> {
  using S = Shape<T, D, RT>;
  using Rows = typename RowLoader<S, PagedAttnArgs<T>>::Rows;

  // copies looked-up rows to `stage`, notes which of them are seen, and commits
  __device__ __forceinline__ void issue(const PagedAttnArgs<T>& a, const Rows& r, uint32_t stage,
                                        unsigned* mask_out) const {
    const int lane = threadIdx.x & 31;
    const int page = r.page, key0 = r.key0, head = r.head;
    const unsigned mask = this->valid_keys(a, r);
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

template <typename T, int D, int RT> struct StateOf;
template <int D, int RT> struct StateOf<bf16, D, RT> { using type = TensorState<D, RT>; };
template <int D> struct StateOf<float, D, 8> { using type = SplitState<D>; };

template <typename T, int D, int RT>
struct Dense {
  using Type = T;
  using Args = PagedAttnArgs<T>;
  using S = Shape<T, D, RT>;
  using State = typename StateOf<T, D, RT>::type;
  using Ld = Loader<T, D, RT>;
  using Team = WholeCta;
  static constexpr int kD = D, kRT = RT;
  static auto kernel() { return paged_attn_kernel<Dense>; }
};

// The instantiation for a head dim, type and group: a CTA takes 8 query rows, in bf16 16 where the
// group has more; larger groups take several CTAs.
template <typename T, int RT, typename F>
auto with_dim(int d, F f) {
  switch (d) {
    case 16: return f(Run<Dense<T, 16, RT>>{});
    case 32: return f(Run<Dense<T, 32, RT>>{});
    case 64: return f(Run<Dense<T, 64, RT>>{});
    default: return f(Run<Dense<T, 128, RT>>{});
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
