// Attention of one new token per sequence over a paged key-value cache of 4-bit codes.  What it computes,
// and how the work is dealt out, are those of paged_attn.cu.
//
// A value of the cache is (n - 8) s: a code n of 0 .. 15 and a scale s for 32 values of a row, E5M3 (the
// upper bits of an fp16 number without its sign: a shift by seven turns it into one).  A row's 32-value
// chunks of 16 bytes stand in the order that lets ldmatrix read eight rows from different banks.
//
// Both products run on the tensor cores in fp16, keys (or value columns) on the instruction's 16 rows.
// ldmatrix takes 16-bit words of four codes, four values of a row, for its elements; with .trans it pairs
// the words of two keys, which is what the value product needs.  The order in which a chunk's values
// then meet the instruction is put into the queries (keys) and the accumulators (values).  Two codes
// become an operand by a mask, and a shift for every other pair:
//
// - keys (bf16): as the bits of an fp16 number a code n is the subnormal n * 2^-24 and n << 4 is 16 n * 2^-24;
//   the 16 is taken out of the queries (an exact division), and the 8 out of the sum where it begins:
//   z = sum over chunks c of s_c (-8 sum_i q_i + sum_i n_i q_i).
// - values, and keys in fp32: 1024's bits above the code, and one fp16 instruction that leaves n - 8.  (The
//   tensor cores cut sums.  Taken as n p from a sum of -8 p, a long context's values, which nearly
//   cancel, lean by 2^-23 of eight times the sum of the weights for every product: 4.8e-6 of an fp32 result
//   at 1000 keys, 1e-3 at a million.)
//
// Queries are scaled by a power of two, their row's largest to 2^14, so that fp16 holds what bf16 does,
// down to 2^-38 of it; weights p are at most 2^15, so that fp16's subnormals begin at 2^-29 of a
// weight's range.  Scales are at most 2 mostly, and p s then stays below fp16's end; where a tile holds
// a larger one, its weights are made smaller by a power of two that is put back where the tile's sums are
// added to the running ones (in fp32, outside the tensor cores: paged_attn.cu says why).  The bf16 twin
// rounds a weight and its product with the scale to fp16's 11 bits; the fp32 twin gives every query and
// every p s as a sum of two fp16 values, 22 bits.
#include "paged_row.cuh"

#include <cuda_fp16.h>

namespace mita {
namespace {

constexpr float kBoost = 15.f;       // log2 of the largest weight

template <typename T, int D, int RT>
struct Q4Shape {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kKeys = 32;                        // of a warp: as many as a mask has bits
  static constexpr int kTile = kWarps * kKeys;
  static constexpr int kSegmentCost = 2;                  // tiles that ending a segment is worth
  static constexpr int kUnrollStart = 1;
  static constexpr int kChunks = D / kQ4Block;            // of a row: 16 bytes and one scale each
  static constexpr int kRowBytes = D / 2;
  static constexpr int kCodes = kKeys * kRowBytes, kScales = kKeys * kChunks;
  static constexpr int kStageBytes = 2 * (kCodes + kScales);      // K's codes, V's, K's scales, V's
  // a warp's sums at an end have a place of their own where a stage does not hold them
  static constexpr bool kOwnSums = RT * D * 4 > kStageBytes;
  static constexpr int kSumBytes = kOwnSums ? kWarps * RT * D * 4 : 0;
  static constexpr int kFit = (196608 - kSumBytes) / (kStageBytes * kWarps);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kOffSums = kOwnSums ? kWarps * kRing : -1;
  static constexpr int kSums = kOwnSums ? RT * D * 4 : kRing;
  static constexpr int kOffMl = kWarps * kRing + kSumBytes;               // [warps][RT][2]
  static constexpr int kOffMask = kOffMl + kWarps * RT * 8;               // [warps][stages]
  static constexpr int kOffJoins = kOffMask + (kWarps * kStages * 4 + 15) / 16 * 16;   // [2]
  static constexpr int kOffBase = kOffJoins + 2 * (int)sizeof(Join);
  static constexpr int kBytes = kOffBase + 16;
  static_assert(kBytes <= 232448 && kStages >= 3 && kStageBytes % 16 == 0, "shared memory");
};

// Chunk c of row r of a page stands at c ^ q4_turn(r).
template <int D>
__device__ __forceinline__ int q4_turn(int r) {
  return D == 128 ? (r >> 1) & 3 : D == 64 ? (r >> 2) & 1 : 0;
}

// c[16 x 8] += a[16 x 16] b[16 x 8], fp16 products summed in fp32
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ uint32_t fma_half(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_half(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Codes 0 and 1 of the two 16-bit words of x (of x >> 8: 2 and 3), as fp16 numbers n * 2^-24 and
// 16 n * 2^-24, or, kSigned, n - 8: with 1024's bits above it a code is 1024 + n or 1024 + 16 n.
template <bool kSigned>
__device__ __forceinline__ uint32_t code_lo(uint32_t x) {
  if constexpr (!kSigned) return x & 0x000f000fu;
  return fma_half((x & 0x000f000fu) | 0x64006400u, 0x3c003c00u, 0xe408e408u);     // - 1032
}
template <bool kSigned>
__device__ __forceinline__ uint32_t code_hi(uint32_t x) {
  if constexpr (!kSigned) return x & 0x00f000f0u;
  return fma_half((x & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, 0xd480d480u);     // / 16 - 72
}

// The scale bytes of a row.
template <int kChunks>
__device__ __forceinline__ uint32_t scale_word(uint32_t base, int key) {
  uint32_t w;
  if constexpr (kChunks == 4)
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(base + key * 4) : "memory");
  else if constexpr (kChunks == 2)
    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w) : "r"(base + key * 2) : "memory");
  else
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(w) : "r"(base + key) : "memory");
  return w;
}
// Scale c of two rows, as two fp16 values.
__device__ __forceinline__ uint32_t scale_pair(uint32_t w0, uint32_t w1, int c) {
  return (__byte_perm(w0, w1, c | c << 4 | (4 + c) << 8 | (4 + c) << 12) & 0x00ff00ffu) << 7;
}
__device__ __forceinline__ float scale_of(uint32_t w, int c) {
  const unsigned short h = (unsigned short)(((w >> (8 * c)) & 0xffu) << 7);
  return __half2float(__ushort_as_half(h));
}

// ---------------------------------------------------------------------------
// One warp's running softmax.  In the score tile a lane has keys lane / 4, + 8 of every 16 and columns
// (lane % 4) * 2, + 1 of each eight query heads; in the value tile the four value columns
// 4 (lane / 4) .. + 3 of every chunk and the same heads.
// ---------------------------------------------------------------------------
template <typename T, int D, int RT>
struct Q4State {
  using S = Q4Shape<T, D, RT>;
  static constexpr bool kSplit = std::is_same<T, float>::value;
  static constexpr int kParts = kSplit ? 2 : 1;      // fp16 values that a factor is given as
  static constexpr int kN = RT / 8, kC = S::kChunks, kU = S::kKeys / 16;
  uint32_t q[kParts][2 * kC][kN][2];
  float off[kC][kN][2];              // -8 times the chunk's sum of the queries
  float o[kC][2][kN][4];
  float m[kN][2], l[kN][2];          // m: the running maximum less kBoost; l: of this lane's keys
  float unit[kN][2];                 // a dot product's unit
  float slope2[kN][2];

  __device__ __forceinline__ void start(const PagedAttnQ4Args<T>& a, int s, int head, int rows) {
    const int lane = threadIdx.x & 31, c2 = lane % 4 * 2;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int r = 8 * n + lane / 4;
      const T* p = a.q + s * a.q_s + (long long)(head + r) * a.q_h + lane % 4 * 8;
      float x[kC][8];
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
#pragma unroll
        for (int i = 0; i < 8; i += Vec<T>::N) {
          if (r < rows) Vec<T>::load(p + c * 32 + i, x[c] + i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (r >= rows) x[c][i] = 0.f;
          top = fmaxf(top, fabsf(x[c][i]));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the power of two at or below the largest, as far as the factors below are numbers
      const int e = min(max((int)(__float_as_uint(top) >> 23), 27), 237);
      const float to = __uint_as_float((unsigned)(254 + 14 - e) << 23);         // 2^14 / 2^(e - 127)
      // of a score tile: 1 / to, and 2^24 where codes are subnormals
      const float one = __uint_as_float((unsigned)(kSplit ? e - 14 : e + 10) << 23);
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = !kSplit && (i & 1) ? 0.0625f : 1.f;
          float lo = x[c][i] * to * f, hi = x[c][i + 4] * to * f;
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            const uint32_t h = pack_half(lo, hi);
            const float2 back = unpack_half(h);
            q[part][2 * c + i / 2][n][i & 1] = h;
            sum += (back.x + back.y) * (1.f / f);
            lo -= back.x;
            hi -= back.y;
          }
        }
        if constexpr (kSplit) continue;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          off[c][n][i] = __shfl_sync(0xffffffffu, sum, (c2 + i) * 4) * -4.76837158203125e-7f;  // 8 / 2^24
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 8 * n + c2 + i;
        unit[n][i] = __shfl_sync(0xffffffffu, one, (c2 + i) * 4);
        slope2[n][i] = a.slopes && c < rows ? a.slopes[head + c] * kLog2e : 0.f;
        m[n][i] = kLowest;
        l[n][i] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[c][t][n][i] = 0.f;
    }
  }

  // Words of two chunks of 16 keys, or (heads of 32) of one chunk of 32 keys: x[0], x[1] the first's
  // keys 0-7 and 8-15, x[2], x[3] the second's.  `first`: chunk, or unit of 16 keys.
  template <bool kTrans>
  __device__ __forceinline__ static void words(uint32_t codes, int u, int c, uint32_t* x) {
    const int lane = threadIdx.x & 31, second = lane >> 4, half = lane >> 3 & 1;
    const int key = 16 * (kC == 1 ? u + second : u) + 8 * half + (lane & 7);
    const int chunk = kC == 1 ? 0 : c + second;
    const uint32_t at = codes + key * S::kRowBytes + (chunk ^ q4_turn<D>(key)) * 16;
    if constexpr (kTrans) ldsm4_t(at, x); else ldsm4(at, x);
  }

  __device__ __forceinline__ void chunk_scores(const uint32_t* x, int c, float s0, float s1,
                                               float (&z)[kN][4]) const {
    const uint32_t y0 = x[0] >> 8, y1 = x[1] >> 8;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float acc[4] = {};
      if constexpr (!kSplit)
        for (int i = 0; i < 4; ++i) acc[i] = off[c][n][i & 1];
#pragma unroll
      for (int part = kParts - 1; part >= 0; --part) {
        mma_f16(acc, code_lo<kSplit>(x[0]), code_lo<kSplit>(x[1]), code_hi<kSplit>(x[0]),
                code_hi<kSplit>(x[1]), q[part][2 * c][n]);
        mma_f16(acc, code_lo<kSplit>(y0), code_lo<kSplit>(y1), code_hi<kSplit>(y0),
                code_hi<kSplit>(y1), q[part][2 * c + 1][n]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) z[n][i] = fmaf(acc[i], i < 2 ? s0 : s1, z[n][i]);
    }
  }

  __device__ __forceinline__ void tile(const ScoreRule& rule, uint32_t stage, int key0,
                                       unsigned mask) {
    const int lane = threadIdx.x & 31;
    const uint32_t vt = stage + S::kCodes, ks = vt + S::kCodes, vs = ks + S::kScales;
    float z[kU][kN][4] = {};
#pragma unroll
    for (int u = 0; u < kU; u += kC == 1 ? 2 : 1) {
#pragma unroll
      for (int c = 0; c < kC; c += 2) {
        uint32_t x[4];
        words<false>(stage, u, c, x);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int uu = kC == 1 ? u + k : u, cc = kC == 1 ? 0 : c + k;
          const uint32_t w0 = scale_word<kC>(ks, 16 * uu + lane / 4);
          const uint32_t w1 = scale_word<kC>(ks, 16 * uu + 8 + lane / 4);
          chunk_scores(x + 2 * k, cc, scale_of(w0, cc), scale_of(w1, cc), z[uu]);
        }
      }
    }
    // z becomes the scores, or stays the sums above where a factor is all that is missing
    float factor[kN][2];
    const bool full = mask == 0xffffffffu;
    if (rule.plain && full) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) factor[n][i] = rule.scale2 * unit[n][i];
    } else {
      bool small = rule.cap > 0.f;
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[u][n][i] *= unit[n][i & 1];
            small &= fabsf(z[u][n][i] * rule.rcap) < kSeries;
          }
      const bool series = __all_sync(0xffffffffu, small);
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 16 * u + lane / 4 + 8 * (i >> 1);
            float& x = z[u][n][i];
            x = !((mask >> j) & 1) ? -INFINITY
                : series           ? score_near_zero(rule, x, slope2[n][i & 1], key0 + j)
                                   : score_of<!kSplit>(rule, x, slope2[n][i & 1], key0 + j);
          }
#pragma unroll
      for (int n = 0; n < kN; ++n) factor[n][0] = factor[n][1] = 1.f;
    }
    // The running maxima are looked for again only where a score is above them.
    bool above = false;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          above |= fmaf(z[u][n][i], factor[n][i & 1], -m[n][i & 1]) > kBoost;
    if (__any_sync(0xffffffffu, above)) {
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = fmaxf(z[0][n][i] * factor[n][i], z[0][n][i + 2] * factor[n][i]);
#pragma unroll
          for (int u = 1; u < kU; ++u)
            top = fmaxf(top, fmaxf(z[u][n][i] * factor[n][i], z[u][n][i + 2] * factor[n][i]));
#pragma unroll
          for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          top = fmaxf(m[n][i], top - kBoost);
          f[i] = exp2_fast(m[n][i] - top);
          l[n][i] *= f[i];
          m[n][i] = top;
        }
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[c][t][n][i] *= f[i & 1];
      }
    }
    // The values' scales: of keys (lane % 4) * 2, + 1, + 8, + 9 of every 16 (the weights' order as right
    // operand), or, where weights are split, lane / 4, + 8 (their order as scores).  What a free row
    // holds is not looked at.
    constexpr int kW = kSplit ? 2 : 4;
    uint32_t w[kU][kW];
    uint32_t large = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        const int key = 16 * u + (kSplit ? lane / 4 + 8 * k : lane % 4 * 2 + (k & 1) + 8 * (k >> 1));
        w[u][k] = scale_word<kC>(vs, key);
        if (!full && !((mask >> key) & 1)) w[u][k] = 0;
        large |= w[u][k];
      }
    float drop = 0.f, up = 1.f;      // of the weights, so that their products with the scales stay finite
    if (__any_sync(0xffffffffu, large & 0x80808080u)) {
      unsigned most = 0;
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int k = 0; k < kW; ++k)
#pragma unroll
          for (int c = 0; c < kC; ++c) most = max(most, (w[u][k] >> (8 * c + 3)) & 31u);
      most = __reduce_max_sync(0xffffffffu, most);
      drop = (float)((int)most - 15);
      up = __uint_as_float((most - 15 + 127) << 23);
    }
    float p[kU][kN][4];
    float sum_l[kN][2] = {};
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[u][n][i] = exp2_fast(fmaf(z[u][n][i], factor[n][i & 1], -m[n][i & 1] - drop));
          sum_l[n][i & 1] += p[u][n][i];
        }
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) l[n][i] = fmaf(sum_l[n][i], up, l[n][i]);
    uint32_t pt[kU][kN][2];          // weights as right operand: keys in pairs, a column a head
    if constexpr (!kSplit) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            pt[u][n][i] = transpose8(pack_half(p[u][n][2 * i], p[u][n][2 * i + 1]));
    }
    // chunk c of the values, x its words of every 16 keys
    auto chunk_values = [&](int c, const uint32_t* const (&x)[kU]) {
      uint32_t ps[kParts][kU][kN][2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if constexpr (kSplit) {
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float s = scale_of(w[u][i], c);
              const float lo = p[u][n][2 * i] * s, hi = p[u][n][2 * i + 1] * s;
              const uint32_t h = pack_half(lo, hi);
              const float2 back = unpack_half(h);
              ps[0][u][n][i] = transpose8(h);
              ps[kParts - 1][u][n][i] = transpose8(pack_half(lo - back.x, hi - back.y));
            }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t s = scale_pair(w[u][(2 * i) % kW], w[u][(2 * i + 1) % kW], c);
#pragma unroll
            for (int n = 0; n < kN; ++n) ps[0][u][n][i] = mul_half(pt[u][n][i], s);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        float sum[2][4] = {};
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const uint32_t x0 = x[u][0], x1 = x[u][1], y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            mma_f16(sum[0], code_lo<true>(x0), code_hi<true>(x0), code_lo<true>(x1),
                    code_hi<true>(x1), ps[part][u][n]);
            mma_f16(sum[1], code_lo<true>(y0), code_hi<true>(y0), code_lo<true>(y1),
                    code_hi<true>(y1), ps[part][u][n]);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[c][t][n][i] = fmaf(sum[t][i], up, o[c][t][n][i]);
      }
    };
    if constexpr (kC == 1) {
      static_assert(kU == 2, "both units' words at once");
      uint32_t x[4];
      words<true>(vt, 0, 0, x);
      chunk_values(0, {x, x + 2});
    } else {
#pragma unroll
      for (int c = 0; c < kC; c += 2) {
        uint32_t x[kU][4];
#pragma unroll
        for (int u = 0; u < kU; ++u) words<true>(vt, u, c, x[u]);
        static_assert(kU == 2, "words of two units");
        chunk_values(c, {x[0], x[1]});
        chunk_values(c + 1, {x[0] + 2, x[1] + 2});
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
  // column c of a row of sums lies at c ^ spread(row): put_o's lanes write to different banks
  __device__ __forceinline__ static int spread(int r) { return r >> 1 & 3; }
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
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[r * D + ((32 * c + 4 * (lane / 4) + k) ^ spread(r))] =
                o[c][k / 2][n][(k & 1) * 2 + i] * f;
      }
  }
};

// ---------------------------------------------------------------------------
// The warp's loader: rows and scales as they lie, 16 keys of a page at a time (a page holds as many).
// ---------------------------------------------------------------------------
template <typename T, int D, int RT>
struct Q4Loader : RowLoader<Q4Shape<T, D, RT>, PagedAttnQ4Args<T>> {
  using S = Q4Shape<T, D, RT>;
  using Rows = typename RowLoader<S, PagedAttnQ4Args<T>>::Rows;

  __device__ __forceinline__ void issue(const PagedAttnQ4Args<T>& a, const Rows& r, uint32_t stage,
                                        unsigned* mask_out) const {
    const int lane = threadIdx.x & 31;
    const unsigned mask = this->valid_keys(a, r);
    if (lane == 0) *mask_out = mask;
    if (mask) {
      const int log2 = a.paged.page_log2, in_page = (1 << log2) - 1;
      // a page's bytes of one head: 16 codes' and one scale byte for every chunk
      const long long head_bytes = (long long)(17 * S::kChunks) << log2;
      const int scales_at = S::kRowBytes << log2;
      constexpr int kRows = 32 / S::kChunks;          // rows a warp copies at once
      const int row0 = lane / S::kChunks;
#pragma unroll
      for (int i = 0; i < S::kChunks; ++i) {
        const int row = i * kRows + row0;
        const int page = __shfl_sync(0xffffffffu, r.page, row);
        const bool live = (mask >> row) & 1;
        const long long off = ((long long)page * a.Hkv + r.head) * head_bytes +
                              ((r.key0 + row) & in_page) * S::kRowBytes + lane % S::kChunks * 16;
        const uint32_t dst = stage + (i * 32 + lane) * 16;
        copy16(dst, a.k_cache + (live ? off : 0), live);
        copy16(dst + S::kCodes, a.v_cache + (live ? off : 0), live);
      }
      // scales, K's and V's: 16 bytes are those of 16 / kChunks rows
      constexpr int kPieces = S::kScales / 16, kEach = 16 / S::kChunks;
      const int piece = lane % kPieces, row = piece * kEach;
      const int page = __shfl_sync(0xffffffffu, r.page, row);
      if (lane < 2 * kPieces) {
        const bool live = (mask >> row) & ((1u << kEach) - 1);
        const long long off = ((long long)page * a.Hkv + r.head) * head_bytes + scales_at +
                              ((r.key0 + row) & in_page) * S::kChunks;
        copy16(stage + 2 * S::kCodes + lane * 16,
               (lane < kPieces ? a.k_cache : a.v_cache) + (live ? off : 0), live);
      }
    }
    copy_commit();
  }
};

template <typename T, int D, int RT>
struct Q4 {
  using Type = T;
  using Args = PagedAttnQ4Args<T>;
  using S = Q4Shape<T, D, RT>;
  using State = Q4State<T, D, RT>;
  using Ld = Q4Loader<T, D, RT>;
  static constexpr int kD = D, kRT = RT;
};

// A CTA takes 8 query rows, in bf16 16 where the group has more; larger groups take several CTAs.
template <typename T, int RT, typename F>
auto with_dim(int d, F f) {
  switch (d) {
    case 32: return f(Run<Q4<T, 32, RT>>{});
    case 64: return f(Run<Q4<T, 64, RT>>{});
    default: return f(Run<Q4<T, 128, RT>>{});
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

size_t paged_attn_q4_ws_bytes(int d, int Hkv, int G, int S, int width, int page_log2, int is_f32,
                              int sms) {
  auto bytes = [&](auto run) { return run.bytes(Hkv, G, S, width, page_log2, sms); };
  return is_f32 ? with_shape<float>(d, G, bytes) : with_shape<bf16>(d, G, bytes);
}

template <typename T>
cudaError_t launch_paged_attn_q4(PagedAttnQ4Args<T> a, int d, void* ws, int sms, cudaStream_t st) {
  return with_shape<T>(d, a.G, [&](auto run) { return run.launch(a, ws, sms, st); });
}

template cudaError_t launch_paged_attn_q4<float>(PagedAttnQ4Args<float>, int, void*, int,
                                                 cudaStream_t);
template cudaError_t launch_paged_attn_q4<bf16>(PagedAttnQ4Args<bf16>, int, void*, int,
                                                cudaStream_t);

}  // namespace mita
