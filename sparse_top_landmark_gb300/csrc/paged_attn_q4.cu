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
// - values, and keys in fp32: one instruction more makes n - 8 of it.  (The tensor cores cut sums.
//   Taken as n p from a sum of -8 p, a long context's values, which nearly cancel, lean by 2^-23 of
//   eight times the sum of the weights for every product: 4.8e-6 of an fp32 result at 1000 keys, 1e-3 at a
//   million.  With a sum of its own for 8 p they do not lean, for 2 % less time, but where a key of value zero has
//   nearly all the weight, what is left of the others is off by 2^-21 of that key's scale: not kept.)  Of two
//   codes of a word the bf16 twin takes the lower one alone and both as a byte, from whose sums the lower
//   one's are taken at the end: an instruction less for four values.
//
// Queries are scaled by a power of two, their row's largest to 2^14, so that fp16 holds what bf16 does, down
// to 2^-34 of it; in fp32 they are sums of two fp16 values, 22 bits.
//
// Weights and scales meet in these ways, since most of the weight may be on keys whose values are small or
// zero, and what the others add is then a small part of a weight's range, or of a scale's:
//
// - bf16: a weight p goes into fp16 times the power of two w of its key's largest scale, and the scale
//   divided by it, 11 bits for the one and again for their product.  The running maximum is p w's, which
//   is 2^10 to 2^14 where it is rounded, so that fp16's subnormals begin at 2^-24 of it; a key
//   without values has w = 0.  A block 2^-21 times its own row's largest loses bits by itself, and the upper
//   code of a byte has 2^-22 of what the block's scales add up to.  (With p
//   and the scale as they are: an output is off by 3 % where a key of value zero stands 15 above the others and
//   their scales are 2^-13, in fp32 with two values for a product too.  With two bf16 values for a
//   weight, as below, the 128 sequences' 120 us are 138: tensor cores.  With one w for a tile whose scales are near
//   each other: 130, the two ways being a branch in the middle of a tile.)
// - fp32: a weight is a sum of three bf16 values, which have fp32's exponents, and the scale is with the
//   code: (n - 8) s has seven bits.
//
// A tile's sums are added to the running ones in fp32, outside the tensor cores: paged_attn.cu says why.
//
// Bound by the latency of instructions: three warps a scheduler issue 0.58 a cycle, half-rate ones half of what their
// pipe takes, the tensor cores 24 %, HBM 57 %.  A tile of 32 keys of 128 takes a warp some 620 instructions (128
// masks and 48 shifts and byte moves for 8192 codes, 64 to make values signed, 48 for
// the scales, 32 products).  Measured (bf16): 128 sequences of up to 8192 keys, 32/8 heads of 128, in 120 us, 4.7 TB/s
// (paged_attn.cu takes 311 us for the same in bf16); one sequence of 1,048,575 keys, 8/2 heads of 64, in
// 47 us; 200 of up to 900 keys in 45 us; one of 333 in 8 us; fp32, 64 of up to 8192, 32/8 heads of 128, in 102 us.
#include "paged_row.cuh"

#include <cuda_fp16.h>

namespace mita {
namespace {

// The running maximum is looked for again only where a lane's weights add up to more than 2^14; the largest
// weight is then 2^10, so that a tile's eight of a lane stay below that.  (bf16: weights times their keys' powers of
// two; weights alone may come to 2^64 where those differ, the largest then being 2^60, whose exponent is rounded
// at 2^-19.)
constexpr float kBoost = 10.f, kMostSum = 16384.f, kRoom = 60.f, kMostWeight = 18446744073709551616.f;

// Shared memory and shape of one instantiation; RT: query rows of a segment.
//
// A CTA has several teams of warps, each with a share of its own: two, or four where there are many segments (256
// sequences of up to 300 keys, 32/8 heads of 128: two 42 us, four 32; 200 of up to 900: 51 and 45).  What follows was
// measured on earlier forms of the kernel, up to 6 % faster or slower than this one: one team 70 us for those 256, two
// 39, four 31; 128 sequences of up to 8192 keys one 153, two 132, later 117, four 115; in fp32, 256 of up to 500 two 55,
// four 48; 128/8 heads, of 16 rows then, two 195, four 209.  Registers
// hold 12 warps' state for heads of 128, 16 for smaller ones (a million keys, heads of 64: teams of 6
// 48 us, of 8 46), 8 where rows are 16 or a factor is two values (fp32, 64 sequences of up to 8192 keys,
// heads of 128: teams of 4 109 us, of 5 117; heads of 64: teams of 4 72, of 8 62).
// A warp takes 64 keys of a tile (32, and three stages instead of two: 147 us for 124), and ending a segment
// is worth one tile (none: fp32 116 us for 109, four teams 131 for 115; two: 123 for 119, four teams 115.4).
template <typename T, int D, int RT, int TEAMS>
struct Q4Shape {
  static constexpr bool kSplit = std::is_same<T, float>::value;
  static constexpr int kTeams = TEAMS;
  static constexpr int kWarps = D == 128 ? (RT > 8 || kSplit ? 8 : 12) : RT > 8 ? 12 : 16;
  static constexpr int kTeamWarps = kWarps / kTeams;
  static constexpr int kThreads = kWarps * 32, kTeamThreads = kTeamWarps * 32;
  static constexpr int kKeys = 64;
  using Mask = unsigned long long;       // a bit a key
  static constexpr int kTile = kTeamWarps * kKeys;
  static constexpr int kSegmentCost = 1;
  static constexpr int kChunks = D / kQ4Block;            // of a row: 16 bytes and one scale each
  static constexpr int kRowBytes = D / 2;
  static constexpr int kCodes = kKeys * kRowBytes, kScales = kKeys * kChunks;
  static constexpr int kStageBytes = 2 * (kCodes + kScales);      // K's codes, V's, K's scales, V's
  // a warp's decoded scales: K's in fp32, V's in 16 bits, two keys side by side (with a number more each, or in
  // bf16 where the scales' bytes stood in the stage)
  static constexpr int kDecodedK = kKeys * kChunks * 4, kDecoded = kDecodedK * (kSplit ? 2 : 1);
  // a team's queries as right operands, [part][heads / 8][chunk][lane] of 16 bytes, what a product
  // starts from, [heads / 8][chunk][lane % 4] of 16 bytes, and [heads] units and slopes; twice where there
  // is room for it
  static constexpr int kN = RT / 8, kParts = kSplit ? 2 : 1;
  static constexpr int kOffStart = kParts * kN * kChunks * 512;
  static constexpr int kOffUnit = kOffStart + (kSplit ? 0 : kN * kChunks * 64);
  static constexpr int kQueries = kOffUnit + RT * 8, kQuerySets = kTeams == 4 && D == 128 ? 1 : 2;
  static constexpr int kRest = kWarps * (kDecoded + RT * 8) +
                               kTeams * (kQuerySets * kQueries + 2 * (int)sizeof(Join) + 16);
  static constexpr int kFit = (232448 - 16 - kRest) / (kWarps * (kStageBytes + (int)sizeof(Mask)));
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kJoinBytes = kTeamWarps * kRing;                   // a team's
  static constexpr int kOffDecoded = kWarps * kRing;                      // [warps]
  static constexpr int kOffQueries = kOffDecoded + kWarps * kDecoded;     // [teams][sets]
  static constexpr int kOffMl = kOffQueries + kTeams * kQuerySets * kQueries;      // [teams][team's warps][RT][2]
  static constexpr int kOffMask = kOffMl + kWarps * RT * 8;               // [warps][stages]
  static constexpr int kOffJoins = kOffMask + (kWarps * kStages * (int)sizeof(Mask) + 15) / 16 * 16;
  static constexpr int kOffBase = kOffJoins + kTeams * 2 * (int)sizeof(Join);
  static constexpr int kBytes = kOffBase + kTeams * 16;
  static_assert(kBytes <= 232448 && kStages >= 2 && kStageBytes % 16 == 0, "shared memory");
  static_assert(RT * D * 4 <= kStageBytes, "a warp's sums in one of its stages");
  static_assert(kTeams == 2 || kTeams == 4, "a counter's fields");
  __device__ __forceinline__ static int warp() { return (threadIdx.x >> 5) % kTeamWarps; }
};

// The warps that work on one share.
template <typename S>
struct Q4Team {
  __device__ __forceinline__ static int team() { return (threadIdx.x >> 5) / S::kTeamWarps; }
  __device__ __forceinline__ static int thread() { return threadIdx.x - team() * S::kTeamThreads; }
  __device__ __forceinline__ static void sync() {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team()), "n"(S::kTeamThreads) : "memory");
  }
};

// Chunk c of row r of a page stands at c ^ q4_turn(r).
template <int D>
__device__ __forceinline__ int q4_turn(int r) {
  return D == 128 ? (r >> 1) & 3 : D == 64 ? (r >> 2) & 1 : 0;
}

// d[16 x 8] = c + a[16 x 16] b[16 x 8], fp16 products summed in fp32
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        const uint32_t* b, float c0, float c1, float c2, float c3) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        const uint32_t* b) {
  mma_f16(c, a0, a1, a2, a3, b, c[0], c[1], c[2], c[3]);
}
// the same with bf16 products
__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         const uint32_t* b, float c0, float c1, float c2, float c3) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         const uint32_t* b) {
  mma_bf16(c, a0, a1, a2, a3, b, c[0], c[1], c[2], c[3]);
}
// An 8 x 8 matrix of 16-bit values, transposed (paged_row.cuh's, free to be moved among the products).
__device__ __forceinline__ uint32_t turn8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
__device__ __forceinline__ uint32_t fma_bf(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Codes 0 and 1 of the two 16-bit words of x (of x >> 8: 2 and 3), as fp16 numbers n * 2^-24 and
// 16 n * 2^-24, or, kSigned, both as (n - 8) * 2^-9.
template <bool kSigned>
__device__ __forceinline__ uint32_t code_lo(uint32_t x) {
  x &= 0x000f000fu;
  return kSigned ? fma_half(x, 0x78007800u, 0xa400a400u) : x;       // * 2^15 - 2^-6
}
template <bool kSigned>
__device__ __forceinline__ uint32_t code_hi(uint32_t x) {
  x &= 0x00f000f0u;
  return kSigned ? fma_half(x, 0x68006800u, 0xa400a400u) : x;       // * 2^11 - 2^-6
}
// A pair of codes of each word, as a byte n1 n0: (16 (n1 - 8) + n0 - 8) * 2^-13
__device__ __forceinline__ uint32_t code_pair(uint32_t x) {
  return fma_half(x, 0x68006800u, 0xa440a440u);                     // * 2^11 - 136 * 2^-13
}
// Codes 0 and 1 of the two words of x as values in bf16: a code n is the subnormal n * 2^-133, m its scale times
// 2^112 (bf16, a key each), so that these are (n - 8) s 2^-21 and 16 (n - 8) s 2^-21, seven bits and exact.
// less: value_less(m).
__device__ __forceinline__ uint32_t value_less(uint32_t m) { return mul_bf(m, 0x80088008u); }     // -8 * 2^-133 m
__device__ __forceinline__ uint32_t value_lo(uint32_t x, uint32_t m, uint32_t less) {
  return fma_bf(x & 0x000f000fu, m, less);
}
__device__ __forceinline__ uint32_t value_hi(uint32_t x, uint32_t m, uint32_t less) {
  return fma_bf(x & 0x00f000f0u, m, mul_bf(less, 0x41804180u));     // 16 of them
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
// The four (two, one) scales of a word as fp16 values: chunks 0 and 2, chunks 1 and 3.
__device__ __forceinline__ uint32_t scales_02(uint32_t w) { return (w & 0x00ff00ffu) << 7; }
__device__ __forceinline__ uint32_t scales_13(uint32_t w) { return w >> 1 & 0x7f807f80u; }
// The largest scale byte of a row, infinities and NaN (248 and above) left out.
template <int kChunks>
__device__ __forceinline__ uint32_t largest_scale(uint32_t w) {
  w &= ~((((w & 0x7f7f7f7fu) + 0x08080808u & w & 0x80808080u) >> 7) * 255u);
  if constexpr (kChunks == 4) w = __vmaxu2(w & 0x00ff00ffu, w >> 8 & 0x00ff00ffu);
  return kChunks == 4 ? max(w & 0xffu, w >> 16) : kChunks == 2 ? max(w & 0xffu, w >> 8) : w;
}
// The same times 2^112 in bf16, whose bits are a scale's 2^-112 times as large; a NaN's become an infinity,
// which makes NaN of every code.
__device__ __forceinline__ uint32_t factors(uint32_t bits) {
  return mul_bf(mul_bf(bits, 0x77807780u), 0x77807780u);            // 2^112 twice
}
__device__ __forceinline__ uint32_t factors_02(uint32_t w) { return factors((w & 0x00ff00ffu) << 4); }
__device__ __forceinline__ uint32_t factors_13(uint32_t w) { return factors(w >> 4 & 0x0ff00ff0u); }

__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void store_shared(uint32_t at, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ void store_shared(uint32_t at, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void store_shared(uint32_t at, const uint32_t (&x)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3])
               : "memory");
}
template <int N>
__device__ __forceinline__ void load_shared(uint32_t at, uint32_t (&x)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at)
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x[0]) : "r"(at) : "memory");
}

// ---------------------------------------------------------------------------
// One warp's running softmax.  In the score tile a lane has keys lane / 4, + 8 of every 16 and columns
// (lane % 4) * 2, + 1 of each eight query heads; in the value tile the four value columns
// 4 (lane / 4) .. + 3 of every chunk and the same heads.
// ---------------------------------------------------------------------------
template <typename T, int D, int RT, int TEAMS>
struct Q4State {
  using S = Q4Shape<T, D, RT, TEAMS>;
  static constexpr bool kSplit = std::is_same<T, float>::value;
  static constexpr int kParts = kSplit ? 2 : 1;      // fp16 values that a query is given as
  static constexpr int kWeights = kSplit ? 3 : 1;    // values that a weight is given as
  static constexpr int kN = RT / 8, kC = S::kChunks;
  // 16 keys are a unit of work, kU of them are worked on together (as many as registers hold: 16 rows of 128
  // have 8 warps; 196 us for 201, and 28.5 for 26.2 with 16 rows of 64), and kP chunks
  static constexpr int kU = !kSplit && (kN == 1 || D == 128) ? 4 : 2, kP = kC == 1 ? 1 : 2;
  unsigned long long o[kC][2][kN][2];   // two heads of a value column each
  float m[kN][2], l[kN][2];          // m: the running maximum less kBoost; l: of this lane's keys
  bool far;                          // a maximum of the warp's is beyond kFar

  // Puts chunk c of a segment's queries to `to`, as every warp of the team will read them.
  __device__ __forceinline__ static void put_queries(const PagedAttnQ4Args<T>& a, int s, int head,
                                                     int rows, int c, uint32_t to) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int r = 8 * n + lane / 4;
      const T* p = a.q + s * a.q_s + (long long)(head + r) * a.q_h + lane % 4 * 8;
      float x[8], y[8], top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      if (r < rows) {
#pragma unroll
        for (int cc = 0; cc < kC; ++cc) {
#pragma unroll
          for (int i = 0; i < 8; i += Vec<T>::N) Vec<T>::load(p + cc * 32 + i, y + i);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            top = fmaxf(top, fabsf(y[i]));
            if (cc == c) x[i] = y[i];
          }
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the power of two at or below the largest, as far as the factors below are numbers
      const int e = min(max((int)(__float_as_uint(top) >> 23), 27), 237);
      const float up = __uint_as_float((unsigned)(254 + 14 - e) << 23);         // 2^14 / 2^(e - 127)
      uint32_t q[kParts][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = !kSplit && (i & 1) ? up * 0.0625f : up;
        float lo = x[i] * f, hi = x[i + 4] * f;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          q[part][i] = pack_half(lo, hi);
          const float2 back = unpack_half(q[part][i]);
          lo -= back.x;
          hi -= back.y;
        }
      }
#pragma unroll
      for (int part = 0; part < kParts; ++part)
        store_shared(to + (((part * kN + n) * kC + c) * 32 + lane) * 16, q[part]);
      if constexpr (!kSplit) {       // -8 times the sum, as products with -8 (and -128) * 2^-24
        float off[4];
        mma_f16(off, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, q[0], 0.f, 0.f, 0.f, 0.f);
        mma_f16(off, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, q[0] + 2);
        if (lane < 4) {
          const uint32_t x4[4] = {__float_as_uint(off[0]), __float_as_uint(off[1]),
                                  __float_as_uint(off[2]), __float_as_uint(off[3])};
          store_shared(to + S::kOffStart + ((n * kC + c) * 4 + lane) * 16, x4);
        }
      }
      if (c == 0 && lane % 4 == 0) {
        // a dot product's unit: 1 / up, and what the codes' numbers are smaller than they: 2^24 or 2^9
        const float one = __uint_as_float((unsigned)(kSplit ? e - 14 + 9 : e - 14 + 24) << 23);
        const float slope = a.slopes && r < rows ? a.slopes[head + r] * kLog2e : 0.f;
        store_shared(to + S::kOffUnit + r * 4, __float_as_uint(one));
        store_shared(to + S::kOffUnit + RT * 4 + r * 4, __float_as_uint(slope));
      }
    }
  }

  __device__ __forceinline__ void start() {
    far = false;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[n][i] = kLowest;
        l[n][i] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) o[c][t][n][i] = 0;
    }
  }
  // a pair of [heads] floats at `at`: those of this lane's columns of tile n
  __device__ __forceinline__ static void pair_of(uint32_t at, int n, float (&x)[2]) {
    uint32_t w[2];
    load_shared(at + (8 * n + (threadIdx.x & 3) * 2) * 4, w);
    x[0] = __uint_as_float(w[0]);
    x[1] = __uint_as_float(w[1]);
  }

  // Words of chunks c .. c + kP - 1 of kM units from unit u0 on: [unit][chunk] keys 0-7 and 8-15.
  template <bool kTrans, int kM>
  __device__ __forceinline__ static void words(uint32_t codes, int u0, int c, uint32_t (&x)[kM][kP][2]) {
    const int lane = threadIdx.x & 31, second = lane >> 4;
#pragma unroll
    for (int i = 0; i < kM * kP / 2; ++i) {      // four matrices: two units', or two chunks'
      const int key = 16 * (u0 + (kP == 1 ? 2 * i + second : i)) + (lane >> 3 & 1) * 8 + (lane & 7);
      const int chunk = kP == 1 ? 0 : c + second;
      const uint32_t at = codes + key * S::kRowBytes + (chunk ^ q4_turn<D>(lane & 7)) * 16;
      uint32_t y[4];
      if constexpr (kTrans) ldsm4_t(at, y); else ldsm4(at, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[kP == 1 ? 2 * i + k / 2 : i][kP == 1 ? 0 : k / 2][k & 1] = y[k];
    }
  }

  // Every lane decodes the scales of two keys (the lanes that use a key's are many: 4 its K's, 8 its V's):
  // from `ks`, K's bytes and then V's, to `sk`, K's as fp32, and V's to `sv`: as value_lo takes them, or, in
  // bf16, times the power of two that brings the row's largest to 2 to 4, whose inverse (zero for a row of
  // zeros) is `unit`, of keys `lane` and `lane` + 32.  A value's scale of a key that is not seen is zero,
  // whatever the row holds.
  __device__ __forceinline__ static void decode_scales(uint32_t ks, uint32_t sk, uint32_t sv,
                                                       typename S::Mask mask, float (&unit)[2]) {
    const int lane = threadIdx.x & 31;
    constexpr int kH = S::kKeys / 32;
    uint32_t wk[kH], wv[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      wk[h] = scale_word<kC>(ks, lane + 32 * h);
      wv[h] = scale_word<kC>(ks + S::kScales, lane + 32 * h);
      if (mask != ~0ull && !((unsigned)(mask >> (32 * h)) >> lane & 1)) wv[h] = 0;
    }
    __syncwarp();                    // they, and the last tile's scales, have been read
    auto put = [&](uint32_t at, uint32_t w) {          // as fp32, [key][chunk]
      const float2 even = unpack_half(scales_02(w)), odd = unpack_half(scales_13(w));
      if constexpr (kC == 4) {
        const uint32_t x[4] = {__float_as_uint(even.x), __float_as_uint(odd.x), __float_as_uint(even.y),
                               __float_as_uint(odd.y)};
        store_shared(at + lane * 16, x);
      } else if constexpr (kC == 2) {
        store_shared(at + lane * 8, __float_as_uint(even.x), __float_as_uint(odd.x));
      } else {
        store_shared(at + lane * 4, __float_as_uint(even.x));
      }
    };
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      put(sk + h * 128 * kC, wk[h]);
      // of two keys, [pair][chunk]: each of the two writes half
      uint32_t even, odd = 0;
      if constexpr (kSplit) {
        even = factors_02(wv[h]);
        if constexpr (kC > 1) odd = factors_13(wv[h]);
      } else {
        const uint32_t top = largest_scale<kC>(wv[h]), e = max(top >> 3, 1u);
        const uint32_t by = ((31u - e) << 10) * 0x10001u;                // 2^(16 - e)
        even = mul_half(scales_02(wv[h]), by);
        if constexpr (kC > 1) odd = mul_half(scales_13(wv[h]), by);
        unit[h] = __uint_as_float(top == 0 ? 0u : (e - 16 + 127) << 23);
      }
      const uint32_t even2 = __shfl_xor_sync(0xffffffffu, even, 1);
      const bool second = lane & 1;
      constexpr int kEach = kSplit ? 8 : 4;            // bytes of a pair's chunk
      const uint32_t to = sv + (16 * h + lane / 2) * kC * kEach;
      if constexpr (kC == 1) {
        if (!second) put_factor(to, __byte_perm(even, even2, 0x5410));
      } else {
        const uint32_t odd2 = __shfl_xor_sync(0xffffffffu, odd, 1);
        if constexpr (kC == 2) {
          put_factor(to + (second ? kEach : 0), second ? __byte_perm(odd2, odd, 0x5410)
                                                       : __byte_perm(even, even2, 0x5410));
        } else {
          const uint32_t sel = second ? 0x3276u : 0x5410u;      // upper halves, or lower ones
          const uint32_t m0 = __byte_perm(even, even2, sel), m1 = __byte_perm(odd, odd2, sel);
          const uint32_t at = to + (second ? 2 * kEach : 0);
          if constexpr (kSplit) {
            const uint32_t x[4] = {m0, value_less(m0), m1, value_less(m1)};
            store_shared(at, x);
          } else {
            store_shared(at, m0, m1);
          }
        }
      }
    }
    __syncwarp();
  }
  __device__ __forceinline__ static void put_factor(uint32_t at, uint32_t m) {
    if constexpr (kSplit) store_shared(at, m, value_less(m)); else store_shared(at, m);
  }

  // z += scale * (codes . q) of 16 keys, x their words of a chunk, q the chunk's queries, `from` what
  // the product starts from
  __device__ __forceinline__ static void chunk_scores(const uint32_t* x, const uint32_t (&q)[kParts][kN][4],
                                                      const uint32_t (&from)[kN][4], uint32_t s0,
                                                      uint32_t s1, float (&z)[kN][4]) {
    const uint32_t y0 = x[0] >> 8, y1 = x[1] >> 8;
    const uint32_t a[8] = {code_lo<kSplit>(x[0]), code_lo<kSplit>(x[1]), code_hi<kSplit>(x[0]),
                           code_hi<kSplit>(x[1]), code_lo<kSplit>(y0), code_lo<kSplit>(y1),
                           code_hi<kSplit>(y0), code_hi<kSplit>(y1)};
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float acc[4];
      if constexpr (kSplit) {
        mma_f16(acc, a[0], a[1], a[2], a[3], q[1][n], 0.f, 0.f, 0.f, 0.f);
        mma_f16(acc, a[4], a[5], a[6], a[7], q[1][n] + 2);
        mma_f16(acc, a[0], a[1], a[2], a[3], q[0][n]);
      } else {
        mma_f16(acc, a[0], a[1], a[2], a[3], q[0][n], __uint_as_float(from[n][0]),
                __uint_as_float(from[n][1]), __uint_as_float(from[n][2]), __uint_as_float(from[n][3]));
      }
      mma_f16(acc, a[4], a[5], a[6], a[7], q[0][n] + 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[n][i] = fmaf(acc[i], __uint_as_float(i < 2 ? s0 : s1), z[n][i]);
    }
  }

  // stage: the warp's rows and scales; key0 the first one's position; `mask` the seen ones
  __device__ __forceinline__ void tile(const ScoreRule& rule, uint32_t queries, uint32_t stage, int key0,
                                       typename S::Mask mask) {
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t ks = stage + 2 * S::kCodes;
    const uint32_t sk = smem_addr(smem) + S::kOffDecoded + (threadIdx.x >> 5) * S::kDecoded;
    const uint32_t sv = kSplit ? sk + S::kDecodedK : ks;
    float unit[2];
    decode_scales(ks, sk, sv, mask, unit);
#pragma unroll 1
    for (int u = 0; u < S::kKeys / 16; u += kU)
      work(rule, queries, stage, sk, sv, unit, u, key0 + 16 * u,
            mask >> (16 * u) & (~0ull >> (64 - 16 * kU)));
  }

  // units of 16 keys u0 .. u0 + kU - 1; mask: their seen keys; sk, sv, unit2: decode_scales'
  __device__ __forceinline__ void work(const ScoreRule& rule, uint32_t queries, uint32_t stage,
                                      uint32_t sk, uint32_t sv, const float (&unit2)[2], int u0, int key0,
                                       typename S::Mask mask) {
    if (kU < S::kKeys / 16 && mask == 0) return;
    const int lane = threadIdx.x & 31;
    const uint32_t vt = stage + S::kCodes;
    const bool full = mask == (~0ull >> (64 - 16 * kU));
    float z[kU][kN][4] = {};
#pragma unroll 1
    for (int c0 = 0; c0 < kC; c0 += kP) {        // (not unrolled: the tile's instructions have to fit their cache)
      uint32_t x[kU][kP][2];
      words<false>(stage, u0, c0, x);
      uint32_t sc[kU][2][kP];
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          load_shared(sk + ((16 * (u0 + u) + lane / 4 + 8 * i) * kC + c0) * 4, sc[u][i]);
#pragma unroll
      for (int k = 0; k < kP; ++k) {
        const int c = c0 + k;
        uint32_t q[kParts][kN][4], from[kN][4];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            load_shared(queries + (((part * kN + n) * kC + c) * 32 + lane) * 16, q[part][n]);
          if constexpr (!kSplit)
            load_shared(queries + S::kOffStart + ((n * kC + c) * 4 + lane % 4) * 16, from[n]);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
          chunk_scores(x[u][k], q, from, sc[u][0][k], sc[u][1][k], z[u]);
      }
    }
    // z becomes the scores, or stays the sums above where a factor is all that is missing
    float factor[kN][2];
#pragma unroll
    for (int n = 0; n < kN; ++n) pair_of(queries + S::kOffUnit, n, factor[n]);
    if (rule.plain && full && !far) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) factor[n][i] *= rule.scale2;
    } else {
      float slope2[kN][2];
#pragma unroll
      for (int n = 0; n < kN; ++n) pair_of(queries + S::kOffUnit + RT * 4, n, slope2[n]);
      bool series = rule.cap > 0.f;
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) z[u][n][i] *= factor[n][i & 1];
      if (series) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) series &= fabsf(z[u][n][i] * rule.rcap) < kSeries;
        series = __all_sync(0xffffffffu, series);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 16 * u + lane / 4 + 8 * (i >> 1);
            float& x = z[u][n][i];
            x = !((mask >> j) & 1) ? -INFINITY
                : rule.plain       ? x * rule.scale2
                : series           ? score_near_zero(rule, x, slope2[n][i & 1], key0 + j)
                                   : score_of<!kSplit>(rule, x, slope2[n][i & 1], key0 + j);
          }
#pragma unroll
      for (int n = 0; n < kN; ++n) factor[n][0] = factor[n][1] = 1.f;
    }
    float unit[kU][2];               // of keys lane / 4 and + 8
    if constexpr (!kSplit) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          unit[u][i] = __shfl_sync(0xffffffffu, kU == 4 ? unit2[u / 2] : u0 ? unit2[1] : unit2[0],
                                   lane / 4 + 8 * i + 16 * (u & 1));
    }
    float p[kU][kN][4], sum_l[kN][2];            // p: what is multiplied with the values' scales
    constexpr float kMost = kSplit ? kMostSum : kMostWeight;
    bool above = false;
    auto weigh = [&] {
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const unsigned long long f = f2pack(factor[n][0], factor[n][1]);
        const unsigned long long less = f2pack(-m[n][0], -m[n][1]);
        unsigned long long sum = 0, scaled = 0;
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float t0, t1;
            f2unpack(fma2(f2pack(z[u][n][2 * i], z[u][n][2 * i + 1]), f, less), t0, t1);
            unsigned long long both = f2pack(exp2_fast(t0), exp2_fast(t1));
            sum = u + i == 0 ? both : add2(sum, both);
            if constexpr (!kSplit) {
              const float by = unit[u][i];
              both = mul2(both, f2pack(by, by));
              scaled = u + i == 0 ? both : add2(scaled, both);
            }
            f2unpack(both, p[u][n][2 * i], p[u][n][2 * i + 1]);
          }
        f2unpack(sum, sum_l[n][0], sum_l[n][1]);
        above |= sum_l[n][0] > kMost || sum_l[n][1] > kMost;
        if constexpr (!kSplit) {
          float t0, t1;
          f2unpack(scaled, t0, t1);
          above |= t0 > kMostSum || t1 > kMostSum;
        }
      }
    };
    weigh();
    if (__any_sync(0xffffffffu, above)) {
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        float top[2] = {-INFINITY, -INFINITY}, f[2];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float t = __fmul_rn(z[u][n][i], factor[n][i & 1]);
            float& to = top[i & 1];
            if constexpr (kSplit) {
              to = fmaxf(to, t - kBoost);
            } else {
              const float by = unit[u][i / 2];
              const float log2 = (float)((int)(__float_as_uint(by) >> 23) - 127);
              to = fmaxf(to, fmaxf(t - kRoom, by > 0.f ? t + log2 - kBoost : -INFINITY));
            }
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int x = 4; x < 32; x *= 2)
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], x));
          top[i] = fmaxf(m[n][i], top[i]);
          f[i] = exp2_fast(m[n][i] - top[i]);
          l[n][i] *= f[i];
          m[n][i] = top[i];
          far |= fabsf(top[i]) > kFar && top[i] > kLowest;
        }
        const unsigned long long ff = f2pack(f[0], f[1]), none = 0;
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) o[c][t][n][i] = fma2(o[c][t][n][i], ff, none);
      }
      far = __any_sync(0xffffffffu, far);
      // (here whatever the maximum: a branch more is 1 % of 200 contexts of up to 900 keys)
#pragma unroll
      for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) z[u][n][i] = __fmul_rn(z[u][n][i], factor[n][i & 1]);
        factor[n][0] = factor[n][1] = 1.f;
      }
      weigh();
    }
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) l[n][i] += sum_l[n][i];
    uint32_t pt[kWeights][kU][kN][2];      // weights as right operand: keys in pairs, a column a head
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float lo = p[u][n][2 * i], hi = p[u][n][2 * i + 1];
          if constexpr (!kSplit) {
            pt[0][u][n][i] = turn8(pack_half(lo, hi));
          } else {
#pragma unroll
            for (int part = 0; part < kWeights; ++part) {
              const uint32_t h = pack_bf(lo, hi);
              pt[part][u][n][i] = turn8(h);
              lo -= __uint_as_float(h << 16);
              hi -= __uint_as_float(h & 0xffff0000u);
            }
          }
        }
    // two units' values at a time; in a loop where heads are large (128: 124 us so, 127 unrolled; a million
    // keys of 64: 45.9 and 45.0)
    constexpr int kUnroll = D <= 64 ? 2 : 1;
#pragma unroll kUnroll
    for (int v0 = 0; v0 < kU; v0 += 2) {
#pragma unroll
      for (int c0 = 0; c0 < kC; c0 += kP) {
        uint32_t x[2][kP][2];
        words<true>(vt, u0 + v0, c0, x);
        // the values' scales, of keys (lane % 4) * 2, + 1 (i = 0), + 8, + 9 (1) of every 16, as the right
        // operand has them
        constexpr int kWords = kSplit ? 2 : 1;
        uint32_t w[2][2][kP * kWords];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            load_shared(sv + ((8 * (u0 + v0 + u) + 4 * i + lane % 4) * kC + c0) * 4 * kWords, w[u][i]);
#pragma unroll
        for (int k = 0; k < kP; ++k) {
          uint32_t y[2][8];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // codes 0 and 1, then 2 and 3 of each word: in bf16 the lower one, and both as a byte
              if constexpr (kSplit) {
                const uint32_t x0 = x[u][k][i], x1 = x0 >> 8;
                const uint32_t f = w[u][i][k * kWords], less = w[u][i][k * kWords + kWords - 1];
                y[u][2 * i] = value_lo(x0, f, less);
                y[u][2 * i + 1] = value_hi(x0, f, less);
                y[u][4 + 2 * i] = value_lo(x1, f, less);
                y[u][5 + 2 * i] = value_hi(x1, f, less);
              } else {
                const uint32_t x0 = x[u][k][i] & 0x00ff00ffu, x1 = __byte_perm(x[u][k][i], 0, 0x4341);
                y[u][2 * i] = code_lo<true>(x0);
                y[u][2 * i + 1] = code_pair(x0);
                y[u][4 + 2 * i] = code_lo<true>(x1);
                y[u][5 + 2 * i] = code_pair(x1);
              }
            }
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            float sum[2][4];
            // the smallest parts first: what a sum is cut by goes with its size
#pragma unroll
            for (int part = kWeights - 1; part >= 0; --part)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t ps[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  ps[i] = pt[part][(kUnroll == 1 ? 0 : v0) + u][n][i];
                  if constexpr (!kSplit) ps[i] = mul_half(ps[i], w[u][i][k]);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  const uint32_t* v = y[u] + 4 * t;
                  if constexpr (kSplit) {
                    if (u == 0 && part == kWeights - 1)
                      mma_bf16(sum[t], v[0], v[1], v[2], v[3], ps, 0.f, 0.f, 0.f, 0.f);
                    else
                      mma_bf16(sum[t], v[0], v[1], v[2], v[3], ps);
                  } else {
                    if (u == 0)
                      mma_f16(sum[t], v[0], v[1], v[2], v[3], ps, 0.f, 0.f, 0.f, 0.f);
                    else
                      mma_f16(sum[t], v[0], v[1], v[2], v[3], ps);
                  }
                }
              }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                o[c0 + k][t][n][i] = add2(f2pack(sum[t][2 * i], sum[t][2 * i + 1]), o[c0 + k][t][n][i]);
          }
        }
      }
      if constexpr (kU > 2 && kUnroll == 1) {    // the next two units' weights
#pragma unroll
        for (int part = 0; part < kWeights; ++part)
#pragma unroll
          for (int u = 0; u + 2 < kU; ++u)
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) pt[part][u][n][i] = pt[part][u + 2][n][i];
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
        float base = m[n][i], sum = l[n][i];
        if constexpr (!kSplit) {
          // A large sum is brought to 2^8, for the sake of its logarithm (whose error goes with its size, and values'
          // powers of two go into it), by what the base can be raised by: of scores beyond 2^24 perhaps nothing.
          if (sum > 4096.f && sum < INFINITY) {
            const float raised = base + (float)((int)(__float_as_uint(sum) >> 23) - 135);
            sum *= exp2_fast(base - raised);
            base = raised;
          }
        }
        if (lane < 4) ml[8 * n + lane * 2 + i] = make_float2(base, sum);
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
        // values are 2^-21 of theirs, or codes 2^-9
        const float f = exp2_fast(m[n][i] - top(r)) * (kSplit ? 2097152.f : 512.f);
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            float x[2], y[2];
            f2unpack(o[c][k / 2][n][0], x[0], x[1]);
            f2unpack(o[c][k / 2][n][1], y[0], y[1]);
            float* to = dst + r * D + 32 * c + 4 * (lane / 4);
            to[k ^ spread(r)] = x[i] * f;
            // 16 times the upper code's; or of a pair (2^-13 of its number), less its lower code
            to[(k + 1) ^ spread(r)] = (kSplit ? y[i] : 16.f * y[i] - x[i]) * (f * 0.0625f);
          }
      }
  }
};

// ---------------------------------------------------------------------------
// A place in a share: the tiles of a segment that lie in it, one after the other, then the next segment's.
// ---------------------------------------------------------------------------
template <typename S>
struct Portion {
  Cursor at;               // t: the next tile
  int left;                // tiles of this segment from here on that are the share's; 0: none

  __device__ __forceinline__ void enter(long long end) {
    left = (int)max(0ll, min((long long)(at.span.tiles - at.t), end - (at.segment + at.t)));
  }
  // the segment behind this one, and whether it begins in the share
  __device__ __forceinline__ bool skip(const PagedLayout& pg, int window, int HR, long long end) {
    at.t = at.span.tiles - 1;
    advance<S>(at, pg, window, HR);
    return at.segment < end;
  }
  __device__ __forceinline__ void step(const PagedLayout& pg, int window, int HR, long long end) {
    ++at.t;
    if (--left > 0) return;
    if (at.t < at.span.tiles || !skip(pg, window, HR, end)) {
      left = 0;
      return;
    }
    enter(end);
  }
};

// ---------------------------------------------------------------------------
// The warp's loader: rows and scales as they lie, 16 keys of a page at a time (a page holds as many).
// ---------------------------------------------------------------------------
template <typename T, int D, int RT, int TEAMS>
struct Q4Loader {
  using S = Q4Shape<T, D, RT, TEAMS>;
  using Mask = typename S::Mask;
  static constexpr Mask kAll = (Mask)(~0ull >> (64 - S::kKeys));
  static constexpr int kEach = S::kKeys / 32;      // keys whose page a lane looks up
  Portion<S> p;
  long long end;           // of the share
  struct Rows {            // a warp's keys of a tile
    int page, key0, head;  // page: of this lane's first key
    Mask mask;             // those to be seen
  };

  __device__ __forceinline__ Rows look_up(const PagedAttnQ4Args<T>& a, int HR) {
    Rows r{0, 0, 0, 0};
    if (p.left == 0) return r;
    r.key0 = p.at.span.base + p.at.t * S::kTile + S::warp() * S::kKeys;
    const int lo = p.at.span.first - r.key0, hi = p.at.span.len - r.key0;
    int key = r.key0 + (threadIdx.x & 31) * kEach;
    if (lo <= 0 && hi >= S::kKeys) {
      r.mask = kAll;
    } else if (lo < S::kKeys && hi > 0) {
      r.mask = (kAll << max(lo, 0)) & (kAll >> max(S::kKeys - hi, 0));
      // lanes whose key is not to be seen read the first one's page
      if (!((r.mask >> ((threadIdx.x & 31) * kEach)) & 1)) key = r.key0 + max(lo, 0);
    }
    if (r.mask) {
      r.head = a.row_blocks == 1 ? p.at.hr : p.at.hr / a.row_blocks;
      r.page = a.paged.table[(long long)p.at.s * a.paged.width + (key >> a.paged.page_log2)];
    }
    p.step(a.paged, a.window, HR, end);
    return r;
  }

  __device__ __forceinline__ static void issue(const PagedAttnQ4Args<T>& a, const Rows& r, uint32_t stage,
                                               Mask* mask_out) {
    const int lane = threadIdx.x & 31;
    Mask mask = r.mask;
    const unsigned wrong =
        __ballot_sync(0xffffffffu, mask != 0 && (unsigned)r.page >= (unsigned)a.paged.num_pages);
    if (wrong) {
      if (lane == 0) flag_error(a.status, kDevErrBadIndex);
      for (int i = 0; i < 32; ++i)
        if ((wrong >> i) & 1) mask &= ~((Mask)((1u << kEach) - 1) << (kEach * i));
    }
    if (lane == 0) *mask_out = mask;
    if (mask) {
      const int log2 = a.paged.page_log2, in_page = (1 << log2) - 1;
      // a page's bytes of one head: 16 codes' and one scale byte for every chunk
      const long long head_bytes = (long long)(17 * S::kChunks) << log2;
      const int scales_at = S::kRowBytes << log2;
      constexpr int kPasses = S::kCodes / 512;
      constexpr int kPieces = S::kScales / 16, kOf = 16 / S::kChunks;      // 16 bytes of scales: kOf rows'
      if (mask == kAll && (1 << log2) >= S::kKeys) {
        // all rows of one page: they and their scales lie one behind the other
        const int row = r.key0 & in_page;
        const long long head0 = ((long long)r.page * a.Hkv + r.head) * head_bytes;
        const long long off = head0 + row * S::kRowBytes + lane * 16;
        const uint8_t *k = a.k_cache + off, *v = a.v_cache + off;
        const uint32_t dst = stage + lane * 16;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          copy16(dst + i * 512, k + i * 512, true);
          copy16(dst + S::kCodes + i * 512, v + i * 512, true);
        }
        if (lane < 2 * kPieces)
          copy16(dst + 2 * S::kCodes,
                 (lane < kPieces ? a.k_cache : a.v_cache) + head0 + scales_at + row * S::kChunks +
                     lane % kPieces * 16,
                 true);
      } else {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int row = (i * 32 + lane) / S::kChunks;
          const int page = __shfl_sync(0xffffffffu, r.page, row / kEach);
          const bool live = (mask >> row) & 1;
          const long long off = ((long long)page * a.Hkv + r.head) * head_bytes +
                                ((r.key0 + row) & in_page) * S::kRowBytes + lane % S::kChunks * 16;
          const uint32_t dst = stage + (i * 32 + lane) * 16;
          copy16(dst, a.k_cache + (live ? off : 0), live);
          copy16(dst + S::kCodes, a.v_cache + (live ? off : 0), live);
        }
        const int piece = lane % kPieces, row = piece * kOf;
        const int page = __shfl_sync(0xffffffffu, r.page, row / kEach);
        if (lane < 2 * kPieces) {
          const bool live = (unsigned)(mask >> row) & ((1u << kOf) - 1);
          const long long off = ((long long)page * a.Hkv + r.head) * head_bytes + scales_at +
                                ((r.key0 + row) & in_page) * S::kChunks;
          copy16(stage + 2 * S::kCodes + lane * 16,
                 (lane < kPieces ? a.k_cache : a.v_cache) + (live ? off : 0), live);
        }
      }
    }
    copy_commit();
  }
};

// Counts a part of the segment that share c0 begins, of n parts in all, as count_up does; returns those
// counted before.  A CTA's shares have one counter, which is enough: segments of at most TEAMS parts
// that one of them but the last begins have a field each (a bit or two more than their parts need), and of
// all others there is one at most, since shares inside of a segment begin none.
template <int TEAMS>
__device__ __forceinline__ int count_part(unsigned long long* counters, int c0, int n,
                                          unsigned long long base) {
  constexpr int kBits = TEAMS == 2 ? 2 : 3, kRest = (TEAMS - 1) * kBits;
  static_assert(TEAMS < 1 << kBits, "a field holds its parts");
  const int which = c0 % TEAMS, shift = which < TEAMS - 1 && n <= TEAMS ? which * kBits : kRest;
  unsigned long long* const counter = counters + c0 / TEAMS;
  unsigned long long old;
  asm volatile("red.relaxed.gpu.global.max.u64 [%0], %1;" ::"l"(counter), "l"(base) : "memory");
  asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], %2;"
               : "=l"(old)
               : "l"(counter), "l"(1ull << shift)
               : "memory");
  const int count = (int)(old - base) >> shift;
  return shift < kRest ? count & ((1 << kBits) - 1) : count;
}
// The most parts that the rest of a counter's bits can count.
constexpr int most_parts(int teams) {
  return (1 << (kCountBits - (teams - 1) * (teams == 2 ? 2 : 3))) - 1;
}

// As paged_attn_kernel (paged_row.cuh), with several shares to a CTA, each a team of warps': ends of segments
// are some thousand cycles of latency, during which other teams have the SM.  And each team has its
// queries in shared memory, put there by a warp for each chunk while the segment before ends.
template <typename K>
__global__ void __launch_bounds__(K::S::kThreads, 1)
paged_attn_q4_kernel(const __grid_constant__ typename K::Args a) {
  using T = typename K::Type;
  using S = typename K::S;
  using State = typename K::State;
  using Ld = typename K::Ld;
  using Team = typename K::Team;
  using Mask = typename S::Mask;
  constexpr int D = K::kD, RT = K::kRT, kTeamWarps = S::kTeamWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, tw = S::warp(), team = Team::team();
  const int worker = blockIdx.x * S::kTeams + team, workers = gridDim.x * S::kTeams;
  const int HR = a.Hkv * a.row_blocks, Hq = a.Hkv * a.G;
  const uint32_t ring = smem_addr(smem) + warp * S::kRing;
  constexpr int kSets = S::kQuerySets;
  const uint32_t queries = smem_addr(smem) + S::kOffQueries + team * kSets * S::kQueries;
  float2* const ml = reinterpret_cast<float2*>(smem + S::kOffMl) + team * kTeamWarps * RT;
  Mask* const masks = reinterpret_cast<Mask*>(smem + S::kOffMask) + warp * S::kStages;
  // of the segment that another share begins, and of the one that another share ends
  Join* const joins = reinterpret_cast<Join*>(smem + S::kOffJoins) + team * 2;
  auto* const base = reinterpret_cast<unsigned long long*>(smem + S::kOffBase) + team * 2;

  griddep_wait();
  griddep_launch();
  unsigned long long call = 0;
  if (threadIdx.x == 0) call = count_call(a.counters + kCallNumber);     // looked at further below
  const Share share = my_share<S>(a.paged, a.window, HR, worker, workers);
  Portion<S> p;
  p.at = share.at;
  const Cursor& at = p.at;
  const bool busy = at.segment + at.t < share.end;
  if (Team::thread() < 2) joins[Team::thread()] = {};  // read behind the barriers of the share's end
  if (busy) p.enter(share.end); else p.left = 0;
  // a segment's first query head and its query rows
  auto head_of = [&](const Cursor& c, int& head, int& rows) {
    const int kv = a.row_blocks == 1 ? c.hr : c.hr / a.row_blocks, rb = c.hr - kv * a.row_blocks;
    head = kv * a.G + rb * RT;
    rows = min(RT, a.G - rb * RT);
  };
  auto put_queries = [&](const Cursor& c, int which) {
    int head, rows;
    head_of(c, head, rows);
    for (int chunk = tw; chunk < S::kChunks; chunk += kTeamWarps)
      State::put_queries(a, c.s, head, rows, chunk, queries + which * S::kQueries);
  };
  Ld ld;
  ld.p = p;
  ld.end = share.end;
  typename Ld::Rows coming{};
  if (busy) {
    typename Ld::Rows rows_of[S::kStages];
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) rows_of[i] = ld.look_up(a, HR);   // their loads together
#pragma unroll 1
    for (int i = 0; i < S::kStages - 1; ++i) {
      ld.issue(a, rows_of[0], ring + i * S::kStageBytes, masks + i);
#pragma unroll
      for (int j = 1; j < S::kStages; ++j) rows_of[j - 1] = rows_of[j];
    }
    coming = rows_of[0];
    put_queries(at, 0);
  }
  // the call's number, from thread 0 to all teams, with the queries
  if (threadIdx.x == 0)
    for (int i = 0; i < S::kTeams; ++i)
      reinterpret_cast<unsigned long long*>(smem + S::kOffBase)[2 * i] = call / kCallStep << kCountBits;
  __syncthreads();
  if (busy) {
    State st;
    ScoreRule rule;
    rule.scale2 = a.scale * kLog2e;
    rule.cap = a.softcap;
    // finite, so that a score of zero stays one under the smallest caps too
    rule.rcap = a.softcap > 0.f ? fminf(fmaxf(a.scale / a.softcap, -FLT_MAX), FLT_MAX) : 0.f;
    rule.plain = a.softcap == 0.f && a.slopes == nullptr && a.scale >= 0.f;
    int slot = 0, next = S::kStages - 1;     // stages: of this tile, of the next one to issue
    int from = at.t, which = 0;
    bool begin = true, seen = false;         // seen: this warp has seen a key of the segment
    do {
      if (begin) {
        rule.last = at.span.len - 1;
        from = at.t;
        st.start();
        begin = seen = false;
        // the next segment's queries are brought near
        Portion<S> then = p;
        if (then.skip(a.paged, a.window, HR, share.end)) {
          int head, rows;
          head_of(then.at, head, rows);
          constexpr int kLines = (D * (int)sizeof(T) + 127) / 128;      // of a row
          const int r = Team::thread() / kLines;
          if (r < rows)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(
                reinterpret_cast<const char*>(a.q + then.at.s * a.q_s + (long long)(head + r) * a.q_h) +
                Team::thread() % kLines * 128));
        }
      }
      copy_wait<S::kStages - 2>();
      __syncwarp();
      ld.issue(a, coming, ring + next * S::kStageBytes, masks + next);
      coming = ld.look_up(a, HR);
      const Mask mask = masks[slot];
      if (mask) {
        seen = true;
        st.tile(rule, queries + which * S::kQueries, ring + slot * S::kStageBytes,
                at.span.base + at.t * S::kTile + tw * S::kKeys, mask);
      }
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
      next = next + 1 == S::kStages ? 0 : next + 1;

      if (p.left > 1) {
        ++p.at.t;
        --p.left;
      } else {
        // join the warps' parts
        const int read = slot == 0 ? S::kStages - 1 : slot - 1;
        const bool ends = at.t + 1 == at.span.tiles;
        int head, rows;
        head_of(at, head, rows);
        st.put_ml(ml + tw * RT);
        Portion<S> then = p;
        const bool more = ends && then.skip(a.paged, a.window, HR, share.end);
        if (more && kSets == 2) put_queries(then.at, which ^ 1);
        Team::sync();
        if (more && kSets == 1) put_queries(then.at, 0);
        const bool whole = ends && from == 0;
        const int part = worker * 2 + (from == 0 ? 1 : 0);
        auto top = [&](int r) {
          float t = ml[r].x;
#pragma unroll
          for (int w = 1; w < kTeamWarps; ++w) t = fmaxf(t, ml[w * RT + r].x);
          return t;
        };
        // Every warp's sums go to the stage that it has just read: no copy goes there until its
        // next tile.
        uint8_t* const sums = smem + team * kTeamWarps * S::kRing + read * S::kStageBytes;
        if (seen) st.put_o(reinterpret_cast<float*>(sums + tw * S::kRing), rows, top);
        Team::sync();
        for (int e = Team::thread(); e < rows * (D / 4); e += S::kTeamThreads) {
          const int r = e / (D / 4), c = e % (D / 4) * 4;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          const float tp = top(r);
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kTeamWarps; ++w) {
            const float2 z = ml[w * RT + r];
            if (z.y == 0.f) continue;          // it has seen nothing of the row, and left no sums
            const float4 y = *reinterpret_cast<const float4*>(sums + w * S::kRing + (r * D + c) * 4);
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
            sum = fmaf(z.y, exp2_fast(z.x - tp), sum);
          }
          // columns c + k of a row stand at c + (k ^ spread)
          const int turn = State::spread(r);
          if (turn & 1) x = make_float4(x.y, x.x, x.w, x.z);
          if (turn & 2) x = make_float4(x.z, x.w, x.x, x.y);
          if (whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            T* to = a.out + ((long long)at.s * Hq + head + r) * D + c;
            to[0] = from_f<T>(x.x * inv);
            to[1] = from_f<T>(x.y * inv);
            to[2] = from_f<T>(x.z * inv);
            to[3] = from_f<T>(x.w * inv);
            if (c == 0 && a.lse) a.lse[(long long)at.s * Hq + head + r] = lse_of(tp, sum);
          } else {
            reinterpret_cast<float4*>(a.part_o)[(((long long)part * RT + r) * D + c) / 4] = x;
            if (c == 0)
              reinterpret_cast<float2*>(a.part_ml)[(long long)part * RT + r] = make_float2(tp, sum);
          }
        }
        Team::sync();
        if (!whole && Team::thread() == 0) {
          // Whoever leaves a segment's last part joins them all, when its own share is done (the
          // others go on meanwhile): the count is asked for now, and looked at then.
          const int c0 = from == 0 ? worker : share_of(at.segment, share.row, workers);
          const int n = share_of(at.segment + at.span.tiles - 1, share.row, workers) - c0 + 1;
          const bool last = count_part<S::kTeams>(a.counters, c0, n, *base) == n - 1;
          joins[from == 0] = {(long long)at.s * Hq + head, c0, last ? n : 0, rows, 0};
        }
        begin = true;
        which = (which + 1) % kSets;
        p = then;
        if (more) p.enter(share.end); else p.left = 0;
      }
    } while (p.left > 0);
    copy_wait<0>();
    Team::sync();
    for (int i = 0; i < 2; ++i) {
      const Join x = joins[i];
      if (x.n == 0) continue;
      join_parts<K>(a.part_ml, a.part_o, a.out + x.row * D, a.lse ? a.lse + x.row : nullptr, x.c, x.n,
                    x.rows, reinterpret_cast<float*>(smem + team * kTeamWarps * S::kRing));
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

template <typename T, int D, int RT, int TEAMS>
struct Q4 {
  using Type = T;
  using Args = PagedAttnQ4Args<T>;
  using S = Q4Shape<T, D, RT, TEAMS>;
  using State = Q4State<T, D, RT, TEAMS>;
  using Ld = Q4Loader<T, D, RT, TEAMS>;
  using Team = Q4Team<S>;
  static constexpr int kD = D, kRT = RT;
  static auto kernel() { return paged_attn_q4_kernel<Q4>; }
};

// Four teams where there are that many segments, and the counters hold a segment's parts: tables of up to 127 tiles
// (24384 tokens for heads of 128, 16256 of them in fp32, 32512 for smaller heads), whatever the lengths.  16 rows are
// better off with two.
template <typename T, int D, int RT, typename F>
auto with_teams(int Hkv, int G, int S, int width, int page_log2, int sms, F f) {
  if constexpr (RT == 8) {
    using Four = Q4<T, D, RT, 4>;
    const long long segments = (long long)S * Hkv * ((G + RT - 1) / RT);
    const long long tiles = (((long long)width << page_log2) + Four::S::kTile - 1) / Four::S::kTile;
    if (segments >= 3LL * sms && tiles <= most_parts(4)) return f(Run<Four>{});
  }
  return f(Run<Q4<T, D, RT, 2>>{});
}

// A CTA takes 8 query rows, in bf16 16 where the group has more (128 sequences of up to 8192 keys, 128/8 heads
// of 128: 201 us, two segments of 8 rows 240; 64/4 heads of 32: 32 and 40); larger groups take several CTAs.
template <typename T, typename F>
auto with_shape(int d, int Hkv, int G, int S, int width, int page_log2, int sms, F f) {
  auto dim = [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    switch (d) {
      case 32: return with_teams<T, 32, RT>(Hkv, G, S, width, page_log2, sms, f);
      case 64: return with_teams<T, 64, RT>(Hkv, G, S, width, page_log2, sms, f);
      default: return with_teams<T, 128, RT>(Hkv, G, S, width, page_log2, sms, f);
    }
  };
  if constexpr (std::is_same<T, bf16>::value) {
    if (G > 8) return dim(std::integral_constant<int, 16>{});
  }
  return dim(std::integral_constant<int, 8>{});
}

}  // namespace

size_t paged_attn_q4_ws_bytes(int d, int Hkv, int G, int S, int width, int page_log2, int is_f32,
                              int sms) {
  auto bytes = [&](auto run) { return run.bytes(Hkv, G, S, width, page_log2, sms); };
  return is_f32 ? with_shape<float>(d, Hkv, G, S, width, page_log2, sms, bytes)
                : with_shape<bf16>(d, Hkv, G, S, width, page_log2, sms, bytes);
}

template <typename T>
cudaError_t launch_paged_attn_q4(PagedAttnQ4Args<T> a, int d, void* ws, int sms, cudaStream_t st) {
  return with_shape<T>(d, a.Hkv, a.G, a.paged.S, a.paged.width, a.paged.page_log2, sms,
                       [&](auto run) { return run.launch(a, ws, sms, st); });
}

template cudaError_t launch_paged_attn_q4<float>(PagedAttnQ4Args<float>, int, void*, int,
                                                 cudaStream_t);
template cudaError_t launch_paged_attn_q4<bf16>(PagedAttnQ4Args<bf16>, int, void*, int,
                                                cudaStream_t);

}  // namespace mita
