// Device helpers shared by the kernels that normalise and rotate heads (norm_rope.cu: whole
// sequences and their gradient; cache_append.cu: new tokens on their way into the cache).
//
// A head row of D values is worked on by D / 8 lanes, a slot.  Lane g holds eight values as two
// groups of four, chosen so that the rotation never leaves the lane and that the lanes' groups lie
// side by side: at 4g and rot/2 + 4g.  With the half-split pairing (i, i + rot/2) each value of
// the one group is the partner of one in the other; with the neighbouring pairing (2i, 2i + 1)
// each group holds two pairs.  The unrotated tail [rot, D) is split into halves likewise.  Hence
// rot % 8 == 0.
//
// A row is a few dozen bytes a lane, so the instructions around them decide whether HBM stays
// the bound (first measured form: 172 warp instructions a row of 128, 82 us for 336 MB; now 90
// and 57 us, of which copying alone takes 56).  So the arithmetic is on pairs of fp32 values (one
// instruction for two), a token's cosines and sines are multiplied with the weights once for all of
// its heads, and rows are normalised two at a time, their sums sharing one tree of shuffles.
#pragma once

#include "common.cuh"

namespace mita {

// Threads of a block in these kernels.
constexpr int kRopeThreads = 256;
// Blocks of an SM: with three, 80 registers a thread would not hold what the kernels keep (1M
// tokens of 2 + 2 heads: 199 us, with two 193 us; the gradient 54 and 49 us for 8192 tokens of 40).
constexpr int kRopeBlocks = 2;

using V2 = unsigned long long;   // two fp32 values
__device__ __forceinline__ V2 mul2(V2 a, V2 b) {
  V2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ V2 swap2(V2 v) {
  float a, b;
  f2unpack(v, a, b);
  return f2pack(b, a);
}
__device__ __forceinline__ float sum2(V2 v) {
  float a, b;
  f2unpack(v, a, b);
  return a + b;
}

// A lane's eight values: (a0, a1), (a2, a3), (b0, b1), (b2, b3).
struct V8 {
  V2 v[4];
};

// Four values of a row as they lie in memory (8 bytes of bf16, 16 of fp32), and as fp32.
template <typename T> struct Raw4;
template <> struct Raw4<float> {
  using Bits = float4;
  __device__ __forceinline__ static void unpack(const Bits& b, V2* o) {
    o[0] = f2pack(b.x, b.y);
    o[1] = f2pack(b.z, b.w);
  }
  __device__ __forceinline__ static Bits pack(const V2* o) {
    Bits b;
    f2unpack(o[0], b.x, b.y);
    f2unpack(o[1], b.z, b.w);
    return b;
  }
};
template <> struct Raw4<bf16> {
  using Bits = uint2;
  __device__ __forceinline__ static void unpack(const Bits& b, V2* o) {
    o[0] = f2pack(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u));
    o[1] = f2pack(__uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
  }
  // the one rounding of a result: to nearest, ties to even
  __device__ __forceinline__ static Bits pack(const V2* o) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float lo, hi;
      f2unpack(o[i], lo, hi);
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint2(w[0], w[1]);
  }
};
template <typename T>
struct Raw8 {
  typename Raw4<T>::Bits a, b;
  __device__ __forceinline__ V8 unpack() const {
    V8 x;
    Raw4<T>::unpack(a, x.v);
    Raw4<T>::unpack(b, x.v + 2);
    return x;
  }
  __device__ __forceinline__ void pack(const V8& x) {
    a = Raw4<T>::pack(x.v);
    b = Raw4<T>::pack(x.v + 2);
  }
  __device__ __forceinline__ void store(T* p, int oa, int ob) const {
    *reinterpret_cast<typename Raw4<T>::Bits*>(p + oa) = a;
    *reinterpret_cast<typename Raw4<T>::Bits*>(p + ob) = b;
  }
};

// Rows on their way from global memory to a thread, two at a time: a ring in shared memory of which
// every thread has its own column, filled by asynchronous copies kPairs ahead of use.  Nobody else
// reads a thread's column, so its own wait is all the synchronisation there is; and rows wait in
// shared memory, not in registers, so that loads are under way all the time.
template <typename T>
struct RowRing {
  using Bits = typename Raw4<T>::Bits;
  static constexpr int kPairs = 16 / (int)sizeof(T) / 2;        // 128 bytes a thread
  static constexpr int kGroup = kRopeThreads * (int)sizeof(Bits);   // [pair][row][group][thread]
  static constexpr int kBytes = kPairs * 4 * kGroup;
  uint32_t mine;          // this thread's column
  uint32_t at = 0;        // the pair that is used, then fetched, next

  __device__ __forceinline__ explicit RowRing(const void* mem)
      : mine((uint32_t)__cvta_generic_to_shared(mem) + threadIdx.x * sizeof(Bits)) {}
  // row 0 or 1 of the pair from p; zeros, and nothing read, where there is none
  template <int row>
  __device__ __forceinline__ void fetch(const T* p, int oa, int ob, bool there) const {
    const uint32_t to = mine + at;
    const int bytes = there ? (int)sizeof(Bits) : 0;
    copy<row * 2 * kGroup>(to, p + oa, bytes);
    copy<row * 2 * kGroup + kGroup>(to, p + ob, bytes);
  }
  __device__ __forceinline__ void next() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    at = (at + 4 * kGroup) & (kBytes - 1);
  }
  // returns once the oldest of kPairs committed pairs is there
  __device__ __forceinline__ static void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPairs - 1) : "memory");
  }
  __device__ __forceinline__ static void drain() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  template <int row>
  __device__ __forceinline__ Raw8<T> get() const {
    const uint32_t from = mine + at;
    return {load<row * 2 * kGroup>(from), load<row * 2 * kGroup + kGroup>(from)};
  }

 private:
  template <int off>
  __device__ __forceinline__ static void copy(uint32_t dst, const T* src, int bytes) {
    if constexpr (sizeof(Bits) == 16)
      asm volatile("cp.async.cg.shared.global [%0 + %1], [%2], 16, %3;" ::"r"(dst), "n"(off),
                   "l"(src), "r"(bytes)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0 + %1], [%2], 8, %3;" ::"r"(dst), "n"(off),
                   "l"(src), "r"(bytes)
                   : "memory");
  }
  template <int off>
  __device__ __forceinline__ static Bits load(uint32_t src) {
    Bits b;
    if constexpr (sizeof(Bits) == 16)
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4 + %5];"
                   : "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
                   : "r"(src), "n"(off)
                   : "memory");
    else
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];"
                   : "=r"(b.x), "=r"(b.y)
                   : "r"(src), "n"(off)
                   : "memory");
    return b;
  }
};

// A slot's way over the tokens of [B, N]: first, first + stride, ..., with the batch and the place in
// it.  step() says whether that stayed in the batch: rows then lie stride tokens further on, which
// is an addition, where a new batch takes a division and products.
struct TokenWalk {
  unsigned t, N;
  int b, n;
  __device__ __forceinline__ TokenWalk(unsigned first, unsigned N_) : t(first), N(N_) { place(); }
  __device__ __forceinline__ bool step(unsigned stride) {
    t += stride;
    n += stride;
    if ((unsigned)n < N) return true;
    place();
    return false;
  }
  __device__ __forceinline__ void place() {
    b = t / N;
    n = t - (unsigned)b * N;
  }
};

// The angle of frequency i at position p is p * inv_freq[i] radians.  In fp32 it would lose
// its fraction of a turn at far positions (an ulp of 10^6 is 1/16 radian), and fp64 arithmetic
// per token is slow on this part.  So each block turns the frequencies once into unsigned
// 64-bit fractions of a turn; p * fraction mod 2^64 is then the exact product modulo one turn
// (the frequency's own rounding, 2^-53 of it, is all that is lost), for any 32-bit p, negative
// ones included.  Frequencies from `half` on are 0: their cosine is 1 and their sine 0, exactly,
// so lanes whose values are not turned need no branch.
template <int D>
__device__ __forceinline__ void rope_table(const double* inv_freq, int half,
                                           unsigned long long* turn) {
  for (int i = threadIdx.x; i < D / 2; i += blockDim.x) {
    double f = i < half ? inv_freq[i] * 0.15915494309189533577 : 0.0;   // 1 / (2 pi)
    f -= rint(f);                                      // whole turns do nothing; |f| <= 1/2
    turn[i] = (unsigned long long)__double2ll_rn(f * 18446744073709551616.0);   // saturates
  }
}

// cos and sin of four pairs, each at its position p: the angle's top 32 bits, less the nearest quarter
// turn, give |x| <= pi / 4 to fp32's 24 bits; the Taylor series of sine to x^9 and of cosine to
// x^10 end below 2e-9 there; the quarter swaps them and sets the signs.
__device__ __forceinline__ void rope_angles(const unsigned long long* const (&turn)[2],
                                            const int (&at)[4], V2* cs, V2* sn) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t quarter[2];     // the nearest quarter turn in the top two bits
    float r[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned long long f = turn[i][j];
      const int p = at[2 * i + j];
      const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32);
      const uint32_t u = __umulhi((uint32_t)p, lo) + (uint32_t)p * hi - (p < 0 ? lo : 0u);
      quarter[j] = u + 0x20000000u;
      r[j] = (float)(int)(u - (quarter[j] & 0xc0000000u));
    }
    auto both = [](float x) { return f2pack(x, x); };
    const V2 x = mul2(f2pack(r[0], r[1]), both(1.4629180792671596e-9f));   // 2 pi / 2^32
    const V2 y = mul2(x, x);
    V2 s = fma2(y, both(2.7557319e-6f), both(-1.9841270e-4f));       // 1/9!, 1/7!
    s = fma2(y, s, both(8.3333333e-3f));                             // 1/5!
    s = fma2(y, s, both(-1.6666667e-1f));                            // 1/3!
    s = fma2(mul2(x, y), s, x);
    V2 c = fma2(y, both(-2.7557319e-7f), both(2.4801587e-5f));       // 1/10!, 1/8!
    c = fma2(y, c, both(-1.3888889e-3f));                            // 1/6!
    c = fma2(y, c, both(4.1666667e-2f));                             // 1/4!
    c = fma2(y, c, both(-0.5f));
    c = fma2(y, c, both(1.f));
    float ss[2], cc[2];
    f2unpack(s, ss[0], ss[1]);
    f2unpack(c, cc[0], cc[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool odd = quarter[j] & 0x40000000u;
      const uint32_t co = __float_as_uint(odd ? ss[j] : cc[j]);
      const uint32_t si = __float_as_uint(odd ? cc[j] : ss[j]);
      cc[j] = __uint_as_float(co ^ ((quarter[j] + 0x40000000u) & 0x80000000u));
      ss[j] = __uint_as_float(si ^ (quarter[j] & 0x80000000u));
    }
    cs[i] = f2pack(cc[0], cc[1]);
    sn[i] = f2pack(ss[0], ss[1]);
  }
}

__device__ __forceinline__ void rope_angles(const unsigned long long* const (&turn)[2], int p,
                                            V2* cs, V2* sn) {
  const int at[4] = {p, p, p, p};
  rope_angles(turn, at, cs, sn);
}

// What a lane knows of its place in a row.
struct RopeLane {
  int a, b;              // its groups of four values
  bool turned;           // whether they are rotated at all
  const unsigned long long* turn[2];   // its four frequencies in rope_table's table, two and two
  __device__ __forceinline__ RopeLane(int g, int D, int rot, bool inter,
                                      const unsigned long long* table) {
    turned = 8 * g < rot;
    a = turned ? 4 * g : rot + (4 * g - rot / 2);
    b = a + (turned ? rot : D - rot) / 2;
    turn[0] = table + (!turned ? rot / 2 : inter ? 2 * g : 4 * g);
    turn[1] = table + (!turned ? rot / 2 : inter ? rot / 4 + 2 * g : 4 * g + 2);
  }
};

// Where a slot's tokens stand, one position for all frequencies (positions [B][N], or 0 .. N - 1).
struct OnePosition {
  const int32_t* positions;
  long long pos_b;
  template <typename Args>
  __device__ __forceinline__ OnePosition(const Args& a, const RopeLane&, const unsigned long long*,
                                         unsigned, unsigned)
      : positions(a.positions), pos_b(a.pos_b) {}
  __device__ __forceinline__ void angles(const RopeLane& lane, const TokenWalk& at, bool live, V2* cs,
                                         V2* sn) {
    rope_angles(lane.turn, positions && live ? positions[at.b * pos_b + at.n] : at.n, cs, sn);
  }
};

// Where they stand on several axes (positions [axes][B][N]), each frequency turning with its axis.  The
// next token's positions are loaded before this one's rows are worked on: a slot's tokens are far
// apart, so that each load is a new line.
struct AxisPositions {
  const int32_t* from[4];          // of this lane's frequencies
  int next[4];
  TokenWalk at;
  long long pos_b;
  unsigned tokens, stride;
  template <typename Args>
  __device__ __forceinline__ AxisPositions(const Args& a, const RopeLane& lane,
                                           const unsigned long long* table, unsigned first,
                                           unsigned stride_)
      : at(first, a.N), pos_b(a.pos_b), tokens((unsigned)a.B * a.N), stride(stride_) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int f = (int)(lane.turn[i / 2] - table) + i % 2;
      int axis = f < a.rot / 2 ? a.freq_axis[f] : 0;
      if (axis < 0 || axis >= a.axes) {
        flag_error(a.status, kDevErrBadIndex);
        axis = 0;
      }
      from[i] = a.positions + axis * a.pos_a;
    }
    load();
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int i = 0; i < 4; ++i) next[i] = at.t < tokens ? from[i][at.b * pos_b + at.n] : 0;
  }
  __device__ __forceinline__ void angles(const RopeLane& lane, const TokenWalk&, bool, V2* cs, V2* sn) {
    int p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = next[i];
    at.step(stride);
    load();
    rope_angles(lane.turn, p, cs, sn);
  }
};

// A token's rotation with the weights worked in: y = x * c + partner(x) * s, the partner of a value
// being the other one of its pair.  (Taken by all lanes: a branch around the second product for
// those that are not turned cost 27 instructions a row of 98 in register moves.)
template <bool INTER>
struct RopeCoef {
  V8 c, s;
  // the rotation by (cs, sn), or back, after the weights w
  __device__ __forceinline__ void set(const V2* cs, const V2* sn, const V8& w, bool back = false) {
    const float sign = back ? -1.f : 1.f;
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float c0, c1, s0, s1;
        f2unpack(cs[i / 2], c0, c1);
        f2unpack(sn[i / 2], s0, s1);
        const float co = i % 2 ? c1 : c0, si = i % 2 ? s1 : s0;
        c.v[i] = mul2(f2pack(co, co), w.v[i]);
        s.v[i] = mul2(f2pack(-sign * si, sign * si), swap2(w.v[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        c.v[i] = mul2(cs[i], w.v[i]);
        c.v[i + 2] = mul2(cs[i], w.v[i + 2]);
        s.v[i] = mul2(mul2(sn[i], f2pack(-sign, -sign)), w.v[i + 2]);
        s.v[i + 2] = mul2(mul2(sn[i], f2pack(sign, sign)), w.v[i]);
      }
    }
  }
  __device__ __forceinline__ V8 of(const V8& x) const {
    V8 y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y.v[i] = fma2(INTER ? swap2(x.v[i]) : x.v[i ^ 2], s.v[i], mul2(x.v[i], c.v[i]));
    return y;
  }
};
__device__ __forceinline__ V8 ones8() {
  const V2 o = f2pack(1.f, 1.f);
  return {{o, o, o, o}};
}
__device__ __forceinline__ V8 weights8(const float* w, const RopeLane& lane) {
  V8 x;
  Raw4<float>::unpack(*reinterpret_cast<const float4*>(w + lane.a), x.v);
  Raw4<float>::unpack(*reinterpret_cast<const float4*>(w + lane.b), x.v + 2);
  return x;
}

// Sums of two values over the D / 8 lanes of a slot (all 32 lanes of the warp call it): one half of
// the slot adds up p, the other q, and f of each half's sum is exchanged at the end.
template <int D, typename F>
__device__ __forceinline__ void slot_sum2(float& p, float& q, F f) {
  constexpr int L = D / 8;
  const bool upper = threadIdx.x & (L / 2);
  float mine = upper ? q : p;
  mine += __shfl_xor_sync(0xffffffffu, upper ? p : q, L / 2);
#pragma unroll
  for (int o = L / 4; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  mine = f(mine);
  const float other = __shfl_xor_sync(0xffffffffu, mine, L / 2);
  p = upper ? other : mine;
  q = upper ? mine : other;
}

// Two rows of a token (the second may be absent: `rows` = 1), normalised where `normed`, rotated and
// stored to y and y + y_h.  All lanes of a warp call it; `live`: this lane has rows; `turned`: its
// values are rotated (a value that is neither normalised nor turned goes through bit for bit).
template <typename T, int D, bool INTER>
__device__ __forceinline__ void rope_pair(const RopeLane& lane, const RopeCoef<INTER>& coef,
                                          Raw8<T> r0, Raw8<T> r1, T* y, long long y_h, int rows,
                                          bool normed, bool turned, bool live, float eps) {
  if (normed) {
    V8 v[2] = {r0.unpack(), r1.unpack()};
    float r[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      V2 ss = mul2(v[k].v[0], v[k].v[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) ss = fma2(v[k].v[j], v[k].v[j], ss);
      r[k] = sum2(ss);
    }
    slot_sum2<D>(r[0], r[1], [&](float s) { return rsqrtf(fmaf(s, 1.f / D, eps)); });
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const V2 rr = f2pack(r[k], r[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[k].v[j] = mul2(v[k].v[j], rr);
    }
    r0.pack(coef.of(v[0]));
    r1.pack(coef.of(v[1]));
  } else if (turned) {
    r0.pack(coef.of(r0.unpack()));
    r1.pack(coef.of(r1.unpack()));
  }
  if (live) {
    r0.store(y, lane.a, lane.b);
    if (rows > 1) r1.store(y + y_h, lane.a, lane.b);
  }
}

// The grid of such a kernel: `tokens` tokens of `heads` rows each, `slots` tokens to a block at a
// time, `blocks` blocks to an SM.  A block goes over its tokens with a run of `run` heads, the
// blockIdx.y-th.  A short run spreads few tokens better; a token's angles and places, worth about
// four rows of arithmetic, are then computed for fewer rows: the least cost is that of the fullest
// SM's share.  No run is longer than kRopeRun: the blocks of the first runs come first, and
// fewer heads' rows are then written at a time, each head's to a place of its own (2 x 8191 tokens
// of 40 heads: runs of 40 65 us, of 20 57 us, of 8 62 us; measured at that shape alone).
constexpr int kRopeRun = 20;
struct RopeGrid {
  int run, x, y;
};
inline RopeGrid rope_grid(long long tokens, int heads, int slots, int blocks, int sms) {
  RopeGrid best{};
  long long least = 0;
  const long long per_run = (tokens + slots - 1) / slots;
  for (int run = 1; run == 1 || (run < 2 * heads && run <= kRopeRun); ++run) {
    const int y = (heads + run - 1) / run;
    if (run > 1 && (heads + y - 1) / y != run) continue;    // runs of equal length only
    long long share = (per_run * y + sms - 1) / sms;
    if (share < blocks) share = blocks;         // an SM's blocks run side by side
    const long long cost = share * (run + 4);
    if (best.run == 0 || cost < least) {
      const long long most = (long long)blocks * sms;
      best = {run, (int)(per_run < most ? per_run : most), y};
      least = cost;
    }
  }
  while (best.y > 65535) {                      // a grid's limit
    best.run *= 2;
    best.y = (heads + best.run - 1) / best.run;
  }
  return best;
}

}  // namespace mita
