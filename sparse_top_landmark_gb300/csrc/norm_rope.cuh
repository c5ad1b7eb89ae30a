// Device helpers shared by the kernels that normalise and rotate heads (norm_rope.cu: whole
// sequences and their gradient; cache_append.cu: new tokens on their way into the cache).
//
// A head row of D values is worked on by D / 8 lanes, a slot.  Lane g holds eight values as two
// groups of four, chosen so that the rotation never leaves the lane: with the half-split pairing
// (i, i + rot/2) the groups start at 4g and rot/2 + 4g, with the neighbouring pairing
// (2i, 2i + 1) at 8g and 8g + 4; the unrotated tail [rot, D) is taken as 8g, 8g + 4 either way.
// Hence rot % 8 == 0.  Either way the lane's pairs are the rotation's frequencies 4g .. 4g + 3.
//
// A row is a few dozen bytes a lane, so the instructions around them decide whether HBM stays
// the bound (first measured form: 172 warp instructions a row of 128, 82 us for 336 MB).  So the
// arithmetic is on pairs of fp32 values (one instruction for two), a token's cosines and sines are
// multiplied with the weights once for all of its heads, and rows are normalised two at a time, their
// sums sharing one tree of shuffles.
#pragma once

#include "common.cuh"

namespace mita {

// Threads of a block in these kernels.
constexpr int kRopeThreads = 256;
constexpr int kRopeBlocks = 3;            // blocks of an SM: forward and append
constexpr int kRopeBackwardBlocks = 2;    // gradient

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
  __device__ __forceinline__ void load(const T* p, int oa, int ob) {
    a = *reinterpret_cast<const typename Raw4<T>::Bits*>(p + oa);
    b = *reinterpret_cast<const typename Raw4<T>::Bits*>(p + ob);
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
  char* mine;             // this thread's column
  int at = 0;             // the pair that is used, then fetched, next

  __device__ __forceinline__ explicit RowRing(char* mem)
      : mine(mem + threadIdx.x * sizeof(Bits)) {}
  // row 0 or 1 of the pair from p
  __device__ __forceinline__ void fetch(int row, const T* p, int oa, int ob) const {
    copy(mine + at + row * 2 * kGroup, p + oa);
    copy(mine + at + row * 2 * kGroup + kGroup, p + ob);
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
  __device__ __forceinline__ Raw8<T> get(int row) const {
    const char* p = mine + at + row * 2 * kGroup;
    return {*reinterpret_cast<const Bits*>(p), *reinterpret_cast<const Bits*>(p + kGroup)};
  }

 private:
  __device__ __forceinline__ static void copy(char* dst, const T* src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (sizeof(Bits) == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
  }
};

// A slot's way over the tokens of [B, N]: first, first + stride, ..., with the batch and the place
// in it (a division only where a step leaves the batch).
struct TokenWalk {
  unsigned t, N;
  int b, n;
  __device__ __forceinline__ TokenWalk(unsigned first, unsigned N_) : t(first), N(N_) { place(); }
  __device__ __forceinline__ void step(unsigned stride) {
    t += stride;
    n += stride;
    if ((unsigned)n >= N) place();
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
// ones included.
__device__ __forceinline__ void rope_table(const double* inv_freq, int half,
                                           unsigned long long* turn) {
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    double f = inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
    f -= rint(f);                                      // whole turns do nothing; |f| <= 1/2
    turn[i] = (unsigned long long)__double2ll_rn(f * 18446744073709551616.0);   // saturates
  }
}

// cos and sin of four pairs at position p: the angle's top 32 bits, less the nearest quarter
// turn, give |x| <= pi / 4 to fp32's 24 bits; the Taylor series of sine to x^9 and of cosine to
// x^10 end below 2e-9 there; the quarter swaps them and sets the signs.
__device__ __forceinline__ void rope_angles(const unsigned long long* turn, int p, V2* cs, V2* sn) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t quarter[2];     // the nearest quarter turn in the top two bits
    float r[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned long long f = turn[2 * i + j];
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

// What a lane knows of its place in a row.
struct RopeLane {
  int a, b;              // its groups of four values
  bool turned;           // whether they are rotated at all
  __device__ __forceinline__ RopeLane(int g, int rot, bool inter) {
    turned = 8 * g < rot;
    const bool split = !inter && turned;
    a = split ? 4 * g : 8 * g;
    b = split ? rot / 2 + 4 * g : 8 * g + 4;
  }
};

// A token's rotation with the weights worked in: y = x * c + partner(x) * s, the partner of a value
// being the other one of its pair.  A lane whose values are not turned has c = w and leaves s out.
template <bool INTER>
struct RopeCoef {
  V8 c, s;
  bool turned;
  // the weights w, and the rotation by (cs, sn); `back`: the rotation back
  __device__ __forceinline__ void set(bool turn, const V2* cs, const V2* sn, const V8& w,
                                      bool back = false) {
    turned = turn;
    c = w;
    s = w;
    if (!turn) return;
    const V2 minus = f2pack(-1.f, -1.f);
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float c0, c1, s0, s1, w0, w1;
        f2unpack(cs[i / 2], c0, c1);
        f2unpack(sn[i / 2], s0, s1);
        f2unpack(w.v[i], w0, w1);
        const float co = i % 2 ? c1 : c0, si = (i % 2 ? s1 : s0) * (back ? -1.f : 1.f);
        c.v[i] = f2pack(co * w0, co * w1);
        s.v[i] = f2pack(-si * w1, si * w0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const V2 neg = mul2(sn[i], minus);
        c.v[i] = mul2(cs[i], w.v[i]);
        c.v[i + 2] = mul2(cs[i], w.v[i + 2]);
        s.v[i] = mul2(back ? sn[i] : neg, w.v[i + 2]);
        s.v[i + 2] = mul2(back ? neg : sn[i], w.v[i]);
      }
    }
  }
  __device__ __forceinline__ V8 of(const V8& x) const {
    V8 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y.v[i] = mul2(x.v[i], c.v[i]);
    if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y.v[i] = fma2(INTER ? swap2(x.v[i]) : x.v[i ^ 2], s.v[i], y.v[i]);
    }
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
// stored to y and y + y_h.  All lanes of a warp call it; `live`: this lane has rows.
template <typename T, int D, bool INTER>
__device__ __forceinline__ void rope_pair(const RopeLane& lane, const RopeCoef<INTER>& coef,
                                          Raw8<T> r0, Raw8<T> r1, T* y, long long y_h, int rows,
                                          bool normed, bool live, float eps) {
  if (normed || coef.turned) {     // else values go through bit for bit
    V8 v[2] = {r0.unpack(), r1.unpack()};
    if (normed) {
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
    }
    r0.pack(coef.of(v[0]));
    r1.pack(coef.of(v[1]));
  }
  if (live) {
    r0.store(y, lane.a, lane.b);
    if (rows > 1) r1.store(y + y_h, lane.a, lane.b);
  }
}

// The grid of such a kernel: `tokens` tokens of `heads` rows each, `slots` tokens to a block at a
// time, `blocks` blocks to an SM.  A block goes over its tokens with a run of `run` heads
// (blockIdx.y).  A short run spreads better; a token's angles and places, worth about four rows of
// arithmetic, are then computed for fewer rows.  The cost is that of the fullest SM's share.
struct RopeGrid {
  int run, x, y;
};
inline RopeGrid rope_grid(long long tokens, int heads, int slots, int blocks, int sms) {
  RopeGrid best{};
  long long least = 0;
  const long long per_run = (tokens + slots - 1) / slots;
  for (int run = 1;; run = 2 * run < heads ? 2 * run : heads) {
    const int y = (heads + run - 1) / run;
    if (y <= 65535) {                           // a grid's limit
      long long share = (per_run * y + sms - 1) / sms;
      if (share < blocks) share = blocks;       // an SM's blocks run side by side
      const long long cost = share * (run + 4);
      if (best.run == 0 || cost < least) {
        const long long most = ((long long)blocks * sms + y - 1) / y;
        best = {run, (int)(per_run < most ? per_run : most), y};
        least = cost;
      }
    }
    if (run >= heads) break;
  }
  return best;
}

}  // namespace mita
