// New tokens' keys and values into a paged cache of 4-bit codes (layout and codes: paged_attn_q4.cu).
//
// For 32 values x of a row, a = max |x|:
//   s = a / 7 rounded to E5M3 (3 bits of mantissa, fp16's exponents; ties to even), at most 61440
//   n = round(min(max(x r, -7), 7)) + 8,   r = (1 / s) (1 - 2^-20) in fp32
// r is a little less than 1 / s, so that x halfway between two codes goes to the one nearer zero, whatever
// the rounding of 1 / s: for bf16 x, whose quotients come no nearer to a half than 1 / 4000 unless they are
// one, codes are those of exact arithmetic.  A block with an infinity or NaN has scale NaN.
//
// A lane has 16 values of a row, two lanes a block of 32; a thread block has one head's rows of neighbouring
// tokens, which mostly lie next to each other in the cache too, and a lane has several tokens' values on
// their way at once.  Bound by HBM for prompts, where it is the instructions that come next: arithmetic
// is on pairs of fp32 values, rounding is an addition, four codes are put together as one number in three
// products, and what only blocks near the ends of the scales need stands behind a vote.  By latency for a
// step.
//
// Measured (8 heads of 128, the rounded values returned too): prompts of 55,068 tokens in 79 us, 6.5 TB/s
// (bf16), and 141 us, 6.8 TB/s (fp32); a step of 200 sequences in 1.9 us.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace mita {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kLaneValues = 16;

using V2 = unsigned long long;   // two fp32 values
__device__ __forceinline__ V2 mul2(V2 a, V2 b) {
  V2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ V2 add2(V2 a, V2 b) {
  V2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ V2 both(float x) { return f2pack(x, x); }

// A lane's values of a row as they lie.
template <typename T> struct Lane16;
template <> struct Lane16<bf16> {
  uint4 w[2];
  __device__ __forceinline__ void load(const bf16* p) {
    w[0] = reinterpret_cast<const uint4*>(p)[0];
    w[1] = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4& v = w[i / 4];
    return i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w;
  }
  // the largest size's bits, as of an fp32 value; as unsigned numbers NaN are above infinity, infinity
  // above all others
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = word(0) & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, word(i) & 0x7fff7fffu);
    return max(m & 0xffff0000u, m << 16);
  }
  __device__ __forceinline__ V2 pair(int i) const {
    return f2pack(__uint_as_float(word(i) << 16), __uint_as_float(word(i) & 0xffff0000u));
  }
  __device__ __forceinline__ static void store(bf16* p, const V2 (&x)[8]) {
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      f2unpack(x[i], lo, hi);
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      o[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
};
template <> struct Lane16<float> {
  float4 w[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ V2 pair(int i) const {
    const float4& v = w[i / 2];
    return i % 2 ? f2pack(v.z, v.w) : f2pack(v.x, v.y);
  }
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) m = max(m, __float_as_uint(x[k]) & 0x7fffffffu);
    }
    return m;
  }
  __device__ __forceinline__ static void store(float* p, const V2 (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 v;
      f2unpack(x[2 * i], v.x, v.y);
      f2unpack(x[2 * i + 1], v.z, v.w);
      reinterpret_cast<float4*>(p)[i] = v;
    }
  }
};

// t >= 0 to the nearest E5M3 value, ties to even
__device__ __forceinline__ float to_e5m3(float t) {
  if (t < 6.103515625e-5f) return rintf(t * 131072.f) * 7.62939453125e-6f;      // steps of 2^-17
  uint32_t b = __float_as_uint(t);
  b = (b + 0x7ffffu + (b >> 20 & 1u)) & 0xfff00000u;
  return fminf(__uint_as_float(b), 61440.f);
}

// Four codes less 8 as one number's digits, and 8 for each: the last 16 bits of the result.
__device__ __forceinline__ uint32_t four_codes(V2 a, V2 b) {
  float n[4];
  f2unpack(a, n[0], n[1]);
  f2unpack(b, n[2], n[3]);
  const float x = fmaf(fmaf(fmaf(n[3], 16.f, n[2]), 16.f, n[1]), 16.f, n[0]);
  return __float_as_uint(x + (8388608.f + 34952.f));
}

// U tokens to a lane.
template <typename T, int U>
__global__ void __launch_bounds__(kAppendThreads)
cache_append_q4_kernel(const __grid_constant__ CacheAppendQ4Args<T> a, int row_lanes_log2) {
  griddep_wait();
  griddep_launch();
  const int lanes = 1 << row_lanes_log2, chunks = lanes / 2;
  const int rows = kAppendThreads >> row_lanes_log2;        // tokens of a block at a time
  const unsigned group = blockIdx.x / (2 * (unsigned)a.kv_heads);
  const int hk = blockIdx.x - group * (2 * (unsigned)a.kv_heads), head = hk >> 1;
  const bool isv = hk & 1;
  const int g = threadIdx.x & (lanes - 1);
  const long long t0 = (long long)group * (rows * U) + (threadIdx.x >> row_lanes_log2);
  const long long x_t = isv ? a.v_t : a.k_t;
  const T* x = (isv ? a.v : a.k) + head * (isv ? a.v_h : a.k_h) + g * kLaneValues + t0 * x_t;
  Lane16<T> v[U];
  long long slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    slot[u] = -1;
    v[u] = {};
    if (t0 + u * rows < a.tokens) {
      slot[u] = a.slots[t0 + u * rows];
      v[u].load(x + u * rows * x_t);
    }
  }
  uint8_t* const cache = isv ? a.v_cache : a.k_cache;
  T* const out = isv ? a.v_out : a.k_out;
  const long long o_t = isv ? a.vo_t : a.ko_t, o_h = isv ? a.vo_h : a.ko_h;
  const int chunk = g >> 1;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t top = v[u].largest();
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const bool odd = top >= 0x7f800000u;
    const float t = __fdiv_rn(__uint_as_float(top), 7.f);
    const float s = odd ? 0.f : to_e5m3(t);
    const float r = s > 0.f ? __fmul_rn(__frcp_rn(s), 1.f - 9.5367431640625e-7f) : 0.f;
    V2 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = mul2(v[u].pair(i), both(r));
    // only scales that were not rounded by a sixteenth at most leave a quotient beyond 7.5
    if (__any_sync(0xffffffffu, t < 6.103515625e-5f || !(t <= 61440.f))) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float lo, hi;
        f2unpack(y[i], lo, hi);
        y[i] = odd ? 0 : f2pack(fminf(fmaxf(lo, -7.f), 7.f), fminf(fmaxf(hi, -7.f), 7.f));
      }
    }
    constexpr float kRound = 12582912.f;         // 1.5 * 2^23: adding it rounds
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = add2(add2(y[i], both(kRound)), both(-kRound));
    const uint32_t w0 = __byte_perm(four_codes(y[0], y[1]), four_codes(y[2], y[3]), 0x5410);
    const uint32_t w1 = __byte_perm(four_codes(y[4], y[5]), four_codes(y[6], y[7]), 0x5410);
    const bool bad = slot[u] < -1 || slot[u] >= a.places;
    if (bad && g == 0) flag_error(a.status, kDevErrBadIndex);
    if (slot[u] < 0 || bad) continue;
    const int row = (int)slot[u] & ((1 << a.page_log2) - 1);
    uint8_t* const base =
        cache + ((((slot[u] >> a.page_log2) * a.kv_heads + head) * (17 * chunks)) << a.page_log2);
    const int turn = chunks == 4 ? (row >> 1) & 3 : chunks == 2 ? (row >> 2) & 1 : 0;
    *reinterpret_cast<uint2*>(base + (long long)row * (16 * chunks) + ((chunk ^ turn) * 16 + (g & 1) * 8)) =
        make_uint2(w0, w1);
    if ((g & 1) == 0) {
      const uint32_t h = __half_as_ushort(__float2half_rn(s));
      base[((long long)(16 * chunks) << a.page_log2) + (long long)row * chunks + chunk] =
          odd ? 255 : (uint8_t)(h >> 7);
    }
    if (out != nullptr) {
      const V2 kept = both(odd ? __uint_as_float(0x7fc00000u) : s);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = mul2(y[i], kept);
      Lane16<T>::store(out + (t0 + u * rows) * o_t + head * o_h + g * kLaneValues, y);
    }
  }
}

}  // namespace

template <typename T>
cudaError_t launch_cache_append_q4(CacheAppendQ4Args<T> a, int d, int sms, cudaStream_t st) {
  const int lanes_log2 = d == 128 ? 3 : d == 64 ? 2 : 1;
  const long long rows = kAppendThreads >> lanes_log2;
  auto blocks = [&](int u) { return (a.tokens + rows * u - 1) / (rows * u) * 2 * a.kv_heads; };
  // 64 bytes of a lane's values on their way (bf16, prompts of 55k tokens of 8 heads of 128: one token a
  // lane 88 us, two 79, four 79; fp32: one 141, two 143), where that leaves blocks for every SM
  constexpr int kMany = 64 / (kLaneValues * (int)sizeof(T));
  const bool many = blocks(kMany) >= 4LL * sms;
  count_launch();
  return launch_pdl(many ? cache_append_q4_kernel<T, kMany> : cache_append_q4_kernel<T, 1>,
                    dim3((unsigned)blocks(many ? kMany : 1)), dim3(kAppendThreads), 0, st, a,
                    lanes_log2);
}

template cudaError_t launch_cache_append_q4<float>(CacheAppendQ4Args<float>, int, int,
                                                   cudaStream_t);
template cudaError_t launch_cache_append_q4<bf16>(CacheAppendQ4Args<bf16>, int, int, cudaStream_t);

}  // namespace mita
