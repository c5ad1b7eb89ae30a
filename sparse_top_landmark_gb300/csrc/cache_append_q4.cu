// New tokens' keys and values into a paged cache of 4-bit codes (layout and codes: paged_attn_q4.cu).
//
// For 32 values x of a row, a = max |x|:
//   s = a / 7 rounded to E5M3 (3 bits of mantissa, fp16's exponents; ties to even), at most 61440
//   n = round(min(max(x r, -7), 7)) + 8,   r = (1 / s) (1 - 2^-20) in fp32
// r is a little less than 1 / s, so that x halfway between two codes goes to the one nearer zero, whatever
// the rounding of 1 / s: for bf16 x, whose quotients come no nearer to a half than 1 / 4000 unless they are
// one, codes are those of exact arithmetic.  A block with an infinity or NaN has scale NaN.
//
// A lane has eight values (16 or 32 bytes of the row), four lanes a block; a thread block has one head's
// rows of neighbouring tokens, which mostly lie next to each other in the cache too.  Bound by HBM for
// prompts, by latency for a step.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace mita {
namespace {

constexpr int kAppendThreads = 256;

// The sizes' upper bits as an unsigned number: NaN is above infinity, infinity above all others.
__device__ __forceinline__ uint32_t size_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// t >= 0 to the nearest E5M3 value, ties to even
__device__ __forceinline__ float to_e5m3(float t) {
  if (t < 6.103515625e-5f) return rintf(t * 131072.f) * 7.62939453125e-6f;      // steps of 2^-17
  uint32_t b = __float_as_uint(t);
  b = (b + 0x7ffffu + (b >> 20 & 1u)) & 0xfff00000u;
  return fminf(__uint_as_float(b), 61440.f);
}

template <typename T, int U>
__global__ void __launch_bounds__(kAppendThreads)
cache_append_q4_kernel(const __grid_constant__ CacheAppendQ4Args<T> a, int row_lanes_log2) {
  griddep_wait();
  griddep_launch();
  const int lanes = 1 << row_lanes_log2, d = 8 * lanes, chunks = lanes / 4;
  const int rows = kAppendThreads >> row_lanes_log2;        // tokens of a block at a time
  const int hk = blockIdx.x % (2 * a.kv_heads), head = hk >> 1;
  const bool isv = hk & 1;
  const int g = threadIdx.x & (lanes - 1);
  const long long t0 = (long long)(blockIdx.x / (2 * a.kv_heads)) * (rows * U) +
                       (threadIdx.x >> row_lanes_log2);
  const T* x = (isv ? a.v : a.k) + head * (isv ? a.v_h : a.k_h) + g * 8;
  const long long x_t = isv ? a.v_t : a.k_t;
  float v[U][8];
  long long slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long t = t0 + u * rows;
    slot[u] = -1;
    if (t < a.tokens) {
      slot[u] = a.slots[t];
#pragma unroll
      for (int i = 0; i < 8; i += Vec<T>::N) Vec<T>::load(x + t * x_t + i, v[u] + i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
    }
  }
  uint8_t* cache = isv ? a.v_cache : a.k_cache;
  T* out = isv ? a.v_out : a.k_out;
  const long long o_t = isv ? a.vo_t : a.ko_t, o_h = isv ? a.vo_h : a.ko_h;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, size_bits(v[u][i]));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool odd = top >= 0x7f800000u;
    const float s = odd ? 0.f : to_e5m3(__fdiv_rn(__uint_as_float(top), 7.f));
    const float r = s > 0.f ? __fmul_rn(__frcp_rn(s), 1.f - 9.5367431640625e-7f) : 0.f;
    const float kept = odd ? __uint_as_float(0x7fc00000u) : s;
    // rounded by the addition to 1.5 * 2^23, whose last bits are then the code
    constexpr float kRound = 12582912.f;
    uint32_t word = 0;
    float back[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = fminf(fmaxf(__fmul_rn(odd ? 0.f : v[u][i], r), -7.f), 7.f);
      const float n = __fadd_rn(y, kRound);
      back[i] = __fsub_rn(n, kRound) * kept;
      word |= ((__float_as_uint(n) + 8u) & 15u) << (4 * i);
    }
    const long long t = t0 + u * rows;
    const bool bad = slot[u] < -1 || slot[u] >= a.places;
    if (bad && g == 0) flag_error(a.status, kDevErrBadIndex);
    if (slot[u] < 0 || bad) continue;
    const int row = (int)(slot[u] & ((1ll << a.page_log2) - 1));
    const long long page = slot[u] >> a.page_log2;
    uint8_t* base = cache + (((page * a.kv_heads + head) * (17 * chunks)) << a.page_log2);
    const int chunk = g >> 2;
    const int turn = chunks == 4 ? (row >> 1) & 3 : chunks == 2 ? (row >> 2) & 1 : 0;
    uint8_t* codes = base + (long long)row * (d / 2) + ((chunk ^ turn) * 16 + (g & 3) * 4);
    *reinterpret_cast<uint32_t*>(codes) = word;
    if ((g & 3) == 0) {
      const uint32_t h = __half_as_ushort(__float2half_rn(s));
      base[((long long)(d / 2) << a.page_log2) + (long long)row * chunks + chunk] =
          odd ? 255 : (uint8_t)(h >> 7);
    }
    if (out != nullptr) {
      T* to = out + t * o_t + head * o_h + g * 8;
#pragma unroll
      for (int i = 0; i < 8; i += Vec<T>::N) Vec<T>::store(to + i, back + i);
    }
  }
}

}  // namespace

template <typename T>
cudaError_t launch_cache_append_q4(CacheAppendQ4Args<T> a, int d, int sms, cudaStream_t st) {
  const int lanes_log2 = d == 128 ? 4 : d == 64 ? 3 : 2;
  const long long rows = kAppendThreads >> lanes_log2;
  auto blocks = [&](int u) { return (a.tokens + rows * u - 1) / (rows * u) * 2 * a.kv_heads; };
  const bool many = blocks(4) >= 4LL * sms;
  count_launch();
  return launch_pdl(many ? cache_append_q4_kernel<T, 4> : cache_append_q4_kernel<T, 1>,
                    dim3((unsigned)blocks(many ? 4 : 1)), dim3(kAppendThreads), 0, st, a,
                    lanes_log2);
}

template cudaError_t launch_cache_append_q4<float>(CacheAppendQ4Args<float>, int, int,
                                                   cudaStream_t);
template cudaError_t launch_cache_append_q4<bf16>(CacheAppendQ4Args<bf16>, int, int, cudaStream_t);

}  // namespace mita
