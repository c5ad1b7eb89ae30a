// Device helpers shared by the kernels that normalise and rotate heads (norm_rope.cu: whole
// sequences and their gradient; cache_append.cu: new tokens on their way into the cache).
//
// A head row of D values is worked on by D / 8 lanes.  Lane g holds eight values as two groups
// of four, chosen so that the rotation never leaves the lane: with the half-split pairing
// (i, i + rot/2) the groups start at 4g and rot/2 + 4g, with the neighbouring pairing
// (2i, 2i + 1) at 8g and 8g + 4; the unrotated tail [rot, D) is taken as 8g, 8g + 4 either way.
// Hence rot % 8 == 0.  Either way the lane's pairs are the rotation's frequencies 4g .. 4g + 3.
#pragma once

#include "common.cuh"

namespace mita {

// Threads of a block in these kernels.
constexpr int kRopeThreads = 256;

// Four values of a row, as loaded (8 bytes of bf16, 16 of fp32) and as fp32.
template <typename T> struct Raw4;
template <> struct Raw4<float> {
  using Bits = float4;
  __device__ __forceinline__ static void unpack(const Bits& b, float* o) {
    o[0] = b.x; o[1] = b.y; o[2] = b.z; o[3] = b.w;
  }
  __device__ __forceinline__ static Bits pack(const float* o) {
    return make_float4(o[0], o[1], o[2], o[3]);
  }
};
template <> struct Raw4<bf16> {
  using Bits = uint2;
  __device__ __forceinline__ static void unpack(const Bits& b, float* o) {
    o[0] = __uint_as_float(b.x << 16);
    o[1] = __uint_as_float(b.x & 0xffff0000u);
    o[2] = __uint_as_float(b.y << 16);
    o[3] = __uint_as_float(b.y & 0xffff0000u);
  }
  // the one rounding of a result: to nearest, ties to even
  __device__ __forceinline__ static Bits pack(const float* o) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o[2], o[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                      *reinterpret_cast<const uint32_t*>(&hi));
  }
};

// Where lane g of a row finds its two groups of four.
__device__ __forceinline__ void rope_groups(int g, int rot, int interleaved, int* a, int* b) {
  const bool split = !interleaved && 8 * g < rot;
  *a = split ? 4 * g : 8 * g;
  *b = split ? rot / 2 + 4 * g : 8 * g + 4;
}

// The angle of frequency i at position p is p * inv_freq[i] radians.  In fp32 it would lose
// its fraction of a turn at far positions (an ulp of 10^6 is 1/16 radian), and fp64 arithmetic
// per token is slow on this part.  So each block turns the frequencies once into unsigned
// 64-bit fractions of a turn; p * fraction mod 2^64 is then the exact product modulo one turn
// (the frequency's own rounding, 2^-53 of it, is all that is lost), for any 32-bit p, negative
// ones included.  The angle's sign and its top 32 bits go to sincospif.
__device__ __forceinline__ void rope_table(const double* inv_freq, int half,
                                           unsigned long long* turn) {
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    double f = inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
    f -= rint(f);                                      // whole turns do nothing; |f| <= 1/2
    turn[i] = (unsigned long long)__double2ll_rn(f * 18446744073709551616.0);   // saturates
  }
}

// cos and sin of lane g's four pairs at position p.
__device__ __forceinline__ void rope_angles(const unsigned long long* turn, int p, float* cs,
                                            float* sn) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long t = (unsigned long long)(long long)p * turn[i];
    sincospif((float)(int)(t >> 32) * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2^-31 half turns
  }
}

// Turns the lane's eight values a, b by its four angles (sign = -1: back).
__device__ __forceinline__ void rope_turn(float* a, float* b, const float* cs, const float* sn,
                                          int interleaved, float sign) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* v = i < 2 ? a + 2 * i : b + 2 * (i - 2);
      const float x = v[0], y = v[1], s = sign * sn[i];
      v[0] = x * cs[i] - y * s;
      v[1] = y * cs[i] + x * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[i], y = b[i], s = sign * sn[i];
      a[i] = x * cs[i] - y * s;
      b[i] = y * cs[i] + x * s;
    }
  }
}

// Sum over the D / 8 lanes of a row (all 32 lanes of the warp call it).
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace mita
