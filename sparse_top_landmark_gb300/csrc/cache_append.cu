// New tokens into a paged key-value cache: keys normalised and rotated on the way, values
// copied, and the new queries normalised and rotated by the same launch.
//
// Token j of a sequence with n new tokens and `len` tokens in all (the new ones included) has
// position len - n + j; that is also its angle's position.  Its key and value rows go to
// row position % page_size of page table[s][position / page_size].
//
// Bound by HBM for prompts (each row read once, written once) and by latency for the one-token
// step, where the lookup of sequence, length and page is a chain of dependent loads; the row
// loads do not depend on it and are issued first.  Lanes, slots and runs of heads are
// those of norm_rope.cu.
#include <algorithm>

#include "kernels.h"
#include "norm_rope.cuh"

namespace mita {
namespace {

constexpr int kAhead = 4;   // heads whose loads are issued together

// The sequence of token t: the last s with seq_start[s] <= t (empty sequences are passed over);
// -1 for a token before the first sequence or behind the last one.
__device__ __forceinline__ int sequence_of(const int32_t* seq_start, int S, int t) {
  if (t < __ldg(seq_start) || t >= __ldg(seq_start + S)) return -1;
  int lo = 0, hi = S;       // seq_start[lo] <= t < seq_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(seq_start + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads)
cache_append_kernel(const __grid_constant__ CacheAppendArgs<T> a) {
  using Bits = typename Raw4<T>::Bits;
  constexpr int L = D / 8;
  __shared__ unsigned long long table[D / 2];
  griddep_wait();
  rope_table(a.inv_freq, a.rot / 2, table);
  __syncthreads();
  const int g = threadIdx.x % L;
  int oa, ob;
  rope_groups(g, a.rot, a.interleaved, &oa, &ob);
  const bool turned = 8 * g < a.rot;
  unsigned long long turn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) turn[i] = turned ? table[4 * g + i] : 0;

  const int nq = (a.q_heads + a.run - 1) / a.run, nk = (a.kv_heads + a.run - 1) / a.run;
  const long long items = (long long)a.tokens * (nq + 2 * nk);
  const long long slots = (long long)gridDim.x * (kRopeThreads / L);
  long long item = (long long)blockIdx.x * (kRopeThreads / L) + threadIdx.x / L;
  const long long warp_first = item - (threadIdx.x % 32) / L;
  const PagedLayout& pg = a.paged;
  for (long long w = warp_first; w < items; w += slots, item += slots) {
    bool live = item < items;
    const long long it = live ? item : items - 1;
    const int chunk = (int)(it / a.tokens);
    const int t = (int)(it - (long long)chunk * a.tokens);
    const int kind = chunk < nq ? 0 : chunk < nq + nk ? 1 : 2;    // q, k, v
    const int h0 = (chunk - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * a.run;
    const int heads = kind == 0 ? a.q_heads : a.kv_heads;
    const T* x = kind == 0 ? a.q + t * a.q_t : kind == 1 ? a.k + t * a.k_t : a.v + t * a.v_t;
    const long long x_h = kind == 0 ? a.q_h : kind == 1 ? a.k_h : a.v_h;
    const float* weight = kind == 0 ? a.q_w : kind == 1 ? a.k_w : nullptr;

    // where the token belongs
    const int s = a.seq_start ? sequence_of(a.seq_start, pg.S, t) : t;
    int pos = 0;
    long long row = 0;
    if (s < 0) {
      live = false;
    } else {
      const int len = pg.lengths[s];
      const int first = a.seq_start ? a.seq_start[s] : t;
      const int end = a.seq_start ? a.seq_start[s + 1] : t + 1;
      pos = len - (end - t);
      if (len == 0) {
        live = false;                        // an idle slot
      } else {
        const int slot = pos >> pg.page_log2;
        int page = -1;
        if (pos >= 0 && len >= end - first && slot < pg.width)
          page = pg.table[(long long)s * pg.width + slot];
        if (page < 0 || page >= pg.num_pages) {
          if (live && g == 0) flag_error(a.status, kDevErrBadIndex);
          live = false;
        }
        row = (((long long)page * a.kv_heads) << pg.page_log2) +
              (pos & ((1 << pg.page_log2) - 1));
      }
    }
    const int h1 = live ? min(h0 + a.run, heads) : h0;
    float cs[4], sn[4];
    if (turned && kind < 2) rope_angles(turn, pos, cs, sn);
    float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
    if (weight) {
      Raw4<float>::unpack(*reinterpret_cast<const float4*>(weight + oa), wa);
      Raw4<float>::unpack(*reinterpret_cast<const float4*>(weight + ob), wb);
    }
    T* y = kind == 0 ? a.q_out + t * a.qo_t : (kind == 1 ? a.k_cache : a.v_cache) + row * D;
    const long long y_h = kind == 0 ? a.qo_h : (long long)D << pg.page_log2;
    for (int h = h0; h < h0 + a.run; h += kAhead) {
      Bits ra[kAhead] = {}, rb[kAhead] = {};
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (h + i < h1) {
          const T* r = x + (h + i) * x_h;
          ra[i] = *reinterpret_cast<const Bits*>(r + oa);
          rb[i] = *reinterpret_cast<const Bits*>(r + ob);
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i >= a.run) break;
        float va[4], vb[4], ss = 0.f;
        Raw4<T>::unpack(ra[i], va);
        Raw4<T>::unpack(rb[i], vb);
#pragma unroll
        for (int j = 0; j < 4; ++j) ss = fmaf(va[j], va[j], fmaf(vb[j], vb[j], ss));
        ss = row_sum<D>(ss);      // by all lanes, whatever their rows are
        if (kind < 2) {           // values go through as loaded
          if (weight) {
            const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              va[j] *= r * wa[j];
              vb[j] *= r * wb[j];
            }
          }
          if (turned) rope_turn(va, vb, cs, sn, a.interleaved, 1.f);
          ra[i] = Raw4<T>::pack(va);
          rb[i] = Raw4<T>::pack(vb);
        }
        if (h + i < h1) {
          T* o = y + (h + i) * y_h;
          *reinterpret_cast<Bits*>(o + oa) = ra[i];
          *reinterpret_cast<Bits*>(o + ob) = rb[i];
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t append_d(CacheAppendArgs<T>& a, int sms, cudaStream_t st) {
  constexpr int kSlots = kRopeThreads / (D / 8);
  const int rows = a.q_heads + 2 * a.kv_heads;
  a.run = 1;
  while (a.run < rows &&
         (long long)a.tokens * ((rows + 2 * a.run - 1) / (2 * a.run)) * (D / 8) >= 4096LL * sms)
    a.run *= 2;
  const long long items = (long long)a.tokens * ((a.q_heads + a.run - 1) / a.run +
                                                 2 * ((a.kv_heads + a.run - 1) / a.run));
  const int grid = (int)std::min<long long>((items + kSlots - 1) / kSlots, 8LL * sms);
  count_launch();
  return launch_pdl(cache_append_kernel<T, D>, dim3(grid), dim3(kRopeThreads), 0, st, a);
}

}  // namespace

template <typename T>
cudaError_t launch_cache_append(CacheAppendArgs<T> a, int d, int sms, cudaStream_t st) {
  switch (d) {
    case 16: return append_d<T, 16>(a, sms, st);
    case 32: return append_d<T, 32>(a, sms, st);
    case 64: return append_d<T, 64>(a, sms, st);
    case 128: return append_d<T, 128>(a, sms, st);
  }
  return cudaErrorInvalidValue;
}

template cudaError_t launch_cache_append<float>(CacheAppendArgs<float>, int, int, cudaStream_t);
template cudaError_t launch_cache_append<bf16>(CacheAppendArgs<bf16>, int, int, cudaStream_t);

}  // namespace mita
