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

// Block (x, y): the y-th run of rows (q heads, k heads, v heads) of the tokens x, x + gridDim.x,
// ..., a slot a token.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
cache_append_kernel(const __grid_constant__ CacheAppendArgs<T> a) {
  constexpr int L = D / 8, kSlots = kRopeThreads / L, K = kRopeAhead<T>;
  __shared__ unsigned long long table[D / 2];
  griddep_wait();
  griddep_launch();
  rope_table(a.inv_freq, a.rot / 2, table);
  __syncthreads();
  const RopeLane lane(threadIdx.x % L, a.rot, INTER);
  const unsigned long long* turn = table + 4 * (threadIdx.x % L);

  const int hq = a.q_heads, hkv = a.kv_heads;
  const int h0 = blockIdx.y * a.run, h1 = min(h0 + a.run, hq + 2 * hkv);
  const PagedLayout& pg = a.paged;
  const int in_page = (1 << pg.page_log2) - 1;
  const unsigned tokens = a.tokens, stride = gridDim.x * kSlots;
  unsigned t = blockIdx.x * kSlots + threadIdx.x / L;
  for (unsigned first = t - (threadIdx.x % 32) / L; first < tokens; first += stride, t += stride) {
    // where the token belongs
    bool live = t < tokens;
    const int s = !live ? -1 : a.seq_start ? sequence_of(a.seq_start, pg.S, t) : (int)t;
    int pos = 0;
    long long row = 0;
    live = s >= 0;
    if (live) {
      const int len = pg.lengths[s];
      const int begin = a.seq_start ? a.seq_start[s] : s;
      const int end = a.seq_start ? a.seq_start[s + 1] : s + 1;
      pos = len - (end - (int)t);
      live = len != 0;                       // else an idle slot
      if (live) {
        const int slot = pos >> pg.page_log2;
        int page = -1;
        if (len >= end - begin && (len - 1) >> pg.page_log2 < pg.width)
          page = pg.table[(long long)s * pg.width + slot];
        live = page >= 0 && page < pg.num_pages;
        if (!live && threadIdx.x % L == 0) flag_error(a.status, kDevErrBadIndex);
        row = (((long long)page * a.kv_heads) << pg.page_log2) + (pos & in_page);
      }
    }
    V2 cs[2], sn[2];
    if (lane.turned && h0 < hq + hkv) rope_angles(turn, pos, cs, sn);
    for (int kind = 0; kind < 3; ++kind) {     // q, k, v
      const int before = kind == 0 ? 0 : kind == 1 ? hq : hq + hkv;
      int h = max(h0 - before, 0);
      const int end = min(h1 - before, kind == 0 ? hq : hkv);
      if (h >= end) continue;
      const long long x_h = kind == 0 ? a.q_h : kind == 1 ? a.k_h : a.v_h;
      const long long y_h = kind == 0 ? a.qo_h : (long long)D << pg.page_log2;
      const T* x = kind == 0 ? a.q + t * a.q_t : kind == 1 ? a.k + t * a.k_t : a.v + t * a.v_t;
      T* y = kind == 0 ? a.q_out + t * a.qo_t : (kind == 1 ? a.k_cache : a.v_cache) + row * D;
      const float* w = kind == 0 ? a.q_w : kind == 1 ? a.k_w : nullptr;
      RopeCoef<INTER> coef;
      coef.set(lane.turned && kind < 2, cs, sn, w ? weights8(w, lane) : ones8());
      x += h * x_h;
      y += h * y_h;
      for (; h < end; h += K, x += K * x_h, y += K * y_h)
        rope_rows<T, D, INTER>(lane, coef, x, x_h, y, y_h, end - h, w != nullptr, live, a.eps);
    }
  }
}

template <typename T, int D>
cudaError_t append_d(CacheAppendArgs<T>& a, int sms, cudaStream_t st) {
  const RopeGrid g = rope_grid(a.tokens, a.q_heads + 2 * a.kv_heads, kRopeThreads / (D / 8),
                               kRopeBlocks, sms);
  a.run = g.run;
  count_launch();
  return launch_pdl(a.interleaved ? cache_append_kernel<T, D, true>
                                  : cache_append_kernel<T, D, false>,
                    dim3(g.x, g.y), dim3(kRopeThreads), 0, st, a);
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
