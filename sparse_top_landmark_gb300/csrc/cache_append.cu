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
//
// Measured (bf16, 32 query and 8 key heads of 128): 24 prompts of 55,068 tokens in 212 us, 6.4
// TB/s; one token in 3.3 us, a step of 200 sequences in 4.6 us.
#include <algorithm>

#include "kernels.h"
#include "norm_rope.cuh"
#include "token_place.h"

namespace mita {
namespace {

// The sequence of token t: the last s with seq_start[s] <= t (empty sequences are passed over);
// -1 for a token before the first sequence or behind the last one.  (Whatever the array holds,
// seq_start[s] <= t < seq_start[s + 1] on return.)
__device__ __forceinline__ int sequence_of(const int32_t* seq_start, int S, int t) {
  if (t < seq_start[0] || t >= seq_start[S]) return -1;
  int lo = 0, hi = S;       // seq_start[lo] <= t < seq_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Block (x, y): the y-th run of rows (q heads, k heads, v heads) of the tokens x, x + gridDim.x,
// ..., a slot a token.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
cache_append_kernel(const __grid_constant__ CacheAppendArgs<T> a) {
  constexpr int L = D / 8, kSlots = kRopeThreads / L;
  __shared__ unsigned long long table[D / 2];
  __shared__ __align__(16) char rows_ahead[RowRing<T>::kBytes];
  griddep_wait();
  griddep_launch();
  RowRing<T> ring(rows_ahead);
  const RopeLane lane(threadIdx.x % L, D, a.rot, INTER, table);

  // this block's rows of a token: those of q, of k, of v, in pairs
  const int heads[3] = {a.q_heads, a.kv_heads, a.kv_heads};
  const int h0 = blockIdx.y * a.run, h1 = min(h0 + a.run, a.q_heads + 2 * a.kv_heads);
  int first[3], rows[3];
#pragma unroll
  for (int k = 0, before = 0; k < 3; before += heads[k++]) {
    first[k] = max(h0 - before, 0);
    rows[k] = max(min(h1 - before, heads[k]) - first[k], 0);
  }
  const unsigned tokens = a.tokens, stride = gridDim.x * kSlots;
  const unsigned t0 = blockIdx.x * kSlots + threadIdx.x / L;
  const unsigned in_warp = (threadIdx.x % 32) / L;

  // The next pair to fetch.  Rows are fetched ahead whether or not their token turns out to have a
  // place: where it has one is a chain of loads of its own.
  unsigned ahead = t0;
  int kind, left;
  const T* x;
  long long x_h;
  auto enter = [&](int k) {        // the first kind from k on that this block has rows of
    if (k == 0 && rows[0] == 0) k = 1;
    if (k == 1 && rows[1] == 0) k = 2;
    kind = k;
    left = k == 0 ? rows[0] : k == 1 ? rows[1] : rows[2];
    x_h = k == 0 ? a.q_h : k == 1 ? a.k_h : a.v_h;
    x = (k == 0 ? a.q + ahead * a.q_t : k == 1 ? a.k + ahead * a.k_t : a.v + ahead * a.v_t) +
        (k == 0 ? first[0] : k == 1 ? first[1] : first[2]) * x_h;
  };
  enter(0);
  auto fetch = [&] {
    ring.template fetch<0>(x, lane.a, lane.b, ahead < tokens);
    ring.template fetch<1>(x + x_h, lane.a, lane.b, ahead < tokens && left > 1);
    ring.next();
    x += 2 * x_h;
    left -= 2;
    if (left <= 0) {
      const bool same = (kind == 0 && rows[1] + rows[2] > 0) || (kind == 1 && rows[2] > 0);
      if (!same) ahead += stride;
      enter(same ? kind + 1 : 0);
    }
  };
#pragma unroll
  for (int i = 0; i < RowRing<T>::kPairs; ++i) fetch();
  rope_table<D>(a.inv_freq, a.rot / 2, table);
  __syncthreads();

  const PagedLayout& pg = a.paged;
  const int in_page = (1 << pg.page_log2) - 1;
  for (unsigned t = t0; t - in_warp < tokens; t += stride) {
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
      live = len != 0;                       // else an idle slot
      if (live) {
        pos = token_position(len, begin, end, (int)t);
        int page = -1;
        if (pos >= 0 && fits_table(len, pg.width, pg.page_log2))
          page = pg.table[(long long)s * pg.width + (pos >> pg.page_log2)];
        live = page >= 0 && page < pg.num_pages;
        if (!live && threadIdx.x % L == 0) flag_error(a.status, kDevErrBadIndex);
        row = (((long long)page * a.kv_heads) << pg.page_log2) + (pos & in_page);
      }
    }
    V2 cs[2], sn[2];
    if (rows[0] + rows[1] > 0) rope_angles(lane.turn, pos, cs, sn);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (rows[k] == 0) continue;
      const long long y_h = k == 0 ? a.qo_h : (long long)D << pg.page_log2;
      T* y = (k == 0 ? a.q_out + t * a.qo_t : (k == 1 ? a.k_cache : a.v_cache) + row * D) +
             first[k] * y_h;
      const float* w = k == 0 ? a.q_w : k == 1 ? a.k_w : nullptr;
      RopeCoef<INTER> coef;
      if (k < 2) coef.set(cs, sn, w ? weights8(w, lane) : ones8());
      for (int i = 0; i < rows[k]; i += 2, y += 2 * y_h) {
        ring.wait();
        rope_pair<T, D, INTER>(lane, coef, ring.template get<0>(), ring.template get<1>(), y, y_h,
                               rows[k] - i, w != nullptr, lane.turned && k < 2, live, a.eps);
        fetch();
      }
    }
  }
  ring.drain();
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
