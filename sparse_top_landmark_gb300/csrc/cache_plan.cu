// The pages of a serving step, dealt out on the device.
//
// Sequence s holds the pages of its lengths[s] tokens.  Where new_tokens[s] = -1 it is done: its pages go
// back onto the stack of free ones, in the order of s and of its table.  Otherwise its n = new_tokens[s]
// tokens need ceil((len + n) / page) - ceil(len / page) more pages; with P(s) the sum of what the sequences
// up to s need, s gets its n tokens if they fit its row of the table and the step's rows and either it
// needs no page or P(s) is at most the number of free ones.  Its pages are the stack's
// P(s - 1)-th from the top and the following.  Every row of the step's packed tokens then has a position
// in its sequence and a place in the cache.
//
// Two running sums over the sequences and some dozen bytes a row: bound by latency.  One cluster does it in
// one launch: each of its CTAs sums over all sequences (what they come to is in its shared memory then),
// they write nothing that another still reads before all have read it, and rows, and pages that come and
// go, are dealt to all warps.
//
// Measured: a step of 200 sequences in 6.9 us (three scans and four dependent loads behind an empty
// kernel's 2), 48 prompts of 88,821 rows and 5,565 pages in 11.8 (a thread a row, pages by threads: 22).
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace mita {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;         // of a cluster, at most

constexpr int kAhead = 4;            // of a lane's loads
constexpr int kNothing = -1, kDone = -2;
// What a sequence comes to.
struct PlanItem {
  int start;      // its first row
  int len;        // tokens before the step
  int first;      // pages taken by those before it; or kNothing, kDone
};

__device__ __forceinline__ int pages_of(int tokens, int page_log2) {
  return (int)(((long long)tokens + (1ll << page_log2) - 1) >> page_log2);
}

// Inclusive sums of N numbers each over the CTA's threads; all threads call it.
template <int N>
__device__ __forceinline__ void block_scan(long long (&x)[N], long long (*warps)[kPlanThreads / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](long long v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = scan(x[i]);
  __syncthreads();                   // the last scan's sums have been read
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 31) warps[i][warp] = x[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long w = warps[i][lane];
    x[i] += __shfl_sync(0xffffffffu, scan(w) - w, warp);
  }
}

__global__ void __launch_bounds__(kPlanThreads)
cache_plan_kernel(const __grid_constant__ CachePlanArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ PlanItem items[];
  __shared__ long long warps[2][kPlanThreads / 32], carry[2];
  __shared__ int last_taken;
  static_assert(kPlanThreads == 1024, "a warp's sum for each lane");
  griddep_wait();
  griddep_launch();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, ctas = gridDim.x;           // the grid is one cluster
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long room = (long long)a.width << a.page_log2;
  if (threadIdx.x == 0) last_taken = 0;

  struct Sequence {
    int fresh, len, held;
    bool done, fit;                  // fit: its tokens, by its own numbers
  };
  auto read = [&](int s) {
    Sequence q{};
    if (s >= a.S) return q;
    const int n = a.new_tokens[s], len = a.lengths[s];
    const bool ok = len >= 0 && len <= room;
    if (rank == 0 && (n < -1 || !ok)) flag_error(a.status, kDevErrBadIndex);
    q.done = n == -1;
    q.fresh = max(n, 0);
    q.len = len;
    q.held = pages_of((int)min((long long)max(len, 0), room), a.page_log2);
    q.fit = ok && n > 0 && (long long)len + n <= room;
    return q;
  };
  int free = *a.free_count;
  const Sequence mine = read(threadIdx.x);                 // of the first ones, mostly all
  if (free < 0 || free > a.num_pages) {
    if (rank == 0 && threadIdx.x == 0) flag_error(a.status, kDevErrBadIndex);
    free = min(max(free, 0), a.num_pages);
  }
  // first the rows, and the pages that come back: pushed onto the stack, from which they may be taken again
  long long pushed = 0, rows = 0;
  for (int s0 = 0; s0 < a.S; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    const Sequence q = s0 == 0 ? mine : read(s);
    const int back = q.done ? q.held : 0;
    long long sum[2] = {back, q.fresh};
    block_scan(sum, warps);
    if (s < a.S) items[s] = {(int)min(rows + sum[1] - q.fresh, (long long)a.tokens + 1), q.len, 0};
    const long long first = free + pushed + sum[0] - back;
    if (warp % ctas == rank) {       // a warp pushes its sequences' pages, one sequence after the other
      for (unsigned left = __ballot_sync(0xffffffffu, back > 0); left != 0; left &= left - 1) {
        const int src = __ffs(left) - 1, n = __shfl_sync(0xffffffffu, back, src);
        const long long to = __shfl_sync(0xffffffffu, first, src);
        const int32_t* row = a.page_table + (long long)(s0 + warp * 32 + src) * a.width;
        for (int i0 = lane; i0 < n; i0 += 32 * kAhead) {
          int page[kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) page[k] = i0 + 32 * k < n ? row[i0 + 32 * k] : 0;
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + 32 * k;
            if (i >= n) continue;
            if (to + i < a.num_pages) a.free_pages[to + i] = page[k];
            if (to + i >= a.num_pages || (unsigned)page[k] >= (unsigned)a.num_pages)
              flag_error(a.status, kDevErrBadIndex);
          }
        }
      }
    }
    if (threadIdx.x == kPlanThreads - 1) {
      carry[0] = pushed + sum[0];
      carry[1] = rows + sum[1];
    }
    __syncthreads();
    pushed = carry[0];
    rows = carry[1];
  }
  const int avail = (int)min(free + pushed, (long long)a.num_pages);
  const int last = (int)min(rows, (long long)a.tokens);     // rows of sequences
  // then who gets what
  long long wanted = 0;
  for (int s0 = 0; s0 < a.S; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    const Sequence q = s0 == 0 ? mine : read(s);
    const int start = s < a.S ? items[s].start : 0;
    const bool fits = q.fit && (long long)start + q.fresh <= a.tokens;
    const int need = fits ? pages_of(q.len + q.fresh, a.page_log2) - q.held : 0;
    long long through[1] = {need};
    block_scan(through, warps);
    through[0] += wanted;
    const bool granted = fits && (need == 0 || through[0] <= avail);
    if (s < a.S) {
      items[s].start = min(start, a.tokens);
      items[s].first = q.done ? kDone : !granted ? kNothing : need == 0 ? 0 : (int)(through[0] - need);
    }
    if (granted && need > 0) atomicMax(&last_taken, (int)through[0]);
    if (threadIdx.x == kPlanThreads - 1) carry[0] = through[0];
    __syncthreads();
    wanted = carry[0];
  }
  // what follows overwrites what was read above, and reads the pages that were pushed
  cluster.sync();

  auto fresh_of = [&](int s) { return (s + 1 < a.S ? items[s + 1].start : last) - items[s].start; };
  for (int s = rank * kPlanThreads + threadIdx.x; s <= a.S; s += ctas * kPlanThreads) {
    a.seq_start[s] = s < a.S ? items[s].start : last;
    if (s == a.S) break;
    const PlanItem q = items[s];
    const int got = q.first >= 0 ? fresh_of(s) : 0;
    a.granted[s] = got;
    a.new_lengths[s] = q.first == kDone ? 0 : q.len + got;
  }
  if (rank == 0 && threadIdx.x == 0) *a.new_free_count = avail - last_taken;
  // a warp a sequence, or several where there are few: the pages it gets
  const int all_warps = ctas * (kPlanThreads / 32), this_warp = rank * (kPlanThreads / 32) + warp;
  const int parts = max(1, all_warps / max(a.S, 1));
  for (int w = this_warp; w < a.S * parts; w += all_warps) {
    const int s = w / parts;
    const PlanItem q = items[s];
    if (q.first < 0) continue;
    const int held = pages_of(q.len, a.page_log2);
    const int need = pages_of(q.len + fresh_of(s), a.page_log2) - held;
    int32_t* to = a.page_table + (long long)s * a.width + held;
    for (int i = (w - s * parts) * 32 + lane; i < need; i += 32 * parts)
      to[i] = a.free_pages[avail - 1 - (q.first + i)];
  }
  // every row's position and place: a warp takes rows one behind the other, mostly of one sequence, and
  // kAhead of a lane's page numbers are on their way at once
  const int in_page = (1 << a.page_log2) - 1;
  const long long steps = ((long long)a.tokens + 31) / 32, each = (steps + all_warps - 1) / all_warps;
  const int t1 = (int)min((this_warp + 1) * each * 32, (long long)a.tokens);
  int lo = 0;                        // the row's sequence, the last one that begins at or before it
  for (long long t0 = this_warp * each * 32 + lane; t0 < t1; t0 += 32 * kAhead) {
    int pos[kAhead], page[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const long long t = t0 + 32 * k;
      pos[k] = 0;
      page[k] = kNothing;            // the row is nobody's
      if (t >= t1 || t >= last) continue;
      if (lo + 1 < a.S && items[lo + 1].start <= t) {
        int hi = a.S;                // items[lo].start <= t < items[hi].start
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (items[mid].start <= t) lo = mid; else hi = mid;
        }
      }
      const PlanItem q = items[lo];
      if (q.first < 0) continue;
      pos[k] = q.len + (int)(t - q.start);
      const int held = pages_of(q.len, a.page_log2), i = pos[k] >> a.page_log2;
      page[k] = i < held ? a.page_table[(long long)lo * a.width + i]
                         : a.free_pages[avail - 1 - (q.first + i - held)];
      if ((unsigned)page[k] >= (unsigned)a.num_pages) {
        flag_error(a.status, kDevErrBadIndex);
        page[k] = kNothing;
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const long long t = t0 + 32 * k;
      if (t >= t1) break;
      a.positions[t] = pos[k];
      a.slots[t] = page[k] < 0 ? -1 : ((long long)page[k] << a.page_log2) + (pos[k] & in_page);
    }
  }
}

}  // namespace

cudaError_t launch_cache_plan(const CachePlanArgs& a, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed{0};        // shared memory, once for each device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxPlanSequences * (int)sizeof(PlanItem));
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  int ctas = 1;
  while (ctas < kPlanCtas && (long long)ctas * kPlanThreads < std::max(a.tokens, a.S)) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = (size_t)std::max(a.S, 1) * sizeof(PlanItem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;     // a CTA alone is a cluster without being called one
  count_launch();
  return cudaLaunchKernelEx(&cfg, cache_plan_kernel, a);
}

}  // namespace mita
