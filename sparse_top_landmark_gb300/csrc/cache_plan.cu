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
// one launch: each of its CTAs sums over all sequences (what they are is in its shared memory then),
// they write nothing that another still reads before all have read it, and the rows are dealt to all
// threads.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace mita {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;         // of a cluster, at most

// What a sequence comes to.
struct PlanItem {
  int start;      // its first row
  int len;        // tokens before the step
  int first;      // pages taken by those before it; -1: it gets nothing
};

__device__ __forceinline__ int pages_of(int tokens, int page_log2) {
  return (int)(((long long)tokens + (1ll << page_log2) - 1) >> page_log2);
}

// Inclusive sums over the CTA's threads; all threads call it.
__device__ __forceinline__ long long block_scan(long long x, long long* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](long long v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  x = scan(x);
  __syncthreads();                   // the last scan's sums have been read
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  const long long w = warps[lane];
  return x + __shfl_sync(0xffffffffu, scan(w) - w, warp);
}

__global__ void __launch_bounds__(kPlanThreads)
cache_plan_kernel(const __grid_constant__ CachePlanArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ PlanItem items[];
  __shared__ long long warps[kPlanThreads / 32], carry[2];
  __shared__ int last_taken;
  static_assert(kPlanThreads == 1024, "a warp's sum for each lane");
  griddep_wait();
  griddep_launch();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, ctas = gridDim.x;           // the grid is one cluster
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
  if (free < 0 || free > a.num_pages) {
    if (rank == 0 && threadIdx.x == 0) flag_error(a.status, kDevErrBadIndex);
    free = min(max(free, 0), a.num_pages);
  }
  // first the pages that come back: pushed onto the stack by CTA 0, from which they may be taken again
  long long pushed = 0;
  for (int s0 = 0; s0 < a.S; s0 += kPlanThreads) {
    const Sequence q = read(s0 + threadIdx.x);
    const long long mine = q.done ? q.held : 0, back = block_scan(mine, warps);
    if (rank == 0) {
      const int32_t* row = a.page_table + (long long)(s0 + threadIdx.x) * a.width;
      long long at = free + pushed + back - mine;
      for (int i = 0; i < mine; ++i, ++at) {
        if (at < a.num_pages) a.free_pages[at] = row[i];
        else flag_error(a.status, kDevErrBadIndex);
      }
    }
    if (threadIdx.x == kPlanThreads - 1) carry[0] = pushed + back;
    __syncthreads();
    pushed = carry[0];
  }
  const int avail = (int)min(free + pushed, (long long)a.num_pages);
  // then who gets what
  long long rows = 0, wanted = 0;
  for (int s0 = 0; s0 < a.S; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    const Sequence q = read(s);
    const long long end = rows + block_scan(q.fresh, warps);
    const bool fits = q.fit && end <= a.tokens;
    const int need = fits ? pages_of(q.len + q.fresh, a.page_log2) - q.held : 0;
    const long long through = wanted + block_scan(need, warps);
    const bool granted = fits && (need == 0 || through <= avail);
    if (s < a.S)
      items[s] = {(int)min(end - q.fresh, (long long)a.tokens), q.len,
                  !granted ? -1 : need == 0 ? 0 : (int)(through - need)};
    if (granted && need > 0) atomicMax(&last_taken, (int)through);
    if (threadIdx.x == kPlanThreads - 1) {
      carry[0] = end;
      carry[1] = through;
    }
    __syncthreads();
    rows = carry[0];
    wanted = carry[1];
  }
  // what follows overwrites what was read above, and reads the pages that CTA 0 has pushed
  cluster.sync();

  const int last = (int)min(rows, (long long)a.tokens);     // rows of sequences
  auto fresh_of = [&](int s) { return (s + 1 < a.S ? items[s + 1].start : last) - items[s].start; };
  for (int s = rank * kPlanThreads + threadIdx.x; s <= a.S; s += ctas * kPlanThreads) {
    a.seq_start[s] = s < a.S ? items[s].start : last;
    if (s == a.S) break;
    const PlanItem q = items[s];
    const int got = q.first >= 0 ? fresh_of(s) : 0;
    a.granted[s] = got;
    a.new_lengths[s] = a.new_tokens[s] == -1 ? 0 : q.len + got;
  }
  if (rank == 0 && threadIdx.x == 0) *a.new_free_count = avail - last_taken;
  // a warp a sequence: the pages it gets
  const int warp = (rank * kPlanThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  for (int s = warp; s < a.S; s += ctas * (kPlanThreads / 32)) {
    const PlanItem q = items[s];
    if (q.first < 0) continue;
    const int held = pages_of(q.len, a.page_log2);
    const int need = pages_of(q.len + fresh_of(s), a.page_log2) - held;
    int32_t* to = a.page_table + (long long)s * a.width + held;
    for (int i = lane; i < need; i += 32) to[i] = a.free_pages[avail - 1 - (q.first + i)];
  }
  // every row's position and place
  const int in_page = (1 << a.page_log2) - 1;
  for (long long t = rank * kPlanThreads + threadIdx.x; t < a.tokens; t += ctas * kPlanThreads) {
    int pos = 0;
    long long slot = -1;
    if (t < last) {
      int lo = 0, hi = a.S;          // items[lo].start <= t < items[hi].start
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (items[mid].start <= t) lo = mid; else hi = mid;
      }
      const PlanItem q = items[lo];
      if (q.first >= 0) {
        pos = q.len + (int)(t - q.start);
        const int held = pages_of(q.len, a.page_log2), i = pos >> a.page_log2;
        const int page = i < held ? a.page_table[(long long)lo * a.width + i]
                                  : a.free_pages[avail - 1 - (q.first + i - held)];
        if (page >= 0 && page < a.num_pages)
          slot = ((long long)page << a.page_log2) + (pos & in_page);
        else
          flag_error(a.status, kDevErrBadIndex);
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
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
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, cache_plan_kernel, a);
}

}  // namespace mita
