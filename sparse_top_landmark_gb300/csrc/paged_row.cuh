// What the paged attention kernels have in common, whatever the cache holds: the row of tiles and its
// shares, the rule of the scores, the kernel around a warp's running softmax, and the join of cut
// segments.  paged_attn.cu says what it computes and how the work is dealt out.
#pragma once

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mita.h"

namespace mita {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum before the first key: below every finite score, and finite, so that
// differences with it need no special case (a score of -inf weighs nothing against it).
constexpr float kLowest = -FLT_MAX;
// Where scores are products, a maximum is taken from them in the same operation.  Where the maximum's own rounding
// may be a sixteenth or more, scores are rounded before, as it was: equal ones have equal weights.
constexpr float kFar = 1048576.f;
constexpr int kMaxPagedCtas = 255;     // CTAs of a call, and counters in its workspace
// Counters carry the number of the call that counts, above the count's kCountBits bits: whatever an
// earlier call left in them is below this one's zero.  (Were a caller to change lengths while they are
// read, CTAs would disagree on how many parts a segment has, and a counter that a segment's join puts
// back to zero would stay where it is, for every later call.)  Behind the counters one word gives the
// calls their numbers: each call adds kCallStep to it, all of its CTAs 1 but the first one, which adds the
// rest; so whichever comes first, each finds the same multiple of kCallStep there.  Nothing has to
// be waited for or put back at the end of a call (333 keys 9.4 us; with a word that counts the CTAs that are
// done, the last of which clears the counters, 10.4 us, and 9.6 where no fence orders the two).
constexpr int kCallNumber = kMaxPagedCtas;
constexpr int kCallStep = 256;
constexpr int kCountBits = 16;
static_assert(kCallStep > kMaxPagedCtas, "a call's CTAs stay within its step");

// A cut segment whose parts are to be joined: the row of its first query, the CTA that begins it,
// its parts (0: nothing to do) and its query rows.
struct Join {
  long long row;
  int c, n, rows, unused;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes, or zeros where `valid` is not set (src is then not read)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// An 8 x 8 matrix of 16-bit values, two of a row in a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// ---------------------------------------------------------------------------
// The row of tiles
// ---------------------------------------------------------------------------
// A sequence's seen keys [first, len), in tiles that start at multiples of `tile`.
struct Span {
  int first, len, base, tiles;
};
__device__ __forceinline__ Span span_of(const PagedLayout& pg, int window, int tile, int s) {
  Span r;
  const long long room = (long long)pg.width << pg.page_log2;
  r.len = (int)min((long long)max(pg.lengths[s], 0), room);
  r.first = window > 0 ? max(r.len - window, 0) : 0;
  r.base = r.first / tile * tile;
  r.tiles = (r.len - r.base + tile - 1) / tile;
  return r;
}

// A place in the row: tile `t` of segment (s, hr), hr = key head * row blocks + block; the segment
// begins at position `segment` of the row, and ends kSegmentCost positions after its last tile's.
struct Cursor {
  int s, hr, t;
  long long segment;
  Span span;
};

template <typename S>
__device__ __forceinline__ void advance(Cursor& c, const PagedLayout& pg, int window, int HR) {
  if (++c.t < c.span.tiles) return;
  c.t = 0;
  c.segment += c.span.tiles + S::kSegmentCost;
  if (++c.hr < HR) return;
  c.hr = 0;
  do {
    if (++c.s >= pg.S) {            // behind the last segment: behind every share
      c.segment = LLONG_MAX / 2;
      return;
    }
    c.span = span_of(pg, window, S::kTile, c.s);
  } while (c.span.tiles == 0);
}

__device__ __forceinline__ long long warp_incl_scan64(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// a / b, which are not negative: 64-bit division is some hundred instructions, and seldom needed.
__device__ __forceinline__ long long quotient(long long a, int b) {
  return a >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

__device__ __forceinline__ long long share_begin(long long row, int n, int c) {
  const long long q = quotient(row, n), r = row - q * n;
  return q * c + min((long long)c, r);
}
// The index of the CTA whose share of a row of that length has position x (one of the n, even where
// a caller changes lengths while they are read, and x lies anywhere).
__device__ __forceinline__ int share_of(long long x, long long row, int n) {
  const long long q = quotient(row, n), r = row - q * n;
  const long long large = r * (q + 1);       // the length of the r shares that are one longer
  if (q == 0) return (int)min(x, (long long)n - 1);
  return (int)min(x < large ? quotient(x, (int)q + 1) : r + quotient(x - large, (int)q),
                  (long long)n - 1);
}

// The length of the row, the place of this CTA's first tile, and the position where its share
// ends (a share may be empty, or hold ends of segments only: the first tile then lies behind).
// Each warp finds them for itself: a running sum over the sequences, of which those behind the
// first batch are summed ahead.  (worker, workers: this CTA and the grid, where a CTA is not several.)
struct Share {
  long long row, end;
  Cursor at;
};
template <typename S>
__device__ __forceinline__ Share my_share(const PagedLayout& pg, int window, int HR, int worker,
                                          int workers) {
  const int lane = threadIdx.x & 31;
  constexpr int kEach = 4, kBatch = 32 * kEach;     // sequences of a lane, and of a warp, at a time
  auto cost_of = [&](int tiles) {
    return tiles > 0 ? (long long)(tiles + S::kSegmentCost) * HR : 0;
  };
  const int each = pg.S <= 32 ? 1 : kEach;
  int tiles[kEach];
  auto load = [&](int s0) {                         // its lane's tiles, and what they cost
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int s = s0 + lane * each + i;
      tiles[i] = i < each && s < pg.S ? span_of(pg, window, S::kTile, s).tiles : 0;
      sum += tiles[i] > 0 ? tiles[i] + S::kSegmentCost : 0;
    }
    return (long long)sum * HR;
  };
  long long rest = 0;                               // behind the first batch: mostly there is none
  for (int s0 = kBatch; s0 < pg.S; s0 += kBatch) rest += load(s0);
  if (pg.S > kBatch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
  }
  long long cost = load(0), incl = warp_incl_scan64(cost);
  Share sh;
  sh.row = __shfl_sync(0xffffffffu, incl, 31) + rest;
  const long long x = share_begin(sh.row, workers, worker);
  sh.end = share_begin(sh.row, workers, worker + 1);
  sh.at.segment = sh.row;
  sh.at.t = 0;
  if (x >= sh.end) return sh;
  int s0 = 0;
  unsigned hit;
  while ((hit = __ballot_sync(0xffffffffu, x < incl)) == 0) {
    const long long run = __shfl_sync(0xffffffffu, incl, 31);
    s0 += kBatch;
    if (s0 >= pg.S) return sh;
    cost = load(s0);
    incl = run + warp_incl_scan64(cost);
  }
  const int src = __ffs(hit) - 1;
  long long start = __shfl_sync(0xffffffffu, incl - cost, src);
  int n = __shfl_sync(0xffffffffu, tiles[0], src);
  sh.at.s = s0 + src * each;
  if (each > 1) {
#pragma unroll
    for (int i = 1; i < kEach; ++i) {
      const int next = __shfl_sync(0xffffffffu, tiles[i], src);
      if (sh.at.s == s0 + src * kEach + i - 1 && x - start >= cost_of(n)) {
        start += cost_of(n);
        n = next;
        ++sh.at.s;
      }
    }
  }
  const int seg = (int)quotient(x - start, n + S::kSegmentCost);
  sh.at.segment = start + (long long)seg * (n + S::kSegmentCost);
  const int in = (int)(x - sh.at.segment);
  sh.at.hr = seg;
  sh.at.t = min(in, n - 1);
  sh.at.span = span_of(pg, window, S::kTile, sh.at.s);
  if (in >= n) advance<S>(sh.at, pg, window, HR);   // it begins behind a segment's last tile
  return sh;
}

// What a tile's scores need besides q and k.
struct ScoreRule {
  float scale2;          // scale * log2(e): the scores of the running softmax are in log2 units
  float cap, rcap;       // softcap (0: none), scale / softcap
  int last;              // len - 1
  bool plain;            // scores are just scale2 * dot, with scale2 >= 0
};
// Below kSeries a capped score is its uncapped one times tanh(x) / x, x = score / softcap, by that
// function's Taylor series in x^2 (up to x^10: what is left out is below 2^-24 there).  So small scores
// under a large cap keep fp32's relative accuracy, and caps up to the largest number, where x itself
// underflows, leave the score as it is.
constexpr float kSeries = 0.4f;
__device__ __forceinline__ float tanh_ratio(float xx) {
  float p = fmaf(xx, -8.8632355e-3f, 2.1869489e-2f);      // -1382/155925, 62/2835
  p = fmaf(xx, p, -5.3968254e-2f);                        // -17/315
  p = fmaf(xx, p, 1.3333333e-1f);                         // 2/15
  p = fmaf(xx, p, -3.3333333e-1f);                        // -1/3
  return fmaf(xx, p, 1.f);
}
// tanh from one exponential and one reciprocal, to 2^-22 absolute: for |x| >= kSeries that is 2^-20 of
// the value, in a quarter of tanhf's instructions.
__device__ __forceinline__ float tanh_fast(float x) {
  const float e = exp2_fast(fabsf(x) * (2.f * kLog2e));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return copysignf(fmaf(-2.f, r, 1.f), x);
}
// The score where the cap's series does (the last 2092 keys of 53 sequences in bf16, cap 30: 37.1 us
// where every score computes both forms, 34.1 where a warp's tile takes this one if all its scores allow it;
// in fp32, 192 of up to 3783, 85.3 and 82.0).
__device__ __forceinline__ float score_near_zero(const ScoreRule& r, float dot, float slope2, int key) {
  const float x = dot * r.rcap;
  return dot * r.scale2 * tanh_ratio(x * x) + slope2 * (float)(key - r.last);
}
template <bool FAST>
__device__ __forceinline__ float score_of(const ScoreRule& r, float dot, float slope2, int key) {
  float z = dot * r.scale2;
  if (r.cap > 0.f) {
    const float x = dot * r.rcap;
    z = fabsf(x) < kSeries ? z * tanh_ratio(x * x)
                           : r.cap * (FAST ? tanh_fast(x) : tanhf(x)) * kLog2e;
  }
  return z + slope2 * (float)(key - r.last);
}

// ln of a sum that is kept relative to 2^base; -inf of an empty one
__device__ __forceinline__ float lse_of(float base, float sum) {
  return sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
}
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }

// ---------------------------------------------------------------------------
// A warp's place in the row, for at most a key a lane: page numbers one tile ahead of the copies, copies
// kStages - 1 tiles ahead of the arithmetic.
// ---------------------------------------------------------------------------
template <typename S, typename Args>
struct RowLoader {
  using Mask = typename S::Mask;         // a bit a key
  static_assert(S::kKeys <= 32 && sizeof(Mask) == 4, "a lane's key");
  static constexpr Mask kAll = ~0u >> (32 - S::kKeys);
  Cursor at;
  long long end;           // of the share
  struct Rows {            // a warp's keys of a tile
    int page, key0, head;  // page: of this lane's key
    Mask mask;             // those to be seen
  };

  __device__ __forceinline__ Rows look_up(const Args& a, int HR) {
    int page = 0, key0 = 0, head = 0;
    Mask mask = 0;
    if (at.segment + at.t >= end) return {0, 0, 0, 0};
    const int warp = S::warp();
    key0 = at.span.base + at.t * S::kTile + warp * S::kKeys;
    const int lo = max(at.span.first - key0, 0), hi = min(at.span.len - key0, S::kKeys);
    if (lo < hi) {
      mask = (kAll << lo) & (kAll >> (S::kKeys - hi));
      head = a.row_blocks == 1 ? at.hr : at.hr / a.row_blocks;
      // lanes whose key is not to be seen read the first one's page
      const int mine = (threadIdx.x & 31) % S::kKeys;
      const int key = key0 + ((mask >> mine) & 1 ? mine : lo);
      page = a.paged.table[(long long)at.s * a.paged.width + (key >> a.paged.page_log2)];
    }
    advance<S>(at, a.paged, a.window, HR);
    return {page, key0, head, mask};
  }

  // the keys of `r` to be seen, without those on invalid pages (which are flagged)
  __device__ __forceinline__ static Mask valid_keys(const Args& a, const Rows& r) {
    Mask mask = r.mask;
    if (mask) {
      const bool bad = r.page < 0 || r.page >= a.paged.num_pages;
      const unsigned wrong = __ballot_sync(0xffffffffu, bad);
      if (wrong) {
        if ((threadIdx.x & 31) == 0) flag_error(a.status, kDevErrBadIndex);
        mask &= ~wrong;
      }
    }
    return mask;
  }
};

// Adds this CTA's part to the word that numbers the calls; returns what it was.
__device__ __forceinline__ unsigned long long count_call(unsigned long long* number) {
  const unsigned long long mine = blockIdx.x == 0 ? kCallStep - (gridDim.x - 1) : 1;
  unsigned long long old;
  asm volatile("atom.relaxed.gpu.global.add.u64 %0, [%1], %2;"
               : "=l"(old)
               : "l"(number), "l"(mine)
               : "memory");
  return old;
}
// Counts one up from `base`, this call's zero, after what this CTA's threads wrote before their last
// barrier, and before what they read after the next one; returns the count before.
__device__ __forceinline__ int count_up(unsigned long long* counter, unsigned long long base) {
  unsigned long long old;
  asm volatile("red.relaxed.gpu.global.max.u64 [%0], %1;" ::"l"(counter), "l"(base) : "memory");
  asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], 1;"
               : "=l"(old)
               : "l"(counter)
               : "memory");
  return (int)(old - base);
}

// The threads that work on one share.
struct WholeCta {
  __device__ __forceinline__ static int thread() { return threadIdx.x; }
  __device__ __forceinline__ static void sync() { __syncthreads(); }
};

// Joins the partials of a cut segment, all of them written: the beginning is CTA c's last part, the
// rest the first parts of CTAs c + 1 .. c + n - 1; out and lse: the segment's rows.  Called by all
// threads of a share (out of line: it should not cost the tile loop registers); `mem`: shared, of
// kThreads * 4 + kGroups * 2 floats.
// D / 4 threads take four columns of a row's parts, kAhead of them on their way at a time, with a
// running maximum; where there are fewer rows than such groups of threads, a row's parts are dealt
// to several groups, which are then joined in their order.
template <typename K, typename T>
__device__ __noinline__ void join_parts(const float* part_ml, const float* part_o, T* out,
                                        float* lse, int c, int n, int rows, float* mem) {
  using Team = typename K::Team;
  constexpr int D = K::kD, RT = K::kRT, kThreads = K::S::kTeamThreads;
  constexpr int kLanes = D / 4, kGroups = kThreads / kLanes, kAhead = RT == 16 ? 16 : 6;
  float4* sums = reinterpret_cast<float4*>(mem);               // [groups][D / 4]
  float2* totals = reinterpret_cast<float2*>(mem + kThreads * 4);   // [groups] (maximum, sum)
  static_assert((kThreads * 4 + kGroups * 2) * 4 <= K::S::kJoinBytes, "shared memory");
  const int thread = Team::thread(), group = thread / kLanes, col = thread % kLanes;
  for (int r0 = 0; r0 < rows; r0 += kGroups) {
    const int now = min(rows - r0, kGroups), share = kGroups / now;
    const int row = group / share, first = group - row * share;
    if (row < now) {
      float base = kLowest, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = first; i0 < n; i0 += share * kAhead) {
        float2 x[kAhead];
        float4 v[kAhead];
        float top = base;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + k * share;
          // written by other CTAs while this one ran: read past the L1
          const long long at = (long long)(i == 0 ? c * 2 + 1 : (c + i) * 2) * RT + r0 + row;
          x[k] = make_float2(kLowest, 0.f);
          v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < n) {
            x[k] = __ldcg(reinterpret_cast<const float2*>(part_ml) + at);
            v[k] = __ldcg(reinterpret_cast<const float4*>(part_o) + at * kLanes + col);
          }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) top = fmaxf(top, x[k].x);
        const float f = exp2_fast(base - top);
        base = top;
        sum *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float w = exp2_fast(x[k].x - top);
          sum = fmaf(w, x[k].y, sum);
          acc.x = fmaf(w, v[k].x, acc.x);
          acc.y = fmaf(w, v[k].y, acc.y);
          acc.z = fmaf(w, v[k].z, acc.z);
          acc.w = fmaf(w, v[k].w, acc.w);
        }
      }
      sums[thread] = acc;
      if (col == 0) totals[group] = make_float2(base, sum);
    }
    Team::sync();
    if (row < now && first == 0) {
      float base = kLowest, sum = 0.f;
      for (int g = 0; g < share; ++g) base = fmaxf(base, totals[group + g].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int g = 0; g < share; ++g) {
        const float2 x = totals[group + g];
        const float4 v = sums[thread + g * kLanes];
        const float w = exp2_fast(x.x - base);
        sum = fmaf(w, x.y, sum);
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      T* to = out + (long long)(r0 + row) * D + col * 4;
      to[0] = from_f<T>(acc.x * inv);
      to[1] = from_f<T>(acc.y * inv);
      to[2] = from_f<T>(acc.z * inv);
      to[3] = from_f<T>(acc.w * inv);
      if (lse && col == 0) lse[r0 + row] = lse_of(base, sum);
    }
    Team::sync();
  }
}

// Brings a segment's query rows near, ahead of State::start.
template <typename K>
__device__ __forceinline__ void prefetch_q(const typename K::Args& a, const Cursor& at) {
  using T = typename K::Type;
  constexpr int D = K::kD, RT = K::kRT;
  const int kv = a.row_blocks == 1 ? at.hr : at.hr / a.row_blocks;
  const int rb = at.hr - kv * a.row_blocks;
  constexpr int kLines = (D * (int)sizeof(T) + 127) / 128;      // of a row
  const int r = (int)threadIdx.x / kLines;
  if (r < min(RT, a.G - rb * RT)) {
    const char* p = reinterpret_cast<const char*>(
        a.q + at.s * a.q_s + (long long)(kv * a.G + rb * RT + r) * a.q_h);
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p + threadIdx.x % kLines * 128));
  }
}

// K: one kind of cache, element type, head dim and block of query rows (its Type, Args, S (the shape),
// State (a warp's running softmax) and Ld (its loader)).
template <typename K>
__global__ void __launch_bounds__(K::S::kThreads, 1)
paged_attn_kernel(const __grid_constant__ typename K::Args a) {
  using T = typename K::Type;
  using S = typename K::S;
  using State = typename K::State;
  using Ld = typename K::Ld;
  constexpr int D = K::kD, RT = K::kRT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int HR = a.Hkv * a.row_blocks, Hq = a.Hkv * a.G;
  uint8_t* ring = smem + warp * S::kRing;
  float2* ml = reinterpret_cast<float2*>(smem + S::kOffMl);
  using Mask = typename S::Mask;
  Mask* masks = reinterpret_cast<Mask*>(smem + S::kOffMask) + warp * S::kStages;
  // of the segment that another CTA begins, and of the one that another CTA ends
  Join* joins = reinterpret_cast<Join*>(smem + S::kOffJoins);

  griddep_wait();
  griddep_launch();
  unsigned long long call = 0;
  if (threadIdx.x == 0) call = count_call(a.counters + kCallNumber);     // looked at further below
  const Share share = my_share<S>(a.paged, a.window, HR, blockIdx.x, gridDim.x);
  Cursor at = share.at;
  if (threadIdx.x < 2) joins[threadIdx.x] = {};        // read behind the barriers of the share's end
  if (at.segment + at.t < share.end) {
    prefetch_q<K>(a, at);
    Ld ld;
    ld.at = at;
    ld.end = share.end;
    typename Ld::Rows rows_of[S::kStages];
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) rows_of[i] = ld.look_up(a, HR);   // their loads together
    // Not unrolled in bf16: a short call waits for its instructions (333 keys: 9.3 us unrolled, 9.1 us
    // so; fp32 loses as much in long ones).
#pragma unroll(S::kUnrollStart)
    for (int i = 0; i < S::kStages - 1; ++i) {
      ld.issue(a, rows_of[0], smem_addr(ring) + i * S::kStageBytes, masks + i);
#pragma unroll
      for (int j = 1; j < S::kStages; ++j) rows_of[j - 1] = rows_of[j];
    }
    typename Ld::Rows coming = rows_of[0];
    // thread 0's alone, kept where it takes no registers
    auto* const base = reinterpret_cast<unsigned long long*>(smem + S::kOffBase);
    if (threadIdx.x == 0) *base = call / kCallStep << kCountBits;
    State st;
    ScoreRule rule;
    rule.scale2 = a.scale * kLog2e;
    rule.cap = a.softcap;
    // finite, so that a score of zero stays one under the smallest caps too
    rule.rcap = a.softcap > 0.f ? fminf(fmaxf(a.scale / a.softcap, -FLT_MAX), FLT_MAX) : 0.f;
    rule.plain = a.softcap == 0.f && a.slopes == nullptr && a.scale >= 0.f;
    int slot = 0, next = S::kStages - 1;     // stages: of this tile, of the next one to issue
    int from = at.t, head = 0, rows = 0;
    bool begin = true;
    do {
      if (begin) {
        const int kv = a.row_blocks == 1 ? at.hr : at.hr / a.row_blocks;
        const int rb = at.hr - kv * a.row_blocks;
        head = kv * a.G + rb * RT;
        rows = min(RT, a.G - rb * RT);
        rule.last = at.span.len - 1;
        from = at.t;
        st.start(a, at.s, head, rows, rule);
        begin = false;
      }
      copy_wait<S::kStages - 2>();
      __syncwarp();
      ld.issue(a, coming, smem_addr(ring) + next * S::kStageBytes, masks + next);
      coming = ld.look_up(a, HR);
      const Mask mask = masks[slot];
      if (mask) {
        const uint32_t stage = smem_addr(ring) + slot * S::kStageBytes;
        st.tile(rule, stage, at.span.base + at.t * S::kTile + warp * S::kKeys, mask);
      }

      const bool ends = at.t + 1 == at.span.tiles;
      if (ends || at.segment + at.t + 1 == share.end) {
        // join the warps' parts: every row's sums are added by one warp
        Cursor then = at;
        advance<S>(then, a.paged, a.window, HR);
        if (ends && then.segment < share.end) prefetch_q<K>(a, then);
        st.put_ml(ml + warp * RT);
        __syncthreads();
        const bool whole = ends && from == 0;
        const int part = blockIdx.x * 2 + (from == 0 ? 1 : 0);
        auto top = [&](int r) {
          float t = ml[r].x;
#pragma unroll
          for (int w = 1; w < S::kWarps; ++w) t = fmaxf(t, ml[w * RT + r].x);
          return t;
        };
        // Every warp's sums go to the stage that it has just read: no copy goes there until its
        // next tile.
        float* const sums = reinterpret_cast<float*>(smem + slot * S::kStageBytes);
        st.put_o(sums + warp * (S::kRing / 4), rows, top);
        __syncthreads();
        for (int r = warp; r < rows; r += S::kWarps) {
          const float base = top(r);
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < S::kWarps; ++w) {
            const float2 x = ml[w * RT + r];
            sum = fmaf(x.y, exp2_fast(x.x - base), sum);
          }
          if (lane == 0) {
            if (!whole)
              reinterpret_cast<float2*>(a.part_ml)[(long long)part * RT + r] =
                  make_float2(base, sum);
            else if (a.lse)
              a.lse[(long long)at.s * Hq + head + r] = lse_of(base, sum);
          }
          const float inv = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
          T* out = a.out + ((long long)at.s * Hq + head + r) * D;
          float* part_o = a.part_o + ((long long)part * RT + r) * D;
#pragma unroll
          for (int c = lane; c < D; c += 32) {
            const float* from_w = sums + r * D + (c ^ State::spread(r));
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) x += from_w[w * (S::kRing / 4)];
            if (whole) out[c] = from_f<T>(x * inv);
            else part_o[c] = x;
          }
        }
        __syncthreads();
        if (!whole && threadIdx.x == 0) {
          // Whoever leaves a segment's last part joins them all, when its own share is done (the
          // others go on meanwhile): the count is asked for now, and looked at then.
          const int c0 = from == 0 ? (int)blockIdx.x : share_of(at.segment, share.row, gridDim.x);
          const int n = share_of(at.segment + at.span.tiles - 1, share.row, gridDim.x) - c0 + 1;
          const bool last = count_up(a.counters + c0, *base) == n - 1;
          joins[from == 0] = {(long long)at.s * Hq + head, c0, last ? n : 0, rows, 0};
        }
        begin = true;
      }
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
      next = next + 1 == S::kStages ? 0 : next + 1;
      advance<S>(at, a.paged, a.window, HR);
    } while (at.segment + at.t < share.end);
    copy_wait<0>();
    __syncthreads();
    for (int i = 0; i < 2; ++i) {
      const Join x = joins[i];
      if (x.n == 0) continue;
      join_parts<K>(a.part_ml, a.part_o, a.out + x.row * D,
                                        a.lse ? a.lse + x.row : nullptr, x.c, x.n, x.rows,
                                        reinterpret_cast<float*>(smem));
    }
  }
  // sequences without a key: zeros, and the logarithm of an empty sum
  for (int s = blockIdx.x; s < a.paged.S; s += gridDim.x) {
    const int len = a.paged.lengths[s];
    if (threadIdx.x == 0 && (len < 0 || len > (long long)a.paged.width << a.paged.page_log2))
      flag_error(a.status, kDevErrBadIndex);
    if (len > 0 && a.paged.width > 0) continue;
    for (int e = threadIdx.x; e < Hq * D; e += S::kThreads)
      a.out[(long long)s * Hq * D + e] = from_f<T>(0.f);
    if (a.lse)
      for (int e = threadIdx.x; e < Hq; e += S::kThreads) a.lse[(long long)s * Hq + e] = -INFINITY;
  }
}

// CTAs for this call: one on each SM, but no more than there can be tiles.  (K::S::kTeams: the shares
// of a CTA; K::kernel: the kernel.)
template <typename K>
int grid_of(int S, int width, int page_log2, int HR, int sms) {
  using Sh = typename K::S;
  const long long keys = (long long)width << page_log2;
  const long long tiles = (keys + Sh::kTile - 1) / Sh::kTile * HR * (long long)S;
  return (int)std::max<long long>(1, std::min<long long>({(long long)sms, tiles, kMaxPagedCtas}));
}

// The counters come first and in the same place for every shape: calls of different shapes can
// have one workspace.
struct Carve {
  size_t ml, o, total;
};
Carve carve(int ctas, int RT, int D) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  Carve c{};
  static_assert((kCallNumber + 1) * sizeof(long long) == MITA_PAGED_COUNTERS, "counters");
  c.ml = MITA_PAGED_COUNTERS;
  c.o = c.ml + up((size_t)ctas * 2 * RT * 2 * sizeof(float));
  c.total = c.o + up((size_t)ctas * 2 * RT * D * sizeof(float));
  return c;
}

template <typename K>
struct Run {
  static constexpr int D = K::kD, RT = K::kRT;
  static size_t bytes(int Hkv, int G, int S, int width, int page_log2, int sms) {
    const int HR = Hkv * ((G + RT - 1) / RT);
    return carve(grid_of<K>(S, width, page_log2, HR, sms) * K::S::kTeams, RT, D).total;
  }
  // the kernel's shared memory, allowed once for each device
  static cudaError_t allow_shared() {
    static std::atomic<unsigned long long> allowed{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (allowed.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(K::kernel(), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             K::S::kBytes);
    if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
  static cudaError_t launch(typename K::Args a, void* ws, int sms, cudaStream_t st) {
    using Sh = typename K::S;
    a.row_blocks = (a.G + RT - 1) / RT;
    const int grid = grid_of<K>(a.paged.S, a.paged.width, a.paged.page_log2,
                                       a.Hkv * a.row_blocks, sms);
    const Carve c = carve(grid * K::S::kTeams, RT, D);
    a.counters = static_cast<unsigned long long*>(ws);
    a.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + c.ml);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + c.o);
    cudaError_t e = allow_shared();
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_pdl(K::kernel(), dim3(grid), dim3(Sh::kThreads), Sh::kBytes, st,
                      a);
  }
};

}  // namespace
}  // namespace mita
