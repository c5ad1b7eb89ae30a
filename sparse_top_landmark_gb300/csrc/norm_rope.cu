// Per-head RMS norm and rotary position rotation of q and k, and the gradient.
//
//   forward   u = w * x * r,  r = 1 / sqrt(mean(x^2) + eps);   y = R(p) u
//   gradient  g = R(p)^T dy;  dw = sum over rows of g * x * r;
//             dx = r * (w * g) - x * r^3 * mean(w * g * x)
//
// R(p) turns pair i of the first `rot` values of a row by the angle p * inv_freq[i].  Everything
// between the loads and the one rounding of each result is fp32.
//
// Bound by HBM: a row is read once and written once (the gradient reads two and writes one),
// and a value costs some ten instructions.  A slot of D / 8 lanes takes one token's heads
// one after the other, so that a token's angles are computed once for all of them, and fetches
// several heads ahead of working on them (kAhead), which keeps enough bytes in flight.
#include "norm_rope.cuh"

#include <algorithm>

#include "kernels.h"

namespace mita {
namespace {

constexpr int kAhead = 4;      // heads whose loads are issued together

// One block of rows: `chunks` runs of up to `run` heads for each token, tokens fastest, so that
// neighbouring slots work on neighbouring tokens of the same heads.
template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads)
norm_rope_kernel(const __grid_constant__ NormRopeArgs<T> a) {
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

  const long long tokens = (long long)a.B * a.N;
  const int nq = (a.part[0].heads + a.run - 1) / a.run;
  const int nk = (a.part[1].heads + a.run - 1) / a.run;
  const long long items = tokens * (nq + nk);
  const long long slots = (long long)gridDim.x * (kRopeThreads / L);
  long long item = (long long)blockIdx.x * (kRopeThreads / L) + threadIdx.x / L;
  // all lanes of a warp stay in the loop together (row_sum shuffles across the warp)
  const long long warp_first = item - (threadIdx.x % 32) / L;
  for (long long w = warp_first; w < items; w += slots, item += slots) {
    const bool live = item < items;
    const long long it = live ? item : items - 1;
    const int chunk = (int)(it / tokens);
    const long long t = it - chunk * tokens;
    const int bt = (int)(t / a.N), n = (int)(t - (long long)bt * a.N);
    const int isk = chunk >= nq;
    const NormRopePart<T>& p = a.part[isk];
    const int h0 = (isk ? chunk - nq : chunk) * a.run;
    const int h1 = live ? min(h0 + a.run, p.heads) : h0;
    float cs[4], sn[4];
    if (turned) rope_angles(turn, a.positions ? a.positions[bt * a.pos_b + n] : n, cs, sn);
    float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
    if (p.w) {
      Raw4<float>::unpack(*reinterpret_cast<const float4*>(p.w + oa), wa);
      Raw4<float>::unpack(*reinterpret_cast<const float4*>(p.w + ob), wb);
    }
    const T* x = p.x + bt * p.x_b + n * p.x_n;
    T* y = p.y + bt * p.y_b + n * p.y_n;
    for (int h = h0; h < h0 + a.run; h += kAhead) {
      typename Raw4<T>::Bits ra[kAhead] = {}, rb[kAhead] = {};
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (h + i < h1) {
          const T* r = x + (h + i) * p.x_h;
          ra[i] = *reinterpret_cast<const typename Raw4<T>::Bits*>(r + oa);
          rb[i] = *reinterpret_cast<const typename Raw4<T>::Bits*>(r + ob);
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i >= a.run) break;
        float va[4], vb[4];
        Raw4<T>::unpack(ra[i], va);
        Raw4<T>::unpack(rb[i], vb);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) ss = fmaf(va[j], va[j], fmaf(vb[j], vb[j], ss));
        ss = row_sum<D>(ss);
        if (p.w) {
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            va[j] *= r * wa[j];
            vb[j] *= r * wb[j];
          }
        }
        if (turned) rope_turn(va, vb, cs, sn, a.interleaved, 1.f);
        if (h + i < h1) {
          T* o = y + (h + i) * p.y_h;
          *reinterpret_cast<typename Raw4<T>::Bits*>(o + oa) = Raw4<T>::pack(va);
          *reinterpret_cast<typename Raw4<T>::Bits*>(o + ob) = Raw4<T>::pack(vb);
        }
      }
    }
  }
}

// The gradient.  A block works on q rows alone (the first a.qblocks blocks) or on k rows alone;
// each lane sums its eight columns of dw over its rows, the block joins them in a fixed order
// and writes one partial row of D; norm_rope_dw_kernel adds the partial rows, again in a fixed
// order: no atomics, so the same inputs give the same bits.
template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads)
norm_rope_backward_kernel(const __grid_constant__ NormRopeBackwardArgs<T> a) {
  constexpr int L = D / 8;
  constexpr int kSlots = kRopeThreads / L;
  __shared__ unsigned long long table[D / 2];
  __shared__ float red[kRopeThreads * 8];
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

  const int isk = (int)blockIdx.x >= a.qblocks;
  const NormRopeBackwardPart<T>& p = a.part[isk];
  const int blk = isk ? blockIdx.x - a.qblocks : blockIdx.x;
  const int blocks = isk ? gridDim.x - a.qblocks : a.qblocks;
  const long long tokens = (long long)a.B * a.N;
  const long long items = tokens * ((p.heads + a.run - 1) / a.run);
  float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
  if (p.w) {
    Raw4<float>::unpack(*reinterpret_cast<const float4*>(p.w + oa), wa);
    Raw4<float>::unpack(*reinterpret_cast<const float4*>(p.w + ob), wb);
  }
  float dwa[4] = {}, dwb[4] = {};
  long long item = (long long)blk * kSlots + threadIdx.x / L;
  const long long warp_first = item - (threadIdx.x % 32) / L;
  for (long long w = warp_first; w < items; w += (long long)blocks * kSlots,
                 item += (long long)blocks * kSlots) {
    const bool live = item < items;
    const long long it = live ? item : items - 1;
    const int chunk = (int)(it / tokens);
    const long long t = it - chunk * tokens;
    const int bt = (int)(t / a.N), n = (int)(t - (long long)bt * a.N);
    const int h0 = chunk * a.run;
    const int h1 = live ? min(h0 + a.run, p.heads) : h0;
    float cs[4], sn[4];
    if (turned) rope_angles(turn, a.positions ? a.positions[bt * a.pos_b + n] : n, cs, sn);
    const T* x = p.x + bt * p.x_b + n * p.x_n;
    const T* dy = p.dy + bt * p.dy_b + n * p.dy_n;
    T* dx = p.dx + bt * p.dx_b + n * p.dx_n;
    constexpr int kPair = 2;
    for (int h = h0; h < h0 + a.run; h += kPair) {
      typename Raw4<T>::Bits xa[kPair] = {}, xb[kPair] = {}, ya[kPair] = {}, yb[kPair] = {};
#pragma unroll
      for (int i = 0; i < kPair; ++i)
        if (h + i < h1) {
          const T* r = dy + (h + i) * p.dy_h;
          ya[i] = *reinterpret_cast<const typename Raw4<T>::Bits*>(r + oa);
          yb[i] = *reinterpret_cast<const typename Raw4<T>::Bits*>(r + ob);
          if (p.w) {
            const T* s = x + (h + i) * p.x_h;
            xa[i] = *reinterpret_cast<const typename Raw4<T>::Bits*>(s + oa);
            xb[i] = *reinterpret_cast<const typename Raw4<T>::Bits*>(s + ob);
          }
        }
#pragma unroll
      for (int i = 0; i < kPair; ++i) {
        if (i >= a.run) break;
        float ga[4], gb[4], va[4], vb[4];
        Raw4<T>::unpack(ya[i], ga);
        Raw4<T>::unpack(yb[i], gb);
        Raw4<T>::unpack(xa[i], va);
        Raw4<T>::unpack(xb[i], vb);
        if (turned) rope_turn(ga, gb, cs, sn, a.interleaved, -1.f);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ss = fmaf(va[j], va[j], fmaf(vb[j], vb[j], ss));
          dot = fmaf(wa[j] * ga[j], va[j], fmaf(wb[j] * gb[j], vb[j], dot));
        }
        ss = row_sum<D>(ss);
        dot = row_sum<D>(dot);
        if (p.w) {
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          const float c = r * r * r * dot * (1.f / D);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (h + i < h1) {
              dwa[j] = fmaf(ga[j], va[j] * r, dwa[j]);
              dwb[j] = fmaf(gb[j], vb[j] * r, dwb[j]);
            }
            ga[j] = r * (wa[j] * ga[j]) - va[j] * c;
            gb[j] = r * (wb[j] * gb[j]) - vb[j] * c;
          }
        }
        if (h + i < h1) {
          T* o = dx + (h + i) * p.dx_h;
          *reinterpret_cast<typename Raw4<T>::Bits*>(o + oa) = Raw4<T>::pack(ga);
          *reinterpret_cast<typename Raw4<T>::Bits*>(o + ob) = Raw4<T>::pack(gb);
        }
      }
    }
  }
  if (p.partial == nullptr) return;
  // [slot][column]: slot s of the block wrote columns oa .. oa + 3 and ob .. ob + 3
  float* mine = red + (threadIdx.x / L) * D;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    mine[oa + j] = dwa[j];
    mine[ob + j] = dwb[j];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int i = 0; i < kSlots; ++i) s += red[i * D + threadIdx.x];
    p.partial[(long long)blk * D + threadIdx.x] = s;
  }
}

// dw[c] = the sum of `blocks` partial rows; blockIdx.x: 0 = q, 1 = k; blockIdx.y: 16 columns.
__global__ void __launch_bounds__(256)
norm_rope_dw_kernel(const float* pq, const float* pk, int qblocks, int kblocks, int D, float* dwq,
                    float* dwk) {
  __shared__ float red[16][17];
  griddep_wait();
  const float* p = blockIdx.x ? pk : pq;
  float* dw = blockIdx.x ? dwk : dwq;
  const int blocks = blockIdx.x ? kblocks : qblocks;
  if (p == nullptr) return;
  const int c = threadIdx.x % 16, r = threadIdx.x / 16;
  const int col = blockIdx.y * 16 + c;
  float s = 0.f;
#pragma unroll 4
  for (int i = r; i < blocks; i += 16) s += p[(long long)i * D + col];
  red[r][c] = s;
  __syncthreads();
  if (r == 0) {
    for (int i = 1; i < 16; ++i) s += red[i][c];
    dw[col] = s;
  }
}

// Heads a slot takes one after the other: as many as still leave every SM its threads twice
// over (a token's angles are then computed once for them), at least one.
int heads_per_run(long long tokens, int heads, int lanes, int sms) {
  int run = 1;
  while (run < heads && tokens * ((heads + 2 * run - 1) / (2 * run)) * lanes >= 4096LL * sms)
    run *= 2;
  return run;
}

template <typename T, int D>
cudaError_t forward_d(NormRopeArgs<T>& a, int sms, cudaStream_t st) {
  constexpr int kSlots = kRopeThreads / (D / 8);
  const long long tokens = (long long)a.B * a.N;
  a.run = heads_per_run(tokens, a.part[0].heads + a.part[1].heads, D / 8, sms);
  const long long items = tokens * ((a.part[0].heads + a.run - 1) / a.run +
                                    (a.part[1].heads + a.run - 1) / a.run);
  const int grid = (int)std::min<long long>((items + kSlots - 1) / kSlots, 8LL * sms);
  count_launch();
  return launch_pdl(norm_rope_kernel<T, D>, dim3(grid), dim3(kRopeThreads), 0, st, a);
}

template <typename T, int D>
cudaError_t backward_d(NormRopeBackwardArgs<T>& a, float* partial, int sms, float* dwq, float* dwk,
                       cudaStream_t st) {
  constexpr int kSlots = kRopeThreads / (D / 8);
  const long long tokens = (long long)a.B * a.N;
  a.run = heads_per_run(tokens, a.part[0].heads + a.part[1].heads, D / 8, sms);
  const long long iq = tokens * ((a.part[0].heads + a.run - 1) / a.run);
  const long long ik = tokens * ((a.part[1].heads + a.run - 1) / a.run);
  const long long bq = (iq + kSlots - 1) / kSlots, bk = (ik + kSlots - 1) / kSlots;
  const int cap = norm_rope_backward_blocks(sms);
  int qb = (int)bq, kb = (int)bk;
  if (bq + bk > cap) {
    // the blocks in proportion to the two parts' rows, one at least for each part that has any
    kb = ik == 0 ? 0 : (int)std::max<long long>(1, cap * ik / (iq + ik));
    qb = cap - kb;
  }
  a.qblocks = qb;
  a.part[0].partial = dwq ? partial : nullptr;
  a.part[1].partial = dwk ? partial + (size_t)qb * D : nullptr;
  count_launch();
  cudaError_t e = launch_pdl(norm_rope_backward_kernel<T, D>, dim3(qb + kb), dim3(kRopeThreads), 0,
                             st, a);
  if (e != cudaSuccess || (!dwq && !dwk)) return e;
  count_launch();
  return launch_pdl(norm_rope_dw_kernel, dim3(2, D / 16), dim3(256), 0, st,
                    (const float*)a.part[0].partial, (const float*)a.part[1].partial, qb, kb, D,
                    dwq, dwk);
}

}  // namespace

int norm_rope_backward_blocks(int sms) { return 4 * sms; }

template <typename T>
cudaError_t launch_norm_rope(NormRopeArgs<T> a, int d, int sms, cudaStream_t st) {
  switch (d) {
    case 16: return forward_d<T, 16>(a, sms, st);
    case 32: return forward_d<T, 32>(a, sms, st);
    case 64: return forward_d<T, 64>(a, sms, st);
    case 128: return forward_d<T, 128>(a, sms, st);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_norm_rope_backward(NormRopeBackwardArgs<T> a, int d, float* partial, int sms,
                                      float* dwq, float* dwk, cudaStream_t st) {
  switch (d) {
    case 16: return backward_d<T, 16>(a, partial, sms, dwq, dwk, st);
    case 32: return backward_d<T, 32>(a, partial, sms, dwq, dwk, st);
    case 64: return backward_d<T, 64>(a, partial, sms, dwq, dwk, st);
    case 128: return backward_d<T, 128>(a, partial, sms, dwq, dwk, st);
  }
  return cudaErrorInvalidValue;
}

template cudaError_t launch_norm_rope<float>(NormRopeArgs<float>, int, int, cudaStream_t);
template cudaError_t launch_norm_rope<bf16>(NormRopeArgs<bf16>, int, int, cudaStream_t);
template cudaError_t launch_norm_rope_backward<float>(NormRopeBackwardArgs<float>, int, float*, int,
                                                      float*, float*, cudaStream_t);
template cudaError_t launch_norm_rope_backward<bf16>(NormRopeBackwardArgs<bf16>, int, float*, int,
                                                     float*, float*, cudaStream_t);

}  // namespace mita
