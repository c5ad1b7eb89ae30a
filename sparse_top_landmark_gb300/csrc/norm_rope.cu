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
// one after the other, so that a token's angles are computed once for all of them.
//
// Measured (bf16, inputs of a fused projection): 2 x 8191 tokens of 40 heads of 128 in 57 us,
// 5.9 TB/s; 1,048,576 tokens of 4 heads of 64 in 193 us, 5.6 TB/s (a third of each token's values
// lies between and is skipped; copying alone takes 175 us); the gradient of 2 x 4096 tokens of 40
// heads of 128 in 49 us, 5.1 TB/s, where it is the instructions that bound it.
#include "norm_rope.cuh"

#include <algorithm>

#include "kernels.h"

namespace mita {
namespace {

// Block (x, y): the y-th run of heads (q's, then k's) of the tokens x, x + gridDim.x, ..., a slot
// a token; neighbouring slots have neighbouring tokens.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
norm_rope_kernel(const __grid_constant__ NormRopeArgs<T> a) {
  constexpr int L = D / 8, kSlots = kRopeThreads / L;
  __shared__ unsigned long long table[D / 2];
  __shared__ __align__(16) char rows_ahead[RowRing<T>::kBytes];
  griddep_wait();
  griddep_launch();
  RowRing<T> ring(rows_ahead);
  const RopeLane lane(threadIdx.x % L, D, a.rot, INTER, table);

  // this block's rows of a token: those of q, then those of k, in pairs
  const int hq = a.part[0].heads, h0 = blockIdx.y * a.run;
  const int h1 = min(h0 + a.run, hq + a.part[1].heads);
  const int first[2] = {h0, max(h0 - hq, 0)};
  const int rows[2] = {max(min(h1, hq) - h0, 0), max(h1 - hq - first[1], 0)};
  const unsigned tokens = (unsigned)a.B * a.N, stride = gridDim.x * kSlots;
  const unsigned t0 = blockIdx.x * kSlots + threadIdx.x / L;
  // all lanes of a warp stay in the loops together, as long as its first lane has a token
  const unsigned in_warp = (threadIdx.x % 32) / L;

  const NormRopePart<T>&q = a.part[0], &k = a.part[1];
  const long long fq = first[0], fk = first[1];

  // the next pair to fetch: token (its rows of q and k), part, place and rows left of the part
  TokenWalk ahead(t0, a.N);
  const T *xq, *xk, *x;
  long long x_h;
  int part, left;
  auto arrive = [&] {
    xq = q.x + ahead.b * q.x_b + ahead.n * q.x_n + fq * q.x_h;
    xk = k.x + ahead.b * k.x_b + ahead.n * k.x_n + fk * k.x_h;
  };
  auto enter = [&](bool isk) {
    part = isk;
    left = isk ? rows[1] : rows[0];
    x_h = isk ? k.x_h : q.x_h;
    x = isk ? xk : xq;
  };
  arrive();
  enter(rows[0] == 0);
  auto fetch = [&] {
    ring.template fetch<0>(x, lane.a, lane.b, ahead.t < tokens);
    ring.template fetch<1>(x + x_h, lane.a, lane.b, ahead.t < tokens && left > 1);
    ring.next();
    x += 2 * x_h;
    left -= 2;
    if (left <= 0) {
      const bool same = part == 0 && rows[1] > 0;
      if (!same) {
        if (ahead.step(stride)) {
          xq += stride * q.x_n;
          xk += stride * k.x_n;
        } else {
          arrive();
        }
      }
      enter(same || rows[0] == 0);
    }
  };
#pragma unroll
  for (int i = 0; i < RowRing<T>::kPairs; ++i) fetch();
  rope_table<D>(a.inv_freq, a.rot / 2, table);
  __syncthreads();
  TokenWalk at(t0, a.N);
  T* y[2];
  auto leave = [&] {
    y[0] = q.y + at.b * q.y_b + at.n * q.y_n + fq * q.y_h;
    y[1] = k.y + at.b * k.y_b + at.n * k.y_n + fk * k.y_h;
  };
  leave();
  while (at.t - in_warp < tokens) {
    const bool live = at.t < tokens;
    V2 cs[2], sn[2];
    rope_angles(lane.turn, a.positions && live ? a.positions[at.b * a.pos_b + at.n] : at.n, cs, sn);
#pragma unroll
    for (int isk = 0; isk < 2; ++isk) {
      const NormRopePart<T>& p = a.part[isk];
      if (rows[isk] == 0) continue;
      RopeCoef<INTER> coef;
      coef.set(cs, sn, p.w ? weights8(p.w, lane) : ones8());
      T* to = y[isk];
      for (int i = rows[isk]; i > 0; i -= 2, to += 2 * p.y_h) {
        ring.wait();
        rope_pair<T, D, INTER>(lane, coef, ring.template get<0>(), ring.template get<1>(), to,
                               p.y_h, i, p.w != nullptr, lane.turned, live, a.eps);
        fetch();
      }
    }
    if (at.step(stride)) {
      y[0] += stride * q.y_n;
      y[1] += stride * k.y_n;
    } else {
      leave();
    }
  }
  ring.drain();
}

// The sum of x, added in pairs: a chain would add up roundings that grow with the sum so far (weight
// gradients of 4096 tokens, 4 heads of 32 in fp32, root mean square against fp64: 2.0e-7 with a block's
// slots in a chain, 1.3e-7 so; torch's fp32 sum of the same terms 0.9e-7).
template <int N>
__device__ __forceinline__ float sum_in_pairs(float (&x)[N]) {
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] += x[i + n];
  return x[0];
}

// The gradient.  A block works on q rows alone (blockIdx.y < a.qruns) or on k rows alone; each
// lane sums its eight columns of dw over its rows, the block joins them in a fixed order and
// writes one partial row of D; norm_rope_dw_kernel adds the partial rows, again in a fixed
// order: no atomics, so the same inputs give the same bits.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
norm_rope_backward_kernel(const __grid_constant__ NormRopeBackwardArgs<T> a) {
  constexpr int L = D / 8, kSlots = kRopeThreads / L;
  __shared__ unsigned long long table[D / 2];
  __shared__ __align__(16) union {
    char rows[RowRing<T>::kBytes];           // a row of dy and its row of x are a pair
    float red[kRopeThreads * 8];
  } mem;
  griddep_wait();
  griddep_launch();
  RowRing<T> ring(mem.rows);
  const RopeLane lane(threadIdx.x % L, D, a.rot, INTER, table);

  const int isk = (int)blockIdx.y >= a.qruns;
  const NormRopeBackwardPart<T>& p = a.part[isk];
  const int run = isk ? blockIdx.y - a.qruns : blockIdx.y;
  const int h0 = run * a.run, rows = min(a.run, p.heads - h0);
  const bool normed = p.w != nullptr;
  const unsigned tokens = (unsigned)a.B * a.N, stride = gridDim.x * kSlots;
  const unsigned t0 = blockIdx.x * kSlots + threadIdx.x / L;
  const unsigned in_warp = (threadIdx.x % 32) / L;

  TokenWalk ahead(t0, a.N);
  int left = rows;
  const T *x0, *dy0, *x, *dy;      // of the token, and of its next row
  auto arrive = [&] {
    x0 = p.x + ahead.b * p.x_b + ahead.n * p.x_n + h0 * p.x_h;
    dy0 = p.dy + ahead.b * p.dy_b + ahead.n * p.dy_n + h0 * p.dy_h;
  };
  arrive();
  x = x0;
  dy = dy0;
  auto fetch = [&] {
    ring.template fetch<0>(dy, lane.a, lane.b, ahead.t < tokens);
    ring.template fetch<1>(x, lane.a, lane.b, ahead.t < tokens && normed);
    ring.next();
    x += p.x_h;
    dy += p.dy_h;
    if (--left == 0) {
      if (ahead.step(stride)) {
        x0 += stride * p.x_n;
        dy0 += stride * p.dy_n;
      } else {
        arrive();
      }
      left = rows;
      x = x0;
      dy = dy0;
    }
  };
#pragma unroll
  for (int i = 0; i < RowRing<T>::kPairs; ++i) fetch();
  rope_table<D>(a.inv_freq, a.rot / 2, table);
  __syncthreads();
  const V8 w = normed ? weights8(p.w, lane) : ones8();
  V8 dw = {};
  for (TokenWalk at(t0, a.N); at.t - in_warp < tokens; at.step(stride)) {
    const bool live = at.t < tokens;
    V2 cs[2], sn[2];
    rope_angles(lane.turn, a.positions && live ? a.positions[at.b * a.pos_b + at.n] : at.n, cs, sn);
    RopeCoef<INTER> back;
    back.set(cs, sn, ones8(), true);
    T* dx = p.dx + at.b * p.dx_b + at.n * p.dx_n + h0 * p.dx_h;
    for (int i = 0; i < rows; ++i, dx += p.dx_h) {
      ring.wait();
      Raw8<T> rg = ring.template get<0>();
      if (normed) {
        // with u = x r: dw += g u, dx = r (w g - u mean(w g u)); a slot without a token has zeros
        const V8 g = back.of(rg.unpack());
        V8 u = ring.template get<1>().unpack(), wg;
        V2 s2 = mul2(u.v[0], u.v[0]);
        wg.v[0] = mul2(w.v[0], g.v[0]);
        V2 d2 = mul2(wg.v[0], u.v[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) {
          s2 = fma2(u.v[j], u.v[j], s2);
          wg.v[j] = mul2(w.v[j], g.v[j]);
          d2 = fma2(wg.v[j], u.v[j], d2);
        }
        float ss = sum2(s2), dot = sum2(d2);
        slot_sum2<D>(ss, dot, [](float s) { return s; });
        const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        const float m = live ? -r * dot * (1.f / D) : 0.f;
        const float ru = live ? r : 0.f;
        const V2 rr = f2pack(ru, ru), mm = f2pack(m, m);
        V8 d;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u.v[j] = mul2(u.v[j], rr);
          dw.v[j] = fma2(g.v[j], u.v[j], dw.v[j]);
          d.v[j] = mul2(fma2(u.v[j], mm, wg.v[j]), rr);
        }
        rg.pack(d);
      } else if (lane.turned) {
        rg.pack(back.of(rg.unpack()));
      }
      if (live) rg.store(dx, lane.a, lane.b);
      fetch();
    }
  }
  ring.drain();
  if (p.partial == nullptr) return;
  // [slot][column]: a slot has every column once
  __syncthreads();                // the ring's last rows are read
  float* red = mem.red;
  float* mine = red + (threadIdx.x / L) * D;
  *reinterpret_cast<float4*>(mine + lane.a) = Raw4<float>::pack(dw.v);
  *reinterpret_cast<float4*>(mine + lane.b) = Raw4<float>::pack(dw.v + 2);
  __syncthreads();
  // every thread adds eight slots of a column in pairs, then a thread the sums of each column
  constexpr int kGroups = kSlots / 8;
  static_assert(kGroups * D == kRopeThreads, "a thread a column and eight slots");
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = red[(threadIdx.x / D * 8 + i) * D + threadIdx.x % D];
  __syncthreads();
  red[threadIdx.x] = sum_in_pairs<8>(s);
  __syncthreads();
  if (threadIdx.x < D) {
    float t[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) t[i] = red[i * D + threadIdx.x];
    p.partial[((long long)run * gridDim.x + blockIdx.x) * D + threadIdx.x] =
        sum_in_pairs<kGroups>(t);
  }
}

// dw[c] = the sum of the partial rows; blockIdx.x: 0 = q, 1 = k; blockIdx.y: 16 columns, four to a
// thread, the rows dealt to 256 threads each.
constexpr int kDwThreads = 1024;
__global__ void __launch_bounds__(kDwThreads)
norm_rope_dw_kernel(const float* pq, const float* pk, int qrows, int krows, int D, float* dwq,
                    float* dwk) {
  __shared__ float4 red[kDwThreads / 32][4];
  griddep_wait();
  const float* p = blockIdx.x ? pk : pq;
  if (p == nullptr) return;
  const int rows = blockIdx.x ? krows : qrows;
  const int c = threadIdx.x % 4, col = blockIdx.y * 16 + c * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = threadIdx.x / 4; i < rows; i += kDwThreads / 4) {
    const float4 x = *reinterpret_cast<const float4*>(p + (long long)i * D + col);
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
#pragma unroll
  for (int o = 4; o < 32; o *= 2) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
    s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
  }
  if (threadIdx.x % 32 < 4) red[threadIdx.x / 32][c] = s;
  __syncthreads();
  if (threadIdx.x < 16) {
    float x[kDwThreads / 32];
#pragma unroll
    for (int w = 0; w < kDwThreads / 32; ++w)
      x[w] = reinterpret_cast<const float*>(red[w])[threadIdx.x];
    (blockIdx.x ? dwk : dwq)[blockIdx.y * 16 + threadIdx.x] = sum_in_pairs<kDwThreads / 32>(x);
  }
}

template <typename T, int D>
cudaError_t forward_d(NormRopeArgs<T>& a, int sms, cudaStream_t st) {
  const RopeGrid g = rope_grid((long long)a.B * a.N, a.part[0].heads + a.part[1].heads,
                               kRopeThreads / (D / 8), kRopeBlocks, sms);
  a.run = g.run;
  count_launch();
  return launch_pdl(a.interleaved ? norm_rope_kernel<T, D, true> : norm_rope_kernel<T, D, false>,
                    dim3(g.x, g.y), dim3(kRopeThreads), 0, st, a);
}

template <typename T, int D>
cudaError_t backward_d(NormRopeBackwardArgs<T>& a, float* partial, int sms, float* dwq, float* dwk,
                       cudaStream_t st) {
  // runs do not cross from q to k: one length for both, chosen for the longer part; the blocks'
  // partial rows have to fit the workspace
  const int hq = a.part[0].heads, hk = a.part[1].heads;
  const RopeGrid g = rope_grid((long long)a.B * a.N, std::max(hq, hk), kRopeThreads / (D / 8),
                               kRopeBlocks, sms);
  a.run = g.run;
  auto runs = [&](int heads) { return (heads + a.run - 1) / a.run; };
  const int most = norm_rope_backward_blocks(sms);
  while (runs(hq) + runs(hk) > most) a.run *= 2;
  a.qruns = runs(hq);
  const int y = a.qruns + runs(hk);
  const int x = std::min(g.x, most / y);
  a.part[0].partial = dwq ? partial : nullptr;
  a.part[1].partial = dwk ? partial + (size_t)x * a.qruns * D : nullptr;
  count_launch();
  cudaError_t e =
      launch_pdl(a.interleaved ? norm_rope_backward_kernel<T, D, true>
                               : norm_rope_backward_kernel<T, D, false>,
                 dim3(x, y), dim3(kRopeThreads), 0, st, a);
  if (e != cudaSuccess || (!dwq && !dwk)) return e;
  count_launch();
  return launch_pdl(norm_rope_dw_kernel, dim3(2, D / 16), dim3(kDwThreads), 0, st,
                    (const float*)a.part[0].partial, (const float*)a.part[1].partial, x * a.qruns,
                    x * (y - a.qruns), D, dwq, dwk);
}

}  // namespace

int norm_rope_backward_blocks(int sms) { return 8 * sms; }

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
