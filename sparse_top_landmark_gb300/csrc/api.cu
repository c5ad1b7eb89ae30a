// C ABI of libmita.so: argument validation, workspace cache, stage
// orchestration.  Every arithmetic step runs in the kernels of this library.
#include "mita.h"

#include <algorithm>
#include <cmath>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>
#include <string>
#include <type_traits>
#include <utility>

#include "common.cuh"
#include "kernels.h"

namespace mita {
namespace {

thread_local std::string g_msg;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_msg = buf;
  return code;
}

int cuda_fail(cudaError_t e, const char* where) {
  return fail(MITA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

struct DevState {
  int* status = nullptr;
  int num_sms = 0;
};

std::mutex g_mu;
std::map<int, DevState> g_dev;
struct WsEntry {
  void* ptr = nullptr;
  size_t bytes = 0;
};
std::map<std::pair<int, cudaStream_t>, WsEntry> g_ws;
std::map<std::pair<int, cudaStream_t>, WsEntry> g_stage;
// Bytes one cached buffer may grow to (0: no limit).  A growth beyond it fails exactly as a
// failed cudaMallocAsync does, before the allocator is called: the host-side way to make the
// allocation failure path run without exhausting a GPU.
std::atomic<unsigned long long> g_ws_limit{0};

int device_state(DevState** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(g_mu);
  DevState& s = g_dev[dev];
  if (s.status == nullptr) {
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    int* p = nullptr;
    e = cudaMalloc(&p, sizeof(int));
    if (e != cudaSuccess) return fail(MITA_ERR_OOM, "status word: %s", cudaGetErrorString(e));
    e = cudaMemset(p, 0, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemset");
    s.status = p;
    s.num_sms = sms;
  }
  *out = &s;
  return MITA_OK;
}

// One buffer per (device, stream) in `cache`, grown (stream-ordered) when a
// call needs more.
int cached_buffer(std::map<std::pair<int, cudaStream_t>, WsEntry>& cache, const char* what,
                  size_t bytes, cudaStream_t st, void** out) {
  *out = nullptr;
  if (bytes == 0) return MITA_OK;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(g_mu);
  WsEntry& w = cache[{dev, st}];
  if (w.bytes >= bytes) {
    *out = w.ptr;
    return MITA_OK;
  }
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  e = cudaStreamIsCapturing(st, &cs);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
  if (cs != cudaStreamCaptureStatusNone)
    return fail(MITA_ERR_UNSUPPORTED,
                "%s must grow to %zu bytes while the stream is capturing; make one "
                "call of this size outside capture first", what, bytes);
  if (w.ptr) {
    e = cudaFreeAsync(w.ptr, st);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFreeAsync");
    w.ptr = nullptr;
    w.bytes = 0;
  }
  const size_t want = bytes + bytes / 8;
  const unsigned long long limit = g_ws_limit.load();
  if (limit != 0 && want > limit)
    return fail(MITA_ERR_OOM, "%s of %zu bytes: above the workspace limit of %llu bytes", what,
                want, limit);
  void* p = nullptr;
  e = cudaMallocAsync(&p, want, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(MITA_ERR_OOM, "%s of %zu bytes: %s", what, want, cudaGetErrorString(e));
  }
  w.ptr = p;
  w.bytes = want;
  *out = p;
  return MITA_OK;
}

int workspace(size_t bytes, cudaStream_t st, void** out) {
  return cached_buffer(g_ws, "workspace", bytes, st, out);
}

// device copies of the host-buffer forward's inputs and output
int staging(size_t bytes, cudaStream_t st, void** out) {
  return cached_buffer(g_stage, "staging buffer", bytes, st, out);
}

// ---------------------------------------------------------------------------
// Validation
// ---------------------------------------------------------------------------
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_ptrs(std::initializer_list<std::pair<const void*, const char*>> ps) {
  for (auto& p : ps) {
    if (p.first == nullptr) return fail(MITA_ERR_INVALID_ARG, "%s is NULL", p.second);
    if (!aligned16(p.first))
      return fail(MITA_ERR_INVALID_ARG, "%s is not 16-byte aligned", p.second);
  }
  return MITA_OK;
}

int check_shape(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1)
    return fail(MITA_ERR_INVALID_ARG, "B, H, N must be >= 1 (got %d, %d, %d)", B, H, N);
  if (d != 16 && d != 32 && d != 64 && d != 128)
    return fail(MITA_ERR_UNSUPPORTED, "head dim d=%d not in {16, 32, 64, 128}", d);
  if ((long long)B * H * N >= (1LL << 31))
    return fail(MITA_ERR_UNSUPPORTED, "B*H*N must be < 2^31");
  return MITA_OK;
}

int check_m(int N, int m) {
  if (m < 1 || m > N) return fail(MITA_ERR_INVALID_ARG, "need 1 <= m <= N (m=%d, N=%d)", m, N);
  return MITA_OK;
}

int check_topk(int N, int topk) {
  if (topk < 1 || topk > N)
    return fail(MITA_ERR_INVALID_ARG, "need 1 <= topk <= N (topk=%d, N=%d)", topk, N);
  if (topk > kMaxTopk)
    return fail(MITA_ERR_UNSUPPORTED, "topk=%d above this build's limit %d", topk, kMaxTopk);
  return MITA_OK;
}

int check_s(int m, int s) {
  if (s < 1 || s > m) return fail(MITA_ERR_INVALID_ARG, "need 1 <= s <= m (s=%d)", s);
  if (s > kMaxRouteS)
    return fail(MITA_ERR_UNSUPPORTED, "s=%d above this build's limit %d", s, kMaxRouteS);
  return MITA_OK;
}

// B*H*N*s route entries must stay below 2^31
int check_entries(int B, int H, int N, int s) {
  if ((long long)B * H * N * s >= (1LL << 31))
    return fail(MITA_ERR_UNSUPPORTED, "B*H*N*s must be < 2^31");
  return MITA_OK;
}

// The landmark grid: lm_h x lm_w when given (both > 0), else 1 x m for a 1D
// sequence (grid_h = 1) and sqrt(m) x sqrt(m) for a 2D grid.
int check_grid(int N, int grid_h, int grid_w, int m, int lm_h = 0, int lm_w = 0,
               int* mh = nullptr, int* mw = nullptr) {
  if (grid_h < 1 || grid_w < 1 || (long long)grid_h * grid_w != N)
    return fail(MITA_ERR_INVALID_ARG, "grid %dx%d does not hold N=%d tokens", grid_h, grid_w, N);
  int h = 1, w = m;
  if (lm_h != 0 || lm_w != 0) {
    if (lm_h < 1 || lm_w < 1 || (long long)lm_h * lm_w != m)
      return fail(MITA_ERR_INVALID_ARG, "landmark grid %dx%d does not hold m=%d landmarks", lm_h,
                  lm_w, m);
    if (grid_h == 1 && lm_h != 1)
      return fail(MITA_ERR_INVALID_ARG, "a 1D sequence pools onto 1 x m landmarks");
    h = lm_h;
    w = lm_w;
  } else if (grid_h != 1) {
    int r = 1;
    while ((r + 1) * (r + 1) <= m) ++r;
    if (r * r != m)
      return fail(MITA_ERR_INVALID_ARG,
                  "2D pooling needs a square m (got %d) or an explicit landmark grid", m);
    h = w = r;
  }
  if (mh) *mh = h;
  if (mw) *mw = w;
  return MITA_OK;
}

int check_options(const mita_options* o) {
  if (o == nullptr) return MITA_OK;
  if (o->shared_temperature != MITA_SHARED_SQRT_D && o->shared_temperature != MITA_SHARED_D)
    return fail(MITA_ERR_INVALID_ARG, "unknown shared_temperature %d", o->shared_temperature);
  if (o->branches != MITA_BRANCHES_BOTH && o->branches != MITA_BRANCHES_ROUTED)
    return fail(MITA_ERR_INVALID_ARG, "unknown branches %d", o->branches);
  return MITA_OK;
}

#define MITA_TRY(x)                  \
  do {                               \
    int rc_ = (x);                   \
    if (rc_ != MITA_OK) return rc_;  \
  } while (0)

#define MITA_CUDA(x, where)                            \
  do {                                                 \
    cudaError_t e_ = (x);                              \
    if (e_ != cudaSuccess) return cuda_fail(e_, where); \
  } while (0)

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// ---------------------------------------------------------------------------
// Stage implementations (T = float or bf16)
// ---------------------------------------------------------------------------
template <typename T>
int pool_impl(const T* q, int B, int H, int N, int d, int gh, int gw, int m, T* qt,
              cudaStream_t st, int lm_h = 0, int lm_w = 0) {
  MITA_TRY(check_shape(B, H, N, d));
  MITA_TRY(check_m(N, m));
  int mh = 0, mw = 0;
  MITA_TRY(check_grid(N, gh, gw, m, lm_h, lm_w, &mh, &mw));
  MITA_TRY(check_ptrs({{q, "q"}, {qt, "q_tilde"}}));
  MITA_CUDA(launch_pool<T>(q, B * H, N, d, gh, gw, mh, mw, qt, st), "pool launch");
  return MITA_OK;
}

template <typename T>
int landmark_impl(const T* qt, const T* k, const T* v, int B, int H, int N, int d, int m,
                  int topk, int32_t* ti, float* vt, cudaStream_t st) {
  MITA_TRY(check_shape(B, H, N, d));
  MITA_TRY(check_m(N, m));
  MITA_TRY(check_topk(N, topk));
  MITA_TRY(check_ptrs({{qt, "q_tilde"}, {k, "k"}, {v, "v"}, {ti, "topk_idx"}, {vt, "v_tilde"}}));
  DevState* ds = nullptr;
  MITA_TRY(device_state(&ds));
  const LandmarkPlan plan =
      plan_landmark(B * H, N, d, m, topk, ds->num_sms, std::is_same<T, bf16>::value);
  void* ws = nullptr;
  MITA_TRY(workspace(landmark_ws_bytes(plan, B * H, N, d, m), st, &ws));
  const LandmarkWs lw = carve_landmark_ws(ws, plan, B * H, N, d, m);
  MITA_CUDA(launch_landmark<T>(qt, k, v, B * H, N, d, m, topk, plan, lw, ti, vt, ds->status, st),
            "landmark launch");
  return MITA_OK;
}

// Tensor-core route for bf16 / d = 64 / m <= 512 when no shared partial is
// requested; the SIMT kernel otherwise.
// per head: a count, then the ambiguous query ids and their fp32 best scores
size_t route_ws_bytes(int BH, int N) { return (size_t)BH * (2 * (size_t)N + 1) * sizeof(int); }

template <typename T>
bool route_uses_tc(int d, int m, int s, const float* lse, const float* so) {
  return std::is_same<T, bf16>::value && s == 1 && !lse && !so && route_tc_supported(d, m);
}
// the shared branch's partial requested (both outputs), s = 1 or 2: the tensor-core kernel
// that reuses the routing logits as the shared logits
template <typename T>
bool route_shared_uses_tc(int d, int m, int s, const float* lse, const float* so) {
  return std::is_same<T, bf16>::value && lse && so && route_shared_tc_supported(d, m, s);
}

template <typename T>
cudaError_t route_dispatch(const T* q, const T* qt, const float* vt, int BH, int N, int d, int m,
                           int s, int32_t* route, float* lse, float* so, DevState* ds, void* ws,
                           cudaStream_t st, int* hist = nullptr, bool* counted = nullptr,
                           bool prezeroed = false, int temp = 0) {
  if constexpr (std::is_same<T, bf16>::value) {
    if (route_uses_tc<T>(d, m, s, lse, so)) {
      if (counted) *counted = hist != nullptr;
      return launch_route_tc(q, qt, BH, N, m, ds->num_sms, route, static_cast<int*>(ws),
                             ds->status, hist, st, prezeroed);
    }
    if (route_shared_uses_tc<T>(d, m, s, lse, so)) {
      if (counted) *counted = hist != nullptr;
      return launch_route_shared_tc(q, qt, vt, BH, N, m, ds->num_sms, temp, 0, route, lse, so,
                                    static_cast<int*>(ws), ds->status, hist, st, prezeroed, s);
    }
  }
  return launch_route<T>(q, qt, vt, BH, N, d, m, s, route, lse, so, st, temp);
}

template <typename T>
int route_impl(const T* q, const T* qt, const float* vt, int B, int H, int N, int d, int m,
               int s, int32_t* route, float* lse, float* so, cudaStream_t st) {
  MITA_TRY(check_shape(B, H, N, d));
  MITA_TRY(check_m(N, m));
  MITA_TRY(check_s(m, s));
  MITA_TRY(check_entries(B, H, N, s));
  MITA_TRY(check_ptrs({{q, "q"}, {qt, "q_tilde"}, {route, "route_idx"}}));
  if (lse || so) MITA_TRY(check_ptrs({{vt, "v_tilde"}}));
  if (so) MITA_TRY(check_ptrs({{so, "shared_o"}}));
  DevState* ds = nullptr;
  MITA_TRY(device_state(&ds));
  void* ws = nullptr;
  if (route_uses_tc<T>(d, m, s, lse, so) || route_shared_uses_tc<T>(d, m, s, lse, so))
    MITA_TRY(workspace(route_ws_bytes(B * H, N), st, &ws));
  MITA_CUDA(route_dispatch<T>(q, qt, vt, B * H, N, d, m, s, route, lse, so, ds, ws, st),
            "route launch");
  return MITA_OK;
}

int bucket_impl(const int32_t* route, int B, int H, int N, int m, int s, int32_t* off,
                int32_t* qidx, cudaStream_t st) {
  if (B < 1 || H < 1 || N < 1) return fail(MITA_ERR_INVALID_ARG, "B, H, N must be >= 1");
  if ((long long)B * H * N >= (1LL << 31)) return fail(MITA_ERR_UNSUPPORTED, "B*H*N >= 2^31");
  MITA_TRY(check_m(N, m));
  MITA_TRY(check_s(m, s));
  MITA_TRY(check_entries(B, H, N, s));
  if (!route || !off || !qidx) return fail(MITA_ERR_INVALID_ARG, "NULL bucket argument");
  DevState* ds = nullptr;
  MITA_TRY(device_state(&ds));
  void* ws = nullptr;
  MITA_TRY(workspace(bucket_ws_bytes(B * H, N * s, m), st, &ws));
  MITA_CUDA(launch_bucket(route, B * H, N, m, ws, off, qidx, ds->status, st, false, s),
            "bucket launch");
  return MITA_OK;
}

template <typename T>
int expert_impl(const T* q, const T* k, const T* v, const T* qt, const float* vt,
                const int32_t* ti, const int32_t* off, const int32_t* qidx, const float* lse,
                const float* so, int B, int H, int N, int d, int m, int topk, int s, T* out,
                cudaStream_t st) {
  MITA_TRY(check_shape(B, H, N, d));
  MITA_TRY(check_m(N, m));
  MITA_TRY(check_topk(N, topk));
  MITA_TRY(check_s(m, s));
  MITA_TRY(check_entries(B, H, N, s));
  MITA_TRY(check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}}));
  if (!ti || !off || !qidx) return fail(MITA_ERR_INVALID_ARG, "NULL index argument");
  if ((lse == nullptr) != (so == nullptr))
    return fail(MITA_ERR_INVALID_ARG, "shared_lse and shared_o must be both set or both NULL");
  if (so == nullptr) MITA_TRY(check_ptrs({{qt, "q_tilde"}, {vt, "v_tilde"}}));
  DevState* ds = nullptr;
  MITA_TRY(device_state(&ds));
  if (s > 1) {
    // per-expert partials, merged per query with the shared branch's partial; without a
    // caller-supplied shared partial it is computed here (the SIMT route, s = 1, into scratch)
    const int BH = B * H;
    const size_t pb = align256(expert_partials_ws_bytes(BH, N, d, s));
    const size_t rb = align256((size_t)BH * N * 4), lb = align256((size_t)BH * N * 4);
    const size_t ob = align256((size_t)BH * N * d * 4);
    const bool tc = std::is_same<T, bf16>::value && expert_tc_supported(d, m, topk);
    const size_t tb = tc ? align256(expert_tc_partials_ws_bytes(BH, N, m, topk, s)) : 0;
    void* wsv = nullptr;
    MITA_TRY(workspace(pb + tb + (so ? 0 : rb + lb + ob), st, &wsv));
    char* ws = static_cast<char*>(wsv);
    if (so == nullptr) {
      int32_t* r1 = reinterpret_cast<int32_t*>(ws + pb + tb);
      float* l1 = reinterpret_cast<float*>(ws + pb + tb + rb);
      float* o1 = reinterpret_cast<float*>(ws + pb + tb + rb + lb);
      MITA_CUDA(launch_route<T>(q, qt, vt, BH, N, d, m, 1, r1, l1, o1, st), "shared partial");
      lse = l1;
      so = o1;
    }
    if constexpr (std::is_same<T, bf16>::value) {
      if (tc) {
        const ExpertPartials part = carve_expert_partials(ws, BH, N, d, s);
        MITA_CUDA(launch_expert_tc_partials(q, k, v, ti, off, qidx, BH, N, m, topk, s,
                                            ds->num_sms, ws + pb, part, ds->status, st),
                  "expert launch");
        MITA_CUDA(launch_expert_merge<T>(lse, so, 0, part, BH, N, d, s, out, ds->status, st),
                  "merge launch");
        return MITA_OK;
      }
    }
    MITA_CUDA(launch_expert_attn<T>(q, k, v, qt, vt, ti, off, qidx, lse, so, BH, N, d, m, topk, s,
                                    ws, out, ds->status, st),
              "expert launch");
    return MITA_OK;
  }
  if constexpr (std::is_same<T, bf16>::value) {
    if (expert_tc_supported(d, m, topk)) {
      // with a carried shared partial the kernel attends over the raw pairs only and merges
      void* ws = nullptr;
      MITA_TRY(workspace(expert_tc_ws_bytes(B * H, N, m, topk), st, &ws));
      MITA_CUDA(launch_expert_tc(q, k, v, qt, vt, ti, off, qidx, B * H, N, m, topk, ds->num_sms,
                                 ws, out, ds->status, st, 0, 0, lse, so, 0),
                "expert launch");
      return MITA_OK;
    }
  }
  MITA_CUDA(launch_expert_attn<T>(q, k, v, qt, vt, ti, off, qidx, lse, so, B * H, N, d, m, topk,
                                  1, nullptr, out, ds->status, st),
            "expert launch");
  return MITA_OK;
}

struct ForwardLayout {
  size_t qt, vt, ti, route, off, qidx, lm, bk, ex, rt, lse, so, total;
  LandmarkPlan plan;
};

ForwardLayout forward_layout(int BH, int N, int d, int m, int topk, int s, size_t esize, int sms) {
  ForwardLayout L{};
  L.plan = plan_landmark(BH, N, d, m, topk, sms, esize == 2);
  const size_t NS = (size_t)N * s;
  size_t o = 0;
  L.qt = o; o += align256((size_t)BH * m * d * esize);
  L.vt = o; o += align256((size_t)BH * m * d * 4);
  L.ti = o; o += align256((size_t)BH * m * topk * 4);
  L.route = o; o += align256((size_t)BH * NS * 4);
  L.off = o; o += align256((size_t)BH * (m + 1) * 4);
  L.qidx = o; o += align256((size_t)BH * NS * 4);
  L.lm = o; o += align256(landmark_ws_bytes(L.plan, BH, N, d, m));
  L.bk = o; o += align256(bucket_ws_bytes(BH, (int)NS, m));
  L.ex = o;
  if (s > 1) {
    o += align256(expert_partials_ws_bytes(BH, N, d, s));
    if (esize == 2 && expert_tc_supported(d, m, topk))
      o += align256(expert_tc_partials_ws_bytes(BH, N, m, topk, s));
  }
  else if (esize == 2 && expert_tc_supported(d, m, topk))
    o += align256(std::max(expert_tc_ws_bytes(BH, N, m, topk),
                           N <= 1024 ? expert_masked_ws_bytes(BH, N, m) : size_t(0)));
  L.rt = o; o += align256(route_ws_bytes(BH, N));
  // s > 1: the shared branch's partial, emitted by the route kernel
  L.lse = o; if (s > 1) o += align256((size_t)BH * N * 4);
  L.so = o; if (s > 1) o += align256((size_t)BH * N * d * 4);
  L.total = o;
  return L;
}

// The forward's counters, cleared by one kernel at its start (a memset between two
// kernels would hold back the next kernel's early launch): the landmark stage's
// slow-row count, the heads' ambiguous-query counts and the bucket histogram.
__global__ void __launch_bounds__(256)
forward_zero_kernel(int* a, long long na, int* b, long long nb, int* c, long long nc) {
  griddep_wait();
  const long long t0 = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long t = t0; t < na; t += stride) a[t] = 0;
  for (long long t = t0; t < nb; t += stride) b[t] = 0;
  for (long long t = t0; t < nc; t += stride) c[t] = 0;
}

template <typename T>
int forward_impl(const T* q, const T* k, const T* v, int B, int H, int N, int d, int gh, int gw,
                 int m, int topk, int s, T* out, cudaStream_t st,
                 const mita_options* opt = nullptr) {
  MITA_TRY(check_shape(B, H, N, d));
  MITA_TRY(check_m(N, m));
  MITA_TRY(check_options(opt));
  const int temp = opt ? opt->shared_temperature : MITA_SHARED_SQRT_D;
  const int routed = opt ? (opt->branches == MITA_BRANCHES_ROUTED) : 0;
  int mh = 0, mw = 0;
  MITA_TRY(check_grid(N, gh, gw, m, opt ? opt->landmark_grid_h : 0,
                      opt ? opt->landmark_grid_w : 0, &mh, &mw));
  MITA_TRY(check_topk(N, topk));
  MITA_TRY(check_s(m, s));
  MITA_TRY(check_entries(B, H, N, s));
  MITA_TRY(check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}}));
  DevState* ds = nullptr;
  MITA_TRY(device_state(&ds));
  const int BH = B * H;
  const ForwardLayout L = forward_layout(BH, N, d, m, topk, s, sizeof(T), ds->num_sms);
  void* wsv = nullptr;
  MITA_TRY(workspace(L.total, st, &wsv));
  char* ws = static_cast<char*>(wsv);
  T* qt = reinterpret_cast<T*>(ws + L.qt);
  float* vt = reinterpret_cast<float*>(ws + L.vt);
  int32_t* ti = reinterpret_cast<int32_t*>(ws + L.ti);
  int32_t* route = reinterpret_cast<int32_t*>(ws + L.route);
  int32_t* off = reinterpret_cast<int32_t*>(ws + L.off);
  int32_t* qidx = reinterpret_cast<int32_t*>(ws + L.qidx);
  const LandmarkWs lw = carve_landmark_ws(ws + L.lm, L.plan, BH, N, d, m);
  {
    const long long nh = (long long)BH * m * (((long long)N * s + kBucketChunk - 1) / kBucketChunk);
    MITA_CUDA(launch_pdl(forward_zero_kernel, dim3((unsigned)std::min<long long>(
                             (nh + 255) / 256 + 1, (long long)ds->num_sms * 4)),
                         dim3(256), 0, st, lw.nslow, 1LL, reinterpret_cast<int*>(ws + L.rt),
                         (long long)BH, reinterpret_cast<int*>(ws + L.bk), nh),
              "counter clearing");
    count_launch();
  }
  MITA_CUDA(launch_pool<T>(q, BH, N, d, gh, gw, mh, mw, qt, st), "pool launch");
  MITA_CUDA(launch_landmark<T>(qt, k, v, BH, N, d, m, topk, L.plan, lw, ti, vt, ds->status, st,
                               true),
            "landmark launch");
  if (s > 1) {
    // top-s routing with the shared branch's partial, grouping of the N*s (query, expert)
    // entries, per-expert partials and their merge
    float* lse = reinterpret_cast<float*>(ws + L.lse);
    float* so = reinterpret_cast<float*>(ws + L.so);
    // routing only: no shared partial (the SIMT route then lists the routes alone); with the
    // shared branch, s = 2 and m <= 256 route on the tensor cores, the shared partial's output
    // in bf16
    int so_bf16 = 0;
    bool counted = false;       // the tensor-core route counts the bucket histogram too
    if constexpr (std::is_same<T, bf16>::value) {
      if (!routed && route_shared_tc_supported(d, m, s)) {
        so_bf16 = 1;
        counted = true;
        MITA_CUDA(launch_route_shared_tc(q, qt, vt, BH, N, m, ds->num_sms, temp, 1, route, lse, so,
                                         reinterpret_cast<int*>(ws + L.rt), ds->status,
                                         reinterpret_cast<int*>(ws + L.bk), st, true, s),
                  "route launch");
      }
    }
    if (!so_bf16)
      MITA_CUDA(route_dispatch<T>(q, qt, vt, BH, N, d, m, s, route, routed ? nullptr : lse,
                                  routed ? nullptr : so, ds, ws + L.rt, st, nullptr, nullptr, true,
                                  temp),
                "route launch");
    MITA_CUDA(launch_bucket(route, BH, N, m, ws + L.bk, off, qidx, ds->status, st, counted, s),
              "bucket launch");
    if constexpr (std::is_same<T, bf16>::value) {
      if (expert_tc_supported(d, m, topk)) {
        // every (query, expert) entry's raw-pair partial on the tensor cores (fp32 outputs:
        // bf16 partials measured beyond the output tolerance), then the merge
        const ExpertPartials part = carve_expert_partials(ws + L.ex, BH, N, d, s);
        void* tws = ws + L.ex + align256(expert_partials_ws_bytes(BH, N, d, s));
        MITA_CUDA(launch_expert_tc_partials(q, k, v, ti, off, qidx, BH, N, m, topk, s,
                                            ds->num_sms, tws, part, ds->status, st),
                  "expert launch");
        MITA_CUDA(launch_expert_merge<T>(routed ? nullptr : lse, routed ? nullptr : so, so_bf16,
                                         part, BH, N, d, s, out, ds->status, st),
                  "merge launch");
        return MITA_OK;
      }
    }
    MITA_CUDA(launch_expert_attn<T>(q, k, v, qt, vt, ti, off, qidx, lse, so, BH, N, d, m, topk, s,
                                    ws + L.ex, out, ds->status, st, temp, routed),
              "expert launch");
    return MITA_OK;
  }
  if constexpr (std::is_same<T, bf16>::value) {
    if (expert_tc_supported(d, m, topk) && expert_masked_preferred(N, m, topk, routed)) {
      // short sequences: each query's expert from the route, then per-head query tiles over
      // all keys masked to that expert's set -- no grouping needed
      MITA_CUDA(route_dispatch<T>(q, qt, vt, BH, N, d, m, 1, route, nullptr, nullptr, ds,
                                  ws + L.rt, st, nullptr, nullptr, true),
                "route launch");
      MITA_CUDA(launch_expert_masked_tc(q, k, v, qt, vt, ti, route, BH, N, m, topk, ds->num_sms,
                                        ws + L.ex, out, ds->status, st, temp, routed),
                "expert launch");
      return MITA_OK;
    }
  }
  // s = 1: the expert kernel recomputes the shared logits q . q~ on the tensor cores rather
  // than taking them from the route stage as a carried partial (measured: the carried split,
  // route_shared_tc + raw-pairs-only expert, is slower at both long workloads)
  // the tensor-core route also counts the bucket stage's (expert, chunk) histogram
  bool counted = false;
  MITA_CUDA(route_dispatch<T>(q, qt, vt, BH, N, d, m, 1, route, nullptr, nullptr, ds, ws + L.rt,
                              st, reinterpret_cast<int*>(ws + L.bk), &counted, true),
            "route launch");
  MITA_CUDA(launch_bucket(route, BH, N, m, ws + L.bk, off, qidx, ds->status, st, counted),
            "bucket launch");
  if constexpr (std::is_same<T, bf16>::value) {
    if (expert_tc_supported(d, m, topk)) {
      MITA_CUDA(launch_expert_tc(q, k, v, qt, vt, ti, off, qidx, BH, N, m, topk, ds->num_sms,
                                 ws + L.ex, out, ds->status, st, temp, routed),
                "expert launch");
      return MITA_OK;
    }
  }
  MITA_CUDA(launch_expert_attn<T>(q, k, v, qt, vt, ti, off, qidx, nullptr, nullptr, BH, N, d, m,
                                  topk, 1, nullptr, out, ds->status, st, temp, routed),
            "expert launch");
  return MITA_OK;
}

template <typename T>
int dense_impl(const T* q, const T* k, const T* v, int B, int H, int N, int d, T* out,
               cudaStream_t st) {
  MITA_TRY(check_shape(B, H, N, d));
  MITA_TRY(check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}}));
  DevState* ds = nullptr;
  MITA_TRY(device_state(&ds));
  const int BH = B * H;
  void* ws = nullptr;
  if constexpr (std::is_same<T, bf16>::value) {
    if (d == 64) {
      MITA_TRY(workspace(dense_tc_ws_bytes(BH, N), st, &ws));
      MITA_CUDA(launch_dense_tc(q, k, v, BH, N, ds->num_sms, ws, out, ds->status, st),
                "dense launch");
      return MITA_OK;
    }
  }
  MITA_TRY(workspace(dense_simt_ws_bytes(BH, N), st, &ws));
  MITA_CUDA(launch_dense_attn<T>(q, k, v, BH, N, d, ws, out, ds->status, st), "dense launch");
  return MITA_OK;
}

// The backward with the selections held constant: the forward's selections and partials
// recomputed by the forward's own kernels, then the gradient kernels (backward.cu).
template <typename T>
int backward_impl(const T* q, const T* k, const T* v, const T* dout, int B, int H, int N, int d,
                  int gh, int gw, int m, int topk, int s, const mita_options* opt, float* dq,
                  float* dk, float* dv, cudaStream_t st) {
  MITA_TRY(check_shape(B, H, N, d));
  MITA_TRY(check_m(N, m));
  MITA_TRY(check_options(opt));
  int mh = 0, mw = 0;
  MITA_TRY(check_grid(N, gh, gw, m, opt ? opt->landmark_grid_h : 0,
                      opt ? opt->landmark_grid_w : 0, &mh, &mw));
  MITA_TRY(check_topk(N, topk));
  MITA_TRY(check_s(m, s));
  MITA_TRY(check_entries(B, H, N, s));
  MITA_TRY(check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {dout, "dout"}, {dq, "dq"}, {dk, "dk"},
                       {dv, "dv"}}));
  const int temp = opt ? opt->shared_temperature : MITA_SHARED_SQRT_D;
  const int routed = opt ? (opt->branches == MITA_BRANCHES_ROUTED) : 0;
  DevState* ds = nullptr;
  MITA_TRY(device_state(&ds));
  const int BH = B * H;
  const size_t BHN = (size_t)BH * N, NS = (size_t)N * s;
  const LandmarkPlan plan = plan_landmark(BH, N, d, m, topk, ds->num_sms, sizeof(T) == 2);
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += align256(bytes); return at; };
  const size_t o_qt = take((size_t)BH * m * d * sizeof(T)), o_vt = take((size_t)BH * m * d * 4);
  const size_t o_ti = take((size_t)BH * m * topk * 4), o_r = take((size_t)BH * NS * 4);
  const size_t o_off = take((size_t)BH * (m + 1) * 4), o_qi = take((size_t)BH * NS * 4);
  const size_t o_lm = take(landmark_ws_bytes(plan, BH, N, d, m));
  const size_t o_bk = take(bucket_ws_bytes(BH, (int)NS, m));
  const size_t o_sl = take(BHN * 4), o_so = take(BHN * d * 4);
  const size_t o_pt = take(expert_partials_ws_bytes(BH, N, d, s));
  const size_t o_lse = take(BHN * 4), o_dn = take(BHN * 4);
  const size_t o_la = take((size_t)BH * m * 4), o_cv = take((size_t)BH * m * 4);
  const size_t o_dqt = take((size_t)BH * m * d * 4), o_dvt = take((size_t)BH * m * d * 4);
  // bf16 with d = 64: the selections are recomputed by the tensor-core route and expert
  // kernels where they apply, and the gradient passes run on the tensor cores
  const bool mma = std::is_same<T, bf16>::value && d == 64;
  const bool tc_expert = mma && expert_tc_supported(d, m, topk);
  const bool tc_route = std::is_same<T, bf16>::value &&
                        (routed ? s == 1 && route_tc_supported(d, m) : route_shared_tc_supported(d, m, s));
  const size_t o_v16 = mma ? take((size_t)BH * m * 64 * 2) : 0;
  const size_t o_dv16 = mma ? take((size_t)BH * m * 64 * 2) : 0;
  const size_t o_rws = tc_route ? take(route_ws_bytes(BH, N)) : 0;
  const size_t o_tcx = tc_expert ? take(expert_tc_partials_ws_bytes(BH, N, m, topk, s)) : 0;
  void* wsv = nullptr;
  MITA_TRY(workspace(o, st, &wsv));
  char* ws = static_cast<char*>(wsv);
  T* qt = reinterpret_cast<T*>(ws + o_qt);
  float* vt = reinterpret_cast<float*>(ws + o_vt);
  int32_t* ti = reinterpret_cast<int32_t*>(ws + o_ti);
  int32_t* route = reinterpret_cast<int32_t*>(ws + o_r);
  int32_t* off = reinterpret_cast<int32_t*>(ws + o_off);
  int32_t* qidx = reinterpret_cast<int32_t*>(ws + o_qi);
  float* sl = reinterpret_cast<float*>(ws + o_sl);
  float* so = reinterpret_cast<float*>(ws + o_so);
  ExpertPartials part;
  part.o = reinterpret_cast<float*>(ws + o_pt);
  part.lse = part.o + BHN * s * d;
  part.pos = reinterpret_cast<int*>(part.lse + BHN * s);
  part.cnt = part.pos + BHN * s;
  // dq, dk, dv are cleared by the gradient launcher where its kernels add rather than store
  MITA_CUDA(cudaMemsetAsync(ws + o_dqt, 0, (o_dvt - o_dqt) + (size_t)BH * m * d * 4, st),
            "clearing scratch");
  MITA_CUDA(launch_pool<T>(q, BH, N, d, gh, gw, mh, mw, qt, st), "pool launch");
  LandmarkWs lw = carve_landmark_ws(ws + o_lm, plan, BH, N, d, m);
  lw.lse_out = reinterpret_cast<float*>(ws + o_la);   // each landmark's softmax normaliser
  MITA_CUDA(launch_landmark<T>(qt, k, v, BH, N, d, m, topk, plan, lw, ti, vt, ds->status, st),
            "landmark launch");
  MITA_CUDA(route_dispatch<T>(q, qt, vt, BH, N, d, m, s, route, routed ? nullptr : sl,
                              routed ? nullptr : so, ds, tc_route ? ws + o_rws : nullptr, st,
                              nullptr, nullptr, false, temp),
            "route launch");
  MITA_CUDA(launch_bucket(route, BH, N, m, ws + o_bk, off, qidx, ds->status, st, false, s),
            "bucket launch");
  if constexpr (std::is_same<T, bf16>::value) {
    if (tc_expert)
      MITA_CUDA(launch_expert_tc_partials(q, k, v, ti, off, qidx, BH, N, m, topk, s,
                                          ds->num_sms, ws + o_tcx, part, ds->status, st),
                "expert partials");
  }
  if (!tc_expert)
    MITA_CUDA(launch_expert_partials<T>(q, k, v, ti, off, qidx, BH, N, d, m, topk, s, part,
                                        ds->status, st),
              "expert partials");
  BwdArgs<T> a{};
  a.q = q; a.k = k; a.v = v; a.dout = dout; a.q_tilde = qt; a.v_tilde = vt;
  a.topk_idx = ti; a.bucket_off = off; a.bucket_qidx = qidx;
  a.sh_lse = routed ? nullptr : sl; a.sh_o = routed ? nullptr : so; a.part = part;
  a.BH = BH; a.N = N; a.m = m; a.topk = topk; a.s = s; a.routed = routed;
  a.c_sh = (float)(temp == MITA_SHARED_D ? 1.0 / d : 1.0 / std::sqrt((double)d));
  a.grid_h = gh; a.grid_w = gw; a.mh = mh; a.mw = mw;
  a.lse = reinterpret_cast<float*>(ws + o_lse); a.Dn = reinterpret_cast<float*>(ws + o_dn);
  a.lseA = reinterpret_cast<float*>(ws + o_la); a.cvt = reinterpret_cast<float*>(ws + o_cv);
  a.dqt = reinterpret_cast<float*>(ws + o_dqt); a.dvt = reinterpret_cast<float*>(ws + o_dvt);
  a.dq = dq; a.dk = dk; a.dv = dv; a.status = ds->status;
  if (mma) {
    a.vt16 = reinterpret_cast<bf16*>(ws + o_v16);
    a.dvt16 = reinterpret_cast<bf16*>(ws + o_dv16);
  }
  MITA_CUDA(launch_backward<T>(a, d, st), "backward launch");
  return MITA_OK;
}

// ---------------------------------------------------------------------------
// q / k preparation and the paged cache
// ---------------------------------------------------------------------------
// The device's state for calls that may be captured: its first use allocates, which would break
// a capture, so that is refused before anything is touched.
int device_state_for(cudaStream_t st, DevState** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  {
    std::lock_guard<std::mutex> lk(g_mu);
    auto it = g_dev.find(dev);
    if (it != g_dev.end() && it->second.status != nullptr) {
      *out = &it->second;
      return MITA_OK;
    }
  }
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  e = cudaStreamIsCapturing(st, &cs);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
  if (cs != cudaStreamCaptureStatusNone)
    return fail(MITA_ERR_UNSUPPORTED,
                "the library's first call on a device cannot be captured; make one outside "
                "capture first");
  return device_state(out);
}

int check_head_dim(int d) {
  if (d != 16 && d != 32 && d != 64 && d != 128)
    return fail(MITA_ERR_UNSUPPORTED, "head dim d=%d not in {16, 32, 64, 128}", d);
  return MITA_OK;
}

int check_aligned(const void* p, size_t to, const char* name) {
  if (p == nullptr) return fail(MITA_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % to != 0)
    return fail(MITA_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, to);
  return MITA_OK;
}

int check_rope(int d, int rot, const double* inv_freq, float eps) {
  if (rot < 0 || rot > d || rot % 8 != 0)
    return fail(MITA_ERR_INVALID_ARG, "rot=%d must be a multiple of 8 in [0, d=%d]", rot, d);
  if (rot > 0) MITA_TRY(check_aligned(inv_freq, 8, "inv_freq"));
  if (!(eps >= 0.f)) return fail(MITA_ERR_INVALID_ARG, "eps must be >= 0");
  return MITA_OK;
}

// Element strides of an array of rows.  Rows must start on 16-byte boundaries; the stride of a
// dimension of size 1 is not looked at.
template <int K>
int row_strides(const int64_t (&given)[K], const int (&size)[K], size_t esize, const char* name,
                long long (&out)[K]) {
  for (int i = 0; i < K; ++i) {
    out[i] = size[i] == 1 ? 0 : given[i];
    if (out[i] < 0 || out[i] % (long long)(16 / esize) != 0)
      return fail(MITA_ERR_INVALID_ARG,
                  "%s: stride %lld is negative or leaves rows off 16-byte boundaries", name,
                  out[i]);
  }
  return MITA_OK;
}

// Rows of a token: the kernels take runs of them, whose ends (at most 2^16 behind the last) are 32-bit
// numbers.
int check_rows(long long rows, const char* name) {
  if (rows > (1LL << 30)) return fail(MITA_ERR_UNSUPPORTED, "%s must be at most 2^30", name);
  return MITA_OK;
}

int check_bhn(int B, int Hq, int Hkv, int N, int d) {
  if (B < 0 || N < 0 || Hq < 1 || Hkv < 0)
    return fail(MITA_ERR_INVALID_ARG, "need B, N, Hkv >= 0 and Hq >= 1 (got %d, %d, %d, %d)", B, N,
                Hkv, Hq);
  MITA_TRY(check_head_dim(d));
  MITA_TRY(check_rows((long long)Hq + Hkv, "Hq+Hkv"));
  const long long most = 1LL << 31;
  if ((long long)B * N >= most || (long long)B * N * ((long long)Hq + Hkv) >= most)
    return fail(MITA_ERR_UNSUPPORTED, "B*(Hq+Hkv)*N must be < 2^31");
  return MITA_OK;
}

int check_positions(const int32_t* positions, int64_t stride) {
  if (positions == nullptr) return MITA_OK;
  if (stride < 0) return fail(MITA_ERR_INVALID_ARG, "positions_stride must be >= 0");
  return check_aligned(positions, 4, "positions");
}

// What the calls with positions of several axes have besides.
struct Axes {
  bool several;
  const int32_t* freq_axis;
  int64_t stride;
  int axes;
};
template <typename P>
Axes axes_of(const P* p) {
  if constexpr (std::is_same<P, mita_qk_norm_rope_axes_params>::value ||
                std::is_same<P, mita_qk_norm_rope_axes_backward_params>::value)
    return {true, p->freq_axis, p->positions_axis_stride, p->axes};
  else
    return {};
}
int check_axes(const Axes& x, const int32_t* positions, int rot) {
  if (x.axes < 1) return fail(MITA_ERR_INVALID_ARG, "axes=%d must be positive", x.axes);
  if (x.stride < 0) return fail(MITA_ERR_INVALID_ARG, "positions_axis_stride must be >= 0");
  MITA_TRY(check_aligned(positions, 4, "positions"));
  return rot > 0 ? check_aligned(x.freq_axis, 4, "freq_axis") : (int)MITA_OK;
}

template <typename T, typename P>
int norm_rope_impl(const P* p, cudaStream_t st) {
  if (p == nullptr) return fail(MITA_ERR_INVALID_ARG, "params is NULL");
  const Axes axes = axes_of(p);
  MITA_TRY(check_bhn(p->B, p->Hq, p->Hkv, p->N, p->d));
  MITA_TRY(check_rope(p->d, p->rot, p->inv_freq, p->eps));
  MITA_TRY(check_positions(p->positions, p->positions_stride));
  if (p->B == 0 || p->N == 0) return MITA_OK;
  if (axes.several) MITA_TRY(check_axes(axes, p->positions, p->rot));
  NormRopeArgs<T> a{};
  auto part = [&](NormRopePart<T>& o, const void* x, void* y, const float* w, int heads,
                  const int64_t (&xs)[3], const int64_t (&ys)[3], const char* nx, const char* ny,
                  const char* nw) {
    if (heads == 0) return (int)MITA_OK;
    MITA_TRY(check_ptrs({{x, nx}, {y, ny}}));
    if (w) MITA_TRY(check_aligned(w, 16, nw));
    long long sx[3], sy[3];
    MITA_TRY(row_strides<3>(xs, {p->B, heads, p->N}, sizeof(T), nx, sx));
    MITA_TRY(row_strides<3>(ys, {p->B, heads, p->N}, sizeof(T), ny, sy));
    o = {static_cast<const T*>(x), static_cast<T*>(y), w, sx[0], sx[1], sx[2], sy[0], sy[1], sy[2],
         heads};
    return (int)MITA_OK;
  };
  MITA_TRY(part(a.part[0], p->q, p->q_out, p->q_weight, p->Hq, p->q_strides, p->q_out_strides, "q",
                "q_out", "q_weight"));
  MITA_TRY(part(a.part[1], p->k, p->k_out, p->k_weight, p->Hkv, p->k_strides, p->k_out_strides,
                "k", "k_out", "k_weight"));
  a.positions = p->positions;
  a.pos_b = p->positions_stride;
  a.inv_freq = p->inv_freq;
  a.B = p->B; a.N = p->N; a.rot = p->rot; a.interleaved = p->interleaved != 0; a.eps = p->eps;
  DevState* ds = nullptr;
  MITA_TRY(device_state_for(st, &ds));
  a.freq_axis = axes.freq_axis; a.pos_a = axes.stride; a.axes = axes.axes; a.status = ds->status;
  MITA_CUDA((axes.several ? launch_norm_rope_axes<T> : launch_norm_rope<T>)(a, p->d, ds->num_sms, st),
            "norm and rotation launch");
  return MITA_OK;
}

int current_sms() {
  int sms = 152, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaGetLastError();
  return sms;
}

int check_workspace(const void* ws, uint64_t have, uint64_t need) {
  if (need == 0) return MITA_OK;
  if (have < need)
    return fail(MITA_ERR_INVALID_ARG, "workspace of %llu bytes: this call needs %llu",
                (unsigned long long)have, (unsigned long long)need);
  return check_aligned(ws, 16, "workspace");
}

uint64_t norm_rope_backward_ws(int d, int sms) {
  return (uint64_t)norm_rope_backward_blocks(sms) * d * sizeof(float);
}

template <typename T, typename P>
int norm_rope_backward_impl(const P* p, cudaStream_t st) {
  if (p == nullptr) return fail(MITA_ERR_INVALID_ARG, "params is NULL");
  const Axes axes = axes_of(p);
  MITA_TRY(check_bhn(p->B, p->Hq, p->Hkv, p->N, p->d));
  MITA_TRY(check_rope(p->d, p->rot, p->inv_freq, p->eps));
  MITA_TRY(check_positions(p->positions, p->positions_stride));
  const bool empty = p->B == 0 || p->N == 0;
  if (axes.several && !empty) MITA_TRY(check_axes(axes, p->positions, p->rot));
  NormRopeBackwardArgs<T> a{};
  float* dws[2] = {nullptr, nullptr};     // of parts with rows
  float* none[2] = {nullptr, nullptr};    // sums over no rows
  auto part = [&](int i, const void* x, const void* dy, void* dx, const float* w, float* dw,
                  int heads, const int64_t (&xs)[3], const int64_t (&dys)[3],
                  const int64_t (&dxs)[3], const char* const (&name)[5]) {
    if (heads == 0 && (!w || !dw)) return (int)MITA_OK;
    if (w) {
      MITA_TRY(check_aligned(w, 16, name[3]));
      MITA_TRY(check_aligned(dw, 4, name[4]));
      (empty || heads == 0 ? none : dws)[i] = dw;
    } else if (dw) {
      return fail(MITA_ERR_INVALID_ARG, "%s given without %s", name[4], name[3]);
    }
    if (empty || heads == 0) return (int)MITA_OK;
    MITA_TRY(check_ptrs({{dy, name[1]}, {dx, name[2]}}));
    if (w) MITA_TRY(check_ptrs({{x, name[0]}}));   // else x is not read
    const int size[3] = {p->B, heads, p->N};
    long long sx[3] = {}, sdy[3], sdx[3];
    if (w) MITA_TRY(row_strides<3>(xs, size, sizeof(T), name[0], sx));
    MITA_TRY(row_strides<3>(dys, size, sizeof(T), name[1], sdy));
    MITA_TRY(row_strides<3>(dxs, size, sizeof(T), name[2], sdx));
    a.part[i] = {static_cast<const T*>(x), static_cast<const T*>(dy), static_cast<T*>(dx), w,
                 nullptr, sx[0], sx[1], sx[2], sdy[0], sdy[1], sdy[2], sdx[0], sdx[1], sdx[2],
                 heads};
    return (int)MITA_OK;
  };
  MITA_TRY(part(0, p->q, p->dq_out, p->dq, p->q_weight, p->dq_weight, p->Hq, p->q_strides,
                p->dq_out_strides, p->dq_strides, {"q", "dq_out", "dq", "q_weight", "dq_weight"}));
  MITA_TRY(part(1, p->k, p->dk_out, p->dk, p->k_weight, p->dk_weight, p->Hkv, p->k_strides,
                p->dk_out_strides, p->dk_strides, {"k", "dk_out", "dk", "k_weight", "dk_weight"}));
  DevState* ds = nullptr;
  if (!empty) {
    if (dws[0] || dws[1])
      MITA_TRY(check_workspace(p->workspace, p->workspace_bytes,
                               norm_rope_backward_ws(p->d, current_sms())));
    MITA_TRY(device_state_for(st, &ds));
  }
  for (float* w : none)
    if (w) MITA_CUDA(cudaMemsetAsync(w, 0, p->d * sizeof(float), st), "weight gradient");
  if (empty) return MITA_OK;
  a.positions = p->positions;
  a.pos_b = p->positions_stride;
  a.inv_freq = p->inv_freq;
  a.B = p->B; a.N = p->N; a.rot = p->rot; a.interleaved = p->interleaved != 0; a.eps = p->eps;
  a.freq_axis = axes.freq_axis; a.pos_a = axes.stride; a.axes = axes.axes; a.status = ds->status;
  MITA_CUDA((axes.several ? launch_norm_rope_axes_backward<T> : launch_norm_rope_backward<T>)(
                a, p->d, static_cast<float*>(p->workspace), ds->num_sms, dws[0], dws[1], st),
            "norm and rotation gradient launch");
  return MITA_OK;
}

int check_pages(int S, int Hkv, int num_pages, int page_size, int width) {
  if (S < 0 || Hkv < 1 || num_pages < 0 || width < 0)
    return fail(MITA_ERR_INVALID_ARG,
                "need S, num_pages, table_width >= 0 and Hkv >= 1 (got %d, %d, %d, %d)", S,
                num_pages, width, Hkv);
  if (page_size < 1 || page_size > kMaxPageSize || (page_size & (page_size - 1)) != 0)
    return fail(MITA_ERR_UNSUPPORTED, "page_size=%d is not a power of two in [1, %d]", page_size,
                kMaxPageSize);
  // positions are 32-bit numbers, those of a tile that begins before the last one included
  if ((long long)width * page_size > (1LL << 31) - (1 << 16))
    return fail(MITA_ERR_UNSUPPORTED, "table_width*page_size must be at most 2^31 - 2^16");
  return MITA_OK;
}

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

template <typename T>
int cache_append_impl(const mita_cache_append_params* p, cudaStream_t st) {
  if (p == nullptr) return fail(MITA_ERR_INVALID_ARG, "params is NULL");
  if (p->tokens < 0 || p->Hq < 0)
    return fail(MITA_ERR_INVALID_ARG, "need tokens, Hq >= 0 (got %d, %d)", p->tokens, p->Hq);
  MITA_TRY(check_pages(p->S, p->Hkv, p->num_pages, p->page_size, p->table_width));
  MITA_TRY(check_head_dim(p->d));
  MITA_TRY(check_rope(p->d, p->rot, p->inv_freq, p->eps));
  if ((long long)p->Hq + 2LL * p->Hkv >= (1LL << 31) ||
      (long long)p->tokens * ((long long)p->Hq + 2LL * p->Hkv) >= (1LL << 31))
    return fail(MITA_ERR_UNSUPPORTED, "tokens*(Hq+2*Hkv) must be < 2^31");
  MITA_TRY(check_rows((long long)p->Hq + 2LL * p->Hkv, "Hq+2*Hkv"));
  if (p->seq_start == nullptr && p->tokens != p->S)
    return fail(MITA_ERR_INVALID_ARG,
                "without seq_start every sequence has one new token (tokens=%d, S=%d)", p->tokens,
                p->S);
  if (p->tokens == 0 || p->S == 0) return MITA_OK;
  CacheAppendArgs<T> a{};
  auto rows = [&](const void* x, int heads, const int64_t (&given)[2], const char* name,
                  long long& t, long long& h) {
    MITA_TRY(check_ptrs({{x, name}}));
    long long s[2];
    MITA_TRY(row_strides<2>(given, {p->tokens, heads}, sizeof(T), name, s));
    t = s[0];
    h = s[1];
    return (int)MITA_OK;
  };
  if (p->Hq > 0) {
    MITA_TRY(rows(p->q, p->Hq, p->q_strides, "q", a.q_t, a.q_h));
    MITA_TRY(rows(p->q_out, p->Hq, p->q_out_strides, "q_out", a.qo_t, a.qo_h));
  }
  MITA_TRY(rows(p->k, p->Hkv, p->k_strides, "k", a.k_t, a.k_h));
  MITA_TRY(rows(p->v, p->Hkv, p->v_strides, "v", a.v_t, a.v_h));
  if (p->num_pages > 0)
    MITA_TRY(check_ptrs({{p->k_cache, "k_cache"}, {p->v_cache, "v_cache"}}));
  if (p->q_weight) MITA_TRY(check_aligned(p->q_weight, 16, "q_weight"));
  if (p->k_weight) MITA_TRY(check_aligned(p->k_weight, 16, "k_weight"));
  if (p->table_width > 0) MITA_TRY(check_aligned(p->page_table, 4, "page_table"));
  MITA_TRY(check_aligned(p->lengths, 4, "lengths"));
  if (p->seq_start) MITA_TRY(check_aligned(p->seq_start, 4, "seq_start"));
  DevState* ds = nullptr;
  MITA_TRY(device_state_for(st, &ds));
  a.q = static_cast<const T*>(p->q);
  a.k = static_cast<const T*>(p->k);
  a.v = static_cast<const T*>(p->v);
  a.q_out = static_cast<T*>(p->q_out);
  a.k_cache = static_cast<T*>(p->k_cache);
  a.v_cache = static_cast<T*>(p->v_cache);
  a.q_w = p->q_weight; a.k_w = p->k_weight; a.inv_freq = p->inv_freq; a.seq_start = p->seq_start;
  a.paged = {p->page_table, p->lengths, p->S, p->table_width, p->num_pages, log2_of(p->page_size)};
  a.tokens = p->tokens; a.q_heads = p->Hq; a.kv_heads = p->Hkv; a.rot = p->rot;
  a.interleaved = p->interleaved != 0; a.eps = p->eps; a.status = ds->status;
  MITA_CUDA(launch_cache_append<T>(a, p->d, ds->num_sms, st), "cache append launch");
  return MITA_OK;
}

int check_paged_attn(int S, int Hq, int Hkv, int d, int num_pages, int page_size, int width) {
  MITA_TRY(check_pages(S, Hkv, num_pages, page_size, width));
  MITA_TRY(check_head_dim(d));
  if (Hq < 1 || Hq % Hkv != 0)
    return fail(MITA_ERR_INVALID_ARG, "Hq=%d must be a positive multiple of Hkv=%d", Hq, Hkv);
  if ((long long)S * Hq >= (1LL << 31))
    return fail(MITA_ERR_UNSUPPORTED, "S*Hq must be < 2^31");
  if ((long long)Hq * d >= (1LL << 31))
    return fail(MITA_ERR_UNSUPPORTED, "Hq*d must be < 2^31");
  return MITA_OK;
}

// C: what the cache is made of; its check of sizes, its workspace and its launch
template <typename T, typename C, typename Check, typename Bytes, typename Launch>
int paged_attn_any(const mita_paged_attn_params* p, cudaStream_t st, Check check, Bytes ws_bytes,
                   Launch launch) {
  if (p == nullptr) return fail(MITA_ERR_INVALID_ARG, "params is NULL");
  MITA_TRY(check(p->S, p->Hq, p->Hkv, p->d, p->num_pages, p->page_size, p->table_width));
  if (!std::isfinite(p->scale)) return fail(MITA_ERR_INVALID_ARG, "scale is not finite");
  if (!(p->softcap >= 0.f) || std::isinf(p->softcap))
    return fail(MITA_ERR_INVALID_ARG, "softcap must be finite and >= 0");
  if (p->window < 0) return fail(MITA_ERR_INVALID_ARG, "window must be >= 0");
  if (p->S == 0) return MITA_OK;
  MITA_TRY(check_ptrs({{p->q, "q"}, {p->out, "out"}}));
  if (p->num_pages > 0)
    MITA_TRY(check_ptrs({{p->k_cache, "k_cache"}, {p->v_cache, "v_cache"}}));
  if (p->table_width > 0) MITA_TRY(check_aligned(p->page_table, 4, "page_table"));
  MITA_TRY(check_aligned(p->lengths, 4, "lengths"));
  if (p->alibi_slopes) MITA_TRY(check_aligned(p->alibi_slopes, 4, "alibi_slopes"));
  if (p->lse) MITA_TRY(check_aligned(p->lse, 4, "lse"));
  long long qs[2];
  MITA_TRY(row_strides<2>(p->q_strides, {p->S, p->Hq}, sizeof(T), "q", qs));
  const int pl = log2_of(p->page_size), G = p->Hq / p->Hkv;
  MITA_TRY(check_workspace(p->workspace, p->workspace_bytes,
                           ws_bytes(p->d, p->Hkv, G, p->S, p->table_width, pl, sizeof(T) == 4,
                                    current_sms())));
  DevState* ds = nullptr;
  MITA_TRY(device_state_for(st, &ds));
  PagedAttnArgs<T, C> a{};
  a.q = static_cast<const T*>(p->q);
  a.k_cache = static_cast<const C*>(p->k_cache);
  a.v_cache = static_cast<const C*>(p->v_cache);
  a.out = static_cast<T*>(p->out);
  a.lse = p->lse;
  a.slopes = p->alibi_slopes; a.q_s = qs[0]; a.q_h = qs[1];
  a.paged = {p->page_table, p->lengths, p->S, p->table_width, p->num_pages, pl};
  a.Hkv = p->Hkv; a.G = G; a.scale = p->scale; a.softcap = p->softcap; a.window = p->window;
  a.status = ds->status;
  MITA_CUDA(launch(a, p->d, p->workspace, ds->num_sms, st), "paged attention launch");
  return MITA_OK;
}

template <typename T>
int paged_attn_impl(const mita_paged_attn_params* p, cudaStream_t st) {
  return paged_attn_any<T, T>(p, st, check_paged_attn, paged_attn_ws_bytes, launch_paged_attn<T>);
}

// The cache in 4 bits: 32 values a scale, and pages of whole 16-byte pieces of scales.
int check_q4(int d, int page_size) {
  if (d < kQ4Block)
    return fail(MITA_ERR_UNSUPPORTED, "head dim d=%d not in {32, 64, 128} of a 4-bit cache", d);
  if (page_size < kQ4Page)
    return fail(MITA_ERR_UNSUPPORTED, "page_size=%d of a 4-bit cache must be at least %d",
                page_size, kQ4Page);
  return MITA_OK;
}

template <typename T>
int cache_append_q4_impl(const mita_cache_append_q4_params* p, cudaStream_t st) {
  if (p == nullptr) return fail(MITA_ERR_INVALID_ARG, "params is NULL");
  if (p->tokens < 0) return fail(MITA_ERR_INVALID_ARG, "need tokens >= 0 (got %d)", p->tokens);
  MITA_TRY(check_pages(0, p->Hkv, p->num_pages, p->page_size, 0));
  MITA_TRY(check_head_dim(p->d));
  MITA_TRY(check_q4(p->d, p->page_size));
  if (p->Hkv >= (1 << 30) || (long long)p->tokens * 2 * p->Hkv >= (1LL << 31))
    return fail(MITA_ERR_UNSUPPORTED, "tokens*2*Hkv must be < 2^31");
  if (p->tokens == 0) return MITA_OK;
  CacheAppendQ4Args<T> a{};
  auto rows = [&](const void* x, const int64_t (&given)[2], const char* name, long long& t,
                  long long& h) {
    MITA_TRY(check_ptrs({{x, name}}));
    long long s[2];
    MITA_TRY(row_strides<2>(given, {p->tokens, p->Hkv}, sizeof(T), name, s));
    t = s[0];
    h = s[1];
    return (int)MITA_OK;
  };
  MITA_TRY(rows(p->k, p->k_strides, "k", a.k_t, a.k_h));
  MITA_TRY(rows(p->v, p->v_strides, "v", a.v_t, a.v_h));
  if (p->k_out) MITA_TRY(rows(p->k_out, p->k_out_strides, "k_out", a.ko_t, a.ko_h));
  if (p->v_out) MITA_TRY(rows(p->v_out, p->v_out_strides, "v_out", a.vo_t, a.vo_h));
  if (p->num_pages > 0)
    MITA_TRY(check_ptrs({{p->k_cache, "k_cache"}, {p->v_cache, "v_cache"}}));
  MITA_TRY(check_aligned(p->slots, 8, "slots"));
  DevState* ds = nullptr;
  MITA_TRY(device_state_for(st, &ds));
  a.k = static_cast<const T*>(p->k);
  a.v = static_cast<const T*>(p->v);
  a.slots = p->slots;
  a.k_cache = static_cast<uint8_t*>(p->k_cache);
  a.v_cache = static_cast<uint8_t*>(p->v_cache);
  a.k_out = static_cast<T*>(p->k_out);
  a.v_out = static_cast<T*>(p->v_out);
  a.places = (long long)p->num_pages * p->page_size;
  a.tokens = p->tokens; a.kv_heads = p->Hkv; a.page_log2 = log2_of(p->page_size);
  a.status = ds->status;
  MITA_CUDA(launch_cache_append_q4<T>(a, p->d, ds->num_sms, st), "4-bit cache append launch");
  return MITA_OK;
}

int check_paged_attn_q4(int S, int Hq, int Hkv, int d, int num_pages, int page_size, int width) {
  MITA_TRY(check_paged_attn(S, Hq, Hkv, d, num_pages, page_size, width));
  return check_q4(d, page_size);
}

template <typename T>
int paged_attn_q4_impl(const mita_paged_attn_params* p, cudaStream_t st) {
  return paged_attn_any<T, uint8_t>(p, st, check_paged_attn_q4, paged_attn_q4_ws_bytes,
                                    launch_paged_attn_q4<T>);
}

int cache_plan_impl(const mita_cache_plan_params* p, cudaStream_t st) {
  if (p == nullptr) return fail(MITA_ERR_INVALID_ARG, "params is NULL");
  if (p->tokens < 0) return fail(MITA_ERR_INVALID_ARG, "need tokens >= 0 (got %d)", p->tokens);
  MITA_TRY(check_pages(p->S, 1, p->num_pages, p->page_size, p->table_width));
  if (p->tokens > (1 << 30)) return fail(MITA_ERR_UNSUPPORTED, "tokens must be at most 2^30");
  if (p->S > kMaxPlanSequences)
    return fail(MITA_ERR_UNSUPPORTED, "S=%d: a plan takes at most %d sequences", p->S,
                kMaxPlanSequences);
  if (p->S > 0) {
    MITA_TRY(check_aligned(p->new_tokens, 4, "new_tokens"));
    MITA_TRY(check_aligned(p->lengths, 4, "lengths"));
    MITA_TRY(check_aligned(p->new_lengths, 4, "new_lengths"));
    MITA_TRY(check_aligned(p->granted, 4, "granted"));
    if (p->table_width > 0) MITA_TRY(check_aligned(p->page_table, 4, "page_table"));
  }
  if (p->num_pages > 0) MITA_TRY(check_aligned(p->free_pages, 4, "free_pages"));
  MITA_TRY(check_aligned(p->free_count, 4, "free_count"));
  MITA_TRY(check_aligned(p->new_free_count, 4, "new_free_count"));
  MITA_TRY(check_aligned(p->seq_start, 4, "seq_start"));
  if (p->tokens > 0) {
    MITA_TRY(check_aligned(p->positions, 4, "positions"));
    MITA_TRY(check_aligned(p->slots, 8, "slots"));
  }
  DevState* ds = nullptr;
  MITA_TRY(device_state_for(st, &ds));
  CachePlanArgs a{};
  a.new_tokens = p->new_tokens; a.lengths = p->lengths; a.new_lengths = p->new_lengths;
  a.page_table = p->page_table; a.free_pages = p->free_pages; a.free_count = p->free_count;
  a.new_free_count = p->new_free_count; a.seq_start = p->seq_start; a.positions = p->positions;
  a.granted = p->granted; a.slots = p->slots;
  a.S = p->S; a.tokens = p->tokens; a.width = p->table_width; a.num_pages = p->num_pages;
  a.page_log2 = log2_of(p->page_size); a.status = ds->status;
  MITA_CUDA(launch_cache_plan(a, st), "cache plan launch");
  return MITA_OK;
}

// Nothing thrown may leave a C entry point.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return MITA_ERR_OOM;      // the host's allocator is all that can throw here
  }
}

// The forward on host buffers.  The host link, not the GPU, bounds this call (H2D and D2H
// each run at about 200 GB/s on this part, whether a copy engine or the SMs drive them), so
// the heads are split into up to kHostGroups groups that pipeline: a copy stream brings in
// group g + 1's q, k, v while `st` runs group g's forward, and a second copy stream takes
// group g's output back meanwhile (the link is full duplex).  Returns after `st` is
// synchronised.
constexpr int kHostGroups = 4;
struct HostPipe {
  cudaStream_t h2d = nullptr, d2h = nullptr;
  cudaEvent_t ev[2 + 2 * kHostGroups] = {};
  std::mutex mu;   // one host-buffer forward at a time per device uses these
};
std::map<int, HostPipe*> g_pipe;

int host_pipe(HostPipe** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(g_mu);
  HostPipe*& p = g_pipe[dev];
  if (p == nullptr) {
    HostPipe* np = new HostPipe();
    e = cudaStreamCreateWithFlags(&np->h2d, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&np->d2h, cudaStreamNonBlocking);
    for (auto& ev : np->ev)
      if (e == cudaSuccess) e = cudaEventCreateWithFlags(&ev, cudaEventDisableTiming);
    if (e != cudaSuccess) {
      delete np;   // (any stream or event created so far is left to the context's teardown)
      return cuda_fail(e, "copy streams");
    }
    p = np;
  }
  *out = p;
  return MITA_OK;
}

template <typename T>
int forward_host_impl(const T* q, const T* k, const T* v, int B, int H, int N, int d, int gh,
                      int gw, int m, int topk, int s, T* out, cudaStream_t st) {
  MITA_TRY(check_shape(B, H, N, d));
  MITA_TRY(check_m(N, m));
  MITA_TRY(check_grid(N, gh, gw, m));
  MITA_TRY(check_topk(N, topk));
  MITA_TRY(check_s(m, s));
  if (!q || !k || !v || !out) return fail(MITA_ERR_INVALID_ARG, "null host pointer");
  const size_t n = (size_t)B * H * N * d;
  const size_t bytes = align256(n * sizeof(T));
  HostPipe* hp = nullptr;
  MITA_TRY(host_pipe(&hp));
  // Held before the staging buffer is looked up: a call that grows (frees and reallocates)
  // the buffer must not do so while another host-buffer forward is still copying into it.
  std::lock_guard<std::mutex> lk(hp->mu);
  void* sv = nullptr;
  MITA_TRY(staging(4 * bytes, st, &sv));
  char* sb = static_cast<char*>(sv);
  T* dq = reinterpret_cast<T*>(sb);
  T* dk = reinterpret_cast<T*>(sb + bytes);
  T* dv = reinterpret_cast<T*>(sb + 2 * bytes);
  T* dout = reinterpret_cast<T*>(sb + 3 * bytes);
  // On an error return, wait for every copy already queued: they read and write the caller's
  // host buffers, which the caller may free as soon as this call returns.
  struct Drain {
    HostPipe* hp;
    cudaStream_t st;
    bool armed = true;
    ~Drain() {
      if (!armed) return;
      cudaStreamSynchronize(hp->h2d);
      cudaStreamSynchronize(hp->d2h);
      cudaStreamSynchronize(st);
    }
  } drain{hp, st};
  const int BH = B * H;
  const int per = (BH + std::min(BH, kHostGroups) - 1) / std::min(BH, kHostGroups);
  const int G = (BH + per - 1) / per;   // groups of `per` heads (the last may be smaller)
  const size_t head = (size_t)N * d;    // elements per head
  cudaEvent_t ev_start = hp->ev[0], ev_done = hp->ev[1];
  MITA_CUDA(cudaEventRecord(ev_start, st), "event");
  MITA_CUDA(cudaStreamWaitEvent(hp->h2d, ev_start, 0), "event wait");
  MITA_CUDA(cudaStreamWaitEvent(hp->d2h, ev_start, 0), "event wait");
  for (int g = 0; g < G; ++g) {
    const size_t o = (size_t)g * per * head, c = (size_t)std::min(per, BH - g * per) * head;
    MITA_CUDA(cudaMemcpyAsync(dq + o, q + o, c * sizeof(T), cudaMemcpyHostToDevice, hp->h2d),
              "copy of q");
    MITA_CUDA(cudaMemcpyAsync(dk + o, k + o, c * sizeof(T), cudaMemcpyHostToDevice, hp->h2d),
              "copy of k");
    MITA_CUDA(cudaMemcpyAsync(dv + o, v + o, c * sizeof(T), cudaMemcpyHostToDevice, hp->h2d),
              "copy of v");
    MITA_CUDA(cudaEventRecord(hp->ev[2 + g], hp->h2d), "event");
  }
  for (int g = 0; g < G; ++g) {
    const int hg = std::min(per, BH - g * per);
    const size_t o = (size_t)g * per * head, c = (size_t)hg * head;
    MITA_CUDA(cudaStreamWaitEvent(st, hp->ev[2 + g], 0), "event wait");
    // the heads are independent: a group runs as one batch of hg heads
    MITA_TRY(forward_impl<T>(dq + o, dk + o, dv + o, 1, hg, N, d, gh, gw, m, topk, s, dout + o,
                             st));
    MITA_CUDA(cudaEventRecord(hp->ev[2 + kHostGroups + g], st), "event");
    MITA_CUDA(cudaStreamWaitEvent(hp->d2h, hp->ev[2 + kHostGroups + g], 0), "event wait");
    MITA_CUDA(cudaMemcpyAsync(out + o, dout + o, c * sizeof(T), cudaMemcpyDeviceToHost, hp->d2h),
              "copy of out");
  }
  MITA_CUDA(cudaEventRecord(ev_done, hp->d2h), "event");
  MITA_CUDA(cudaStreamWaitEvent(st, ev_done, 0), "event wait");
  MITA_CUDA(cudaStreamSynchronize(st), "synchronisation");
  drain.armed = false;   // every stream is idle: st waited for the last copy out
  return MITA_OK;
}

}  // namespace

int report_error(int code, const char* text) { return fail(code, "%s", text); }

}  // namespace mita

using mita::bf16;

namespace mita {
std::atomic<unsigned long long> g_launches{0};
void count_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }
}  // namespace mita

extern "C" {

int mita_pool(const void* q, int B, int H, int N, int d, int grid_h, int grid_w, int m,
              void* q_tilde, mita_stream_t stream) {
  return mita::pool_impl<bf16>(static_cast<const bf16*>(q), B, H, N, d, grid_h, grid_w, m,
                               static_cast<bf16*>(q_tilde), stream);
}
int mita_pool_grid(const void* q, int B, int H, int N, int d, int grid_h, int grid_w,
                   int landmark_grid_h, int landmark_grid_w, void* q_tilde, mita_stream_t stream) {
  return mita::pool_impl<bf16>(static_cast<const bf16*>(q), B, H, N, d, grid_h, grid_w,
                               landmark_grid_h * landmark_grid_w, static_cast<bf16*>(q_tilde),
                               stream, landmark_grid_h, landmark_grid_w);
}
int mita_pool_grid_f32(const float* q, int B, int H, int N, int d, int grid_h, int grid_w,
                       int landmark_grid_h, int landmark_grid_w, float* q_tilde,
                       mita_stream_t stream) {
  return mita::pool_impl<float>(q, B, H, N, d, grid_h, grid_w, landmark_grid_h * landmark_grid_w,
                                q_tilde, stream, landmark_grid_h, landmark_grid_w);
}
int mita_pool_f32(const float* q, int B, int H, int N, int d, int grid_h, int grid_w, int m,
                  float* q_tilde, mita_stream_t stream) {
  return mita::pool_impl<float>(q, B, H, N, d, grid_h, grid_w, m, q_tilde, stream);
}

int mita_landmark_topk_shared(const void* q_tilde, const void* k, const void* v, int B, int H,
                              int N, int d, int m, int topk, int32_t* topk_idx, float* v_tilde,
                              mita_stream_t stream) {
  return mita::landmark_impl<bf16>(static_cast<const bf16*>(q_tilde),
                                   static_cast<const bf16*>(k), static_cast<const bf16*>(v), B,
                                   H, N, d, m, topk, topk_idx, v_tilde, stream);
}
int mita_landmark_topk_shared_f32(const float* q_tilde, const float* k, const float* v, int B,
                                  int H, int N, int d, int m, int topk, int32_t* topk_idx,
                                  float* v_tilde, mita_stream_t stream) {
  return mita::landmark_impl<float>(q_tilde, k, v, B, H, N, d, m, topk, topk_idx, v_tilde,
                                    stream);
}

int mita_route(const void* q, const void* q_tilde, const float* v_tilde, int B, int H, int N,
               int d, int m, int s, int32_t* route_idx, float* shared_lse, float* shared_o,
               mita_stream_t stream) {
  return mita::route_impl<bf16>(static_cast<const bf16*>(q), static_cast<const bf16*>(q_tilde),
                                v_tilde, B, H, N, d, m, s, route_idx, shared_lse, shared_o,
                                stream);
}
int mita_route_f32(const float* q, const float* q_tilde, const float* v_tilde, int B, int H,
                   int N, int d, int m, int s, int32_t* route_idx, float* shared_lse,
                   float* shared_o, mita_stream_t stream) {
  return mita::route_impl<float>(q, q_tilde, v_tilde, B, H, N, d, m, s, route_idx, shared_lse,
                                 shared_o, stream);
}

int mita_bucket(const int32_t* route_idx, int B, int H, int N, int m, int s,
                int32_t* bucket_off, int32_t* bucket_qidx, mita_stream_t stream) {
  return mita::bucket_impl(route_idx, B, H, N, m, s, bucket_off, bucket_qidx, stream);
}

int mita_expert_attn(const void* q, const void* k, const void* v, const void* q_tilde,
                     const float* v_tilde, const int32_t* topk_idx, const int32_t* bucket_off,
                     const int32_t* bucket_qidx, const float* shared_lse, const float* shared_o,
                     int B, int H, int N, int d, int m, int topk, int s, void* out,
                     mita_stream_t stream) {
  return mita::expert_impl<bf16>(
      static_cast<const bf16*>(q), static_cast<const bf16*>(k), static_cast<const bf16*>(v),
      static_cast<const bf16*>(q_tilde), v_tilde, topk_idx, bucket_off, bucket_qidx, shared_lse,
      shared_o, B, H, N, d, m, topk, s, static_cast<bf16*>(out), stream);
}
int mita_expert_attn_f32(const float* q, const float* k, const float* v, const float* q_tilde,
                         const float* v_tilde, const int32_t* topk_idx,
                         const int32_t* bucket_off, const int32_t* bucket_qidx,
                         const float* shared_lse, const float* shared_o, int B, int H, int N,
                         int d, int m, int topk, int s, float* out, mita_stream_t stream) {
  return mita::expert_impl<float>(q, k, v, q_tilde, v_tilde, topk_idx, bucket_off, bucket_qidx,
                                  shared_lse, shared_o, B, H, N, d, m, topk, s, out, stream);
}

int mita_forward(const void* q, const void* k, const void* v, int B, int H, int N, int d,
                 int grid_h, int grid_w, int m, int topk, int s, void* out,
                 mita_stream_t stream) {
  return mita::forward_impl<bf16>(static_cast<const bf16*>(q), static_cast<const bf16*>(k),
                                  static_cast<const bf16*>(v), B, H, N, d, grid_h, grid_w, m,
                                  topk, s, static_cast<bf16*>(out), stream);
}
int mita_forward_f32(const float* q, const float* k, const float* v, int B, int H, int N, int d,
                     int grid_h, int grid_w, int m, int topk, int s, float* out,
                     mita_stream_t stream) {
  return mita::forward_impl<float>(q, k, v, B, H, N, d, grid_h, grid_w, m, topk, s, out, stream);
}

int mita_forward_ex(const void* q, const void* k, const void* v, int B, int H, int N, int d,
                    int grid_h, int grid_w, int m, int topk, int s, const mita_options* options,
                    void* out, mita_stream_t stream) {
  return mita::forward_impl<bf16>(static_cast<const bf16*>(q), static_cast<const bf16*>(k),
                                  static_cast<const bf16*>(v), B, H, N, d, grid_h, grid_w, m, topk,
                                  s, static_cast<bf16*>(out), stream, options);
}
int mita_forward_ex_f32(const float* q, const float* k, const float* v, int B, int H, int N,
                        int d, int grid_h, int grid_w, int m, int topk, int s,
                        const mita_options* options, float* out, mita_stream_t stream) {
  return mita::forward_impl<float>(q, k, v, B, H, N, d, grid_h, grid_w, m, topk, s, out, stream,
                                   options);
}

int mita_dense_attn(const void* q, const void* k, const void* v, int B, int H, int N, int d,
                    void* out, mita_stream_t stream) {
  return mita::dense_impl<bf16>(static_cast<const bf16*>(q), static_cast<const bf16*>(k),
                                static_cast<const bf16*>(v), B, H, N, d, static_cast<bf16*>(out),
                                stream);
}
int mita_dense_attn_f32(const float* q, const float* k, const float* v, int B, int H, int N,
                        int d, float* out, mita_stream_t stream) {
  return mita::dense_impl<float>(q, k, v, B, H, N, d, out, stream);
}

int mita_backward(const void* q, const void* k, const void* v, const void* dout, int B, int H,
                  int N, int d, int grid_h, int grid_w, int m, int topk, int s,
                  const mita_options* options, float* dq, float* dk, float* dv,
                  mita_stream_t stream) {
  return mita::backward_impl<bf16>(static_cast<const bf16*>(q), static_cast<const bf16*>(k),
                                   static_cast<const bf16*>(v), static_cast<const bf16*>(dout), B,
                                   H, N, d, grid_h, grid_w, m, topk, s, options, dq, dk, dv,
                                   stream);
}
int mita_backward_f32(const float* q, const float* k, const float* v, const float* dout, int B,
                      int H, int N, int d, int grid_h, int grid_w, int m, int topk, int s,
                      const mita_options* options, float* dq, float* dk, float* dv,
                      mita_stream_t stream) {
  return mita::backward_impl<float>(q, k, v, dout, B, H, N, d, grid_h, grid_w, m, topk, s,
                                    options, dq, dk, dv, stream);
}

int mita_forward_host(const void* q, const void* k, const void* v, int B, int H, int N, int d,
                      int grid_h, int grid_w, int m, int topk, int s, void* out,
                      mita_stream_t stream) {
  return mita::forward_host_impl<bf16>(static_cast<const bf16*>(q), static_cast<const bf16*>(k),
                                       static_cast<const bf16*>(v), B, H, N, d, grid_h, grid_w,
                                       m, topk, s, static_cast<bf16*>(out), stream);
}
int mita_forward_host_f32(const float* q, const float* k, const float* v, int B, int H, int N,
                          int d, int grid_h, int grid_w, int m, int topk, int s, float* out,
                          mita_stream_t stream) {
  return mita::forward_host_impl<float>(q, k, v, B, H, N, d, grid_h, grid_w, m, topk, s, out,
                                        stream);
}

int mita_qk_norm_rope(const mita_qk_norm_rope_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::norm_rope_impl<bf16>(params, stream); });
}
int mita_qk_norm_rope_f32(const mita_qk_norm_rope_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::norm_rope_impl<float>(params, stream); });
}

int mita_qk_norm_rope_backward(const mita_qk_norm_rope_backward_params* params,
                               mita_stream_t stream) {
  return mita::guarded([&] { return mita::norm_rope_backward_impl<bf16>(params, stream); });
}
int mita_qk_norm_rope_backward_f32(const mita_qk_norm_rope_backward_params* params,
                                   mita_stream_t stream) {
  return mita::guarded([&] { return mita::norm_rope_backward_impl<float>(params, stream); });
}
uint64_t mita_qk_norm_rope_backward_workspace_bytes(int d) {
  if (d != 16 && d != 32 && d != 64 && d != 128) return 0;
  return mita::norm_rope_backward_ws(d, mita::current_sms());
}

int mita_qk_norm_rope_axes(const mita_qk_norm_rope_axes_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::norm_rope_impl<bf16>(params, stream); });
}
int mita_qk_norm_rope_axes_f32(const mita_qk_norm_rope_axes_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::norm_rope_impl<float>(params, stream); });
}

int mita_qk_norm_rope_axes_backward(const mita_qk_norm_rope_axes_backward_params* params,
                                    mita_stream_t stream) {
  return mita::guarded([&] { return mita::norm_rope_backward_impl<bf16>(params, stream); });
}
int mita_qk_norm_rope_axes_backward_f32(const mita_qk_norm_rope_axes_backward_params* params,
                                        mita_stream_t stream) {
  return mita::guarded([&] { return mita::norm_rope_backward_impl<float>(params, stream); });
}

int mita_cache_append(const mita_cache_append_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::cache_append_impl<bf16>(params, stream); });
}
int mita_cache_append_f32(const mita_cache_append_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::cache_append_impl<float>(params, stream); });
}

int mita_paged_attn(const mita_paged_attn_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::paged_attn_impl<bf16>(params, stream); });
}
int mita_paged_attn_f32(const mita_paged_attn_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::paged_attn_impl<float>(params, stream); });
}
uint64_t mita_paged_attn_workspace_bytes(int S, int Hq, int Hkv, int d, int page_size,
                                         int table_width, int is_f32) {
  if (mita::guarded([&] {
        return mita::check_paged_attn(S, Hq, Hkv, d, 0, page_size, table_width);
      }) != MITA_OK)
    return 0;
  return mita::paged_attn_ws_bytes(d, Hkv, Hq / Hkv, S, table_width, mita::log2_of(page_size),
                                   is_f32, mita::current_sms());
}

int mita_paged_attn_q4(const mita_paged_attn_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::paged_attn_q4_impl<bf16>(params, stream); });
}
int mita_paged_attn_q4_f32(const mita_paged_attn_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::paged_attn_q4_impl<float>(params, stream); });
}
uint64_t mita_paged_attn_q4_workspace_bytes(int S, int Hq, int Hkv, int d, int page_size,
                                            int table_width, int is_f32) {
  if (mita::guarded([&] {
        return mita::check_paged_attn_q4(S, Hq, Hkv, d, 0, page_size, table_width);
      }) != MITA_OK)
    return 0;
  return mita::paged_attn_q4_ws_bytes(d, Hkv, Hq / Hkv, S, table_width, mita::log2_of(page_size),
                                      is_f32, mita::current_sms());
}

int mita_cache_append_q4(const mita_cache_append_q4_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::cache_append_q4_impl<bf16>(params, stream); });
}
int mita_cache_append_q4_f32(const mita_cache_append_q4_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::cache_append_q4_impl<float>(params, stream); });
}

int mita_cache_plan(const mita_cache_plan_params* params, mita_stream_t stream) {
  return mita::guarded([&] { return mita::cache_plan_impl(params, stream); });
}

uint64_t mita_forward_workspace_bytes(int B, int H, int N, int d, int m, int topk, int s,
                                      int is_f32) {
  if (mita::check_shape(B, H, N, d) || mita::check_m(N, m) || mita::check_topk(N, topk) ||
      mita::check_s(m, s) || mita::check_entries(B, H, N, s))
    return 0;
  int sms = 152;
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaGetLastError();
  return mita::forward_layout(B * H, N, d, m, topk, s, is_f32 ? 4 : 2, sms).total;
}

const char* mita_status_string(int status) {
  switch (status) {
    case MITA_OK: return "ok";
    case MITA_ERR_INVALID_ARG: return "invalid argument";
    case MITA_ERR_UNSUPPORTED: return "unsupported by this build";
    case MITA_ERR_CUDA: return "CUDA error";
    case MITA_ERR_OOM: return "out of device memory";
    case MITA_ERR_DEVICE_CHECK: return "a kernel flagged inconsistent input data";
    default: return "unknown status";
  }
}

const char* mita_last_error_message(void) { return mita::g_msg.c_str(); }

int mita_get_last_device_error(mita_stream_t stream, int* bits) {
  if (bits) *bits = 0;
  mita::DevState* ds = nullptr;
  int rc = mita::device_state(&ds);
  if (rc != MITA_OK) return rc;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return mita::cuda_fail(e, "cudaStreamSynchronize");
  int v = 0;
  e = cudaMemcpy(&v, ds->status, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return mita::cuda_fail(e, "cudaMemcpy");
  e = cudaMemset(ds->status, 0, sizeof(int));
  if (e != cudaSuccess) return mita::cuda_fail(e, "cudaMemset");
  if (bits) *bits = v;
  return v ? mita::fail(MITA_ERR_DEVICE_CHECK, "device status bits 0x%x", v) : MITA_OK;
}

uint64_t mita_kernel_launches(void) { return mita::g_launches.load(std::memory_order_relaxed); }

int mita_check_bounded_wait(int* gave_up, mita_stream_t stream) {
  if (!gave_up) return mita::fail(MITA_ERR_INVALID_ARG, "mita_check_bounded_wait: NULL gave_up");
  mita::DevState* ds = nullptr;
  int rc = mita::device_state(&ds);
  if (rc != MITA_OK) return rc;
  const cudaError_t e = mita::launch_bounded_wait_probe(ds->status, gave_up, stream);
  return e == cudaSuccess ? MITA_OK : mita::cuda_fail(e, "mita_check_bounded_wait launch");
}

uint64_t mita_workspace_set_limit(uint64_t bytes) {
  return mita::g_ws_limit.exchange(bytes);
}

int mita_workspace_release(void) {
  std::lock_guard<std::mutex> lk(mita::g_mu);
  int prev = 0;
  cudaGetDevice(&prev);
  for (auto* cache : {&mita::g_ws, &mita::g_stage}) {
    for (auto& kv : *cache) {
      if (kv.second.ptr) {
        cudaSetDevice(kv.first.first);
        cudaDeviceSynchronize();
        cudaFree(kv.second.ptr);
      }
    }
    cache->clear();
  }
  cudaSetDevice(prev);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MITA_OK : mita::cuda_fail(e, "workspace release");
}

}  // extern "C"
