// Gradient norms, clipping and AdamW over packed tensors: the gfx950 kernels and the host
// side of psgd_clip.h.
//
// A tile is at most kTile consecutive elements of one tensor.  Sums of squares are held in
// float64; every reduction has a fixed order.
//
//   cl_norm    per (tile, slice): the tile's sum of squares, or its largest magnitude
//   cl_final   per slice: the tensors' and the slice's norm, the clip coefficient, and for
//              AdamW the step count and the step's scalars
//   cl_scale   per (tile, slice): out = c * g
//   cl_adamw   per tile: the weight update

#include <hip/hip_runtime.h>
#include <hip/hip_ext.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <map>
#include <new>
#include <string>
#include <vector>

#include "plan.hpp"
#include "psgd_clip.h"

namespace psgd {
namespace clip {

constexpr int kTile = 16384;  // elements per tile
constexpr int kThreads = 256;
constexpr int kFinalThreads = 1024;

struct ClTile {
  int64_t begin;   // element offset of the tile in a slice
  int32_t len;     // elements in the tile (kTile except at a tensor's end)
  int32_t matrix;  // 1: the tensor has more than one row and more than one column
};

struct ClLayer {
  int32_t tile0, ntiles;  // the tensor's tiles
};

// The AdamW step's scalars, written by cl_final for cl_adamw.
struct AwState {
  float coef;
  float step_size;  // lr / (1 - beta1^t)
  float inv_sqrt;   // 1 / sqrt(1 - beta2^t)
  int32_t skip;
};

struct AwArgs {
  double lr, beta1, beta2;
  int64_t* step;  // NULL: not an AdamW call
  AwState* state;
  int32_t have_norm;  // 0: no norm was taken, c = 1
  int32_t skip_nonfinite;
};

enum KernelId { kNorm = 0, kFinal, kScale, kAdamw, kNumK };
const char* const kNames[kNumK] = {"cl_norm", "cl_final", "cl_scale", "cl_adamw"};

}  // namespace clip
}  // namespace psgd

struct psgd_clip_plan {
  int32_t n_slices = 0;
  psgd_dtype dtype = PSGD_F32;
  std::vector<psgd_clip_layer_info> info;
  std::vector<psgd::clip::ClLayer> layers;
  std::vector<psgd::clip::ClTile> tiles;
  int64_t worker_stride = 0, numel = 0;
  uint64_t ws_part = 0, ws_tensor = 0, ws_coef = 0, ws_aw = 0, workspace_bytes = 0;
  std::map<int, void*> dev;  // device copy of the layer and tile tables, per HIP device
  bool timing = false;
  std::vector<psgd::PendingTiming> pending;
  std::vector<hipEvent_t> event_pool;
  psgd::KernelStat stats[psgd::clip::kNumK];
};

namespace psgd {
namespace clip {
namespace {

// ------------------------------------------------------------------ device helpers
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4f load4(const float* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const v4f*>(p));
}

// Four bfloat16 values widened exactly to float32.
__device__ __forceinline__ v4f load4(const uint16_t* p) {
  const v2u u = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(p));
  v4f r;
  r.x = __uint_as_float(u.x << 16);
  r.y = __uint_as_float(u.x & 0xffff0000u);
  r.z = __uint_as_float(u.y << 16);
  r.w = __uint_as_float(u.y & 0xffff0000u);
  return r;
}

__device__ __forceinline__ void store4(float* p, v4f v) {
  __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(p));
}

// Rounded to nearest even (the hardware conversion; NaN stays NaN).
__device__ __forceinline__ void store4(uint16_t* p, v4f v) {
  const v2u u = __builtin_bit_cast(v2u, __builtin_convertvector(v, v4b));
  __builtin_nontemporal_store(u, reinterpret_cast<v2u*>(p));
}

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) {
  *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// The first n (1..4) elements of a unit; the rest is padding or another tensor's.
template <typename T>
__device__ __forceinline__ void store_upto(T* p, v4f v, int n) {
  if (n >= 4) {
    store4(p, v);
    return;
  }
  for (int j = 0; j < n; ++j) store1(p + j, v[j]);
}

// Partial norms.  L2: a float64 sum of squares.  MAX: the largest magnitude as its bit
// pattern, whose unsigned order is that of magnitudes with NaN above infinity, so a NaN
// is carried to the result.
struct L2 {
  typedef double acc_t;
  static __device__ __forceinline__ double zero() { return 0.0; }
  static __device__ __forceinline__ void take(double& a, float x) { a = fma(double(x), double(x), a); }
  static __device__ __forceinline__ double join(double a, double b) { return a + b; }
  static __device__ __forceinline__ double norm(double a) { return sqrt(a); }
};

struct Max {
  typedef uint32_t acc_t;
  static __device__ __forceinline__ uint32_t zero() { return 0u; }
  static __device__ __forceinline__ void take(uint32_t& a, float x) { a = max(a, __float_as_uint(x) & 0x7fffffffu); }
  static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ double norm(uint32_t a) { return double(__uint_as_float(a)); }
};

template <typename N>
__device__ __forceinline__ typename N::acc_t wave_join(typename N::acc_t a) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) a = N::join(a, __shfl_xor(a, d));
  return a;
}

// Every thread gets the joined value of the block; `lds` holds one value per wave.
template <typename N>
__device__ __forceinline__ typename N::acc_t block_join(typename N::acc_t a, typename N::acc_t* lds) {
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, nw = blockDim.x >> 6;
  a = wave_join<N>(a);
  if (lane == 0) lds[wid] = a;
  __syncthreads();
  a = lds[0];
  for (int i = 1; i < nw; ++i) a = N::join(a, lds[i]);
  __syncthreads();
  return a;
}

// c = 1 if norm <= max_norm, else max_norm / norm; NaN for a NaN norm.
__device__ __forceinline__ float clip_coef(double norm, double max_norm) {
  return norm <= max_norm ? 1.0f : float(max_norm / norm);
}

// ------------------------------------------------------------------ kernels
template <typename GT, typename N>
__global__ __launch_bounds__(kThreads) void cl_norm(const ClTile* __restrict__ tiles, const GT* __restrict__ grads,
                                                    typename N::acc_t* __restrict__ part, int64_t stride) {
  __shared__ typename N::acc_t lds[kThreads / 64];
  const ClTile t = tiles[blockIdx.x];
  const GT* g = grads + int64_t(blockIdx.y) * stride + t.begin;
  typename N::acc_t acc = N::zero();
#pragma unroll 4
  for (int e = int(threadIdx.x) * 4; e < t.len; e += kThreads * 4) {
    const v4f v = load4(g + e);  // a tensor's padding reaches the next multiple of 64 elements
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e + j < t.len) N::take(acc, v[j]);
  }
  acc = block_join<N>(acc, lds);
  if (threadIdx.x == 0) part[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = acc;
}

template <typename N>
__global__ __launch_bounds__(kFinalThreads) void cl_final(const ClLayer* __restrict__ layers, int n_layers, int n_tiles,
                                                          const typename N::acc_t* __restrict__ part,
                                                          double max_norm, float* __restrict__ norms,
                                                          float* __restrict__ tensor_norms, float* __restrict__ coefs,
                                                          float* __restrict__ ws_coef, AwArgs aw) {
  __shared__ typename N::acc_t lds[kFinalThreads / 64];
  const int slice = blockIdx.x;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  double norm = 0.0;
  float c = 1.0f;
  if (aw.step == nullptr || aw.have_norm) {
    typename N::acc_t acc = N::zero();
    for (int l = wid; l < n_layers; l += kFinalThreads / 64) {
      const ClLayer L = layers[l];
      const typename N::acc_t* p = part + int64_t(slice) * n_tiles + L.tile0;
      typename N::acc_t a = N::zero();
      for (int i = lane; i < L.ntiles; i += 64) a = N::join(a, p[i]);
      a = wave_join<N>(a);
      if (lane == 0) {
        if (tensor_norms != nullptr) tensor_norms[int64_t(slice) * n_layers + l] = float(N::norm(a));
        acc = N::join(acc, a);
      }
    }
    acc = block_join<N>(acc, lds);
    norm = N::norm(acc);
    c = clip_coef(norm, max_norm);
  }
  if (threadIdx.x != 0) return;
  if (norms != nullptr) norms[slice] = float(norm);
  if (coefs != nullptr) coefs[slice] = c;
  ws_coef[slice] = c;
  if (aw.step != nullptr) {
    AwState s;
    s.coef = c;
    s.skip = aw.skip_nonfinite && !isfinite(float(norm)) ? 1 : 0;
    const int64_t t = *aw.step + 1;
    s.step_size = float(aw.lr / (1.0 - pow(aw.beta1, double(t))));
    s.inv_sqrt = float(1.0 / sqrt(1.0 - pow(aw.beta2, double(t))));
    *aw.state = s;
    if (!s.skip) *aw.step = t;
  }
}

template <typename GT>
__global__ __launch_bounds__(kThreads) void cl_scale(const ClTile* __restrict__ tiles, const GT* grads, GT* out,
                                                     const float* __restrict__ ws_coef, int64_t stride) {
  const float c = ws_coef[blockIdx.y];
  if (c == 1.0f && grads == out) return;
  const ClTile t = tiles[blockIdx.x];
  const int64_t base = int64_t(blockIdx.y) * stride + t.begin;
#pragma unroll 4
  for (int e = int(threadIdx.x) * 4; e < t.len; e += kThreads * 4)
    store_upto(out + base + e, load4(grads + base + e) * c, t.len - e);
}

template <typename GT>
__global__ __launch_bounds__(kThreads) void cl_adamw(const ClTile* __restrict__ tiles, const GT* __restrict__ update,
                                                     float* __restrict__ params, float* __restrict__ exp_avg,
                                                     float* __restrict__ exp_avg_sq, uint16_t* __restrict__ copy,
                                                     const AwState* __restrict__ state, float beta1, float om_beta1,
                                                     float beta2, float om_beta2, float eps, float decay,
                                                     int matrices_only) {
  const AwState s = *state;
  if (s.skip) return;
  const ClTile t = tiles[blockIdx.x];
  const float d = matrices_only && !t.matrix ? 0.0f : decay;
  for (int e = int(threadIdx.x) * 4; e < t.len; e += kThreads * 4) {
    const int64_t at = t.begin + e;
    const v4f g = load4(update + at) * s.coef;
    v4f x = load4(params + at), m = load4(exp_avg + at), v = load4(exp_avg_sq + at);
    m = beta1 * m + om_beta1 * g;
    v = beta2 * v + om_beta2 * (g * g);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float den = sqrtf(v[j]) * s.inv_sqrt + eps;
      x[j] = fmaf(-d, x[j], x[j]) - s.step_size * (m[j] / den);
    }
    const int n = t.len - e;
    store_upto(params + at, x, n);
    store_upto(exp_avg + at, m, n);
    store_upto(exp_avg_sq + at, v, n);
    if (copy != nullptr) store_upto(copy + at, x, n);
  }
}

// ------------------------------------------------------------------ host helpers
psgd_status fail(psgd_status s, const std::string& msg) {
  set_error(msg);
  return s;
}

psgd_status hip_fail(const char* what, hipError_t e) {
  return fail(PSGD_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

// What an exception thrown inside an entry point becomes (the message fits without an
// allocation).
psgd_status no_memory() {
  set_error("out of memory");
  return PSGD_ERR_NO_MEMORY;
}

uint64_t a256(uint64_t x) { return (x + 255) / 256 * 256; }

struct DevTables {
  const ClLayer* layers;
  const ClTile* tiles;
};

psgd_status device_tables(const char* fn, psgd_clip_plan* plan, hipStream_t st, DevTables* out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail("hipGetDevice", e);
  const uint64_t bl = a256(plan->layers.size() * sizeof(ClLayer));
  const uint64_t bt = a256(plan->tiles.size() * sizeof(ClTile));
  auto it = plan->dev.find(dev);
  if (it == plan->dev.end()) {
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    e = hipStreamIsCapturing(st, &cs);
    if (e != hipSuccess) return hip_fail("hipStreamIsCapturing", e);
    if (cs != hipStreamCaptureStatusNone)
      return fail(PSGD_ERR_INVALID_ARG, std::string(fn) + ": a plan can be captured into a graph only after an eager "
                                            "call of the plan on this device");
    it = plan->dev.emplace(dev, nullptr).first;
    void* base = nullptr;
    e = hipMalloc(&base, bl + bt);
    if (e != hipSuccess) {
      plan->dev.erase(it);
      return fail(PSGD_ERR_NO_MEMORY, std::string("hipMalloc of the plan's device tables: ") + hipGetErrorString(e));
    }
    char* b = static_cast<char*>(base);
    e = hipMemcpy(b, plan->layers.data(), plan->layers.size() * sizeof(ClLayer), hipMemcpyHostToDevice);
    if (e == hipSuccess)
      e = hipMemcpy(b + bl, plan->tiles.data(), plan->tiles.size() * sizeof(ClTile), hipMemcpyHostToDevice);
    if (e != hipSuccess) {
      (void)hipFree(base);
      plan->dev.erase(it);
      return hip_fail("hipMemcpy of the plan's device tables", e);
    }
    it->second = base;
  }
  char* b = static_cast<char*>(it->second);
  out->layers = reinterpret_cast<const ClLayer*>(b);
  out->tiles = reinterpret_cast<const ClTile*>(b + bl);
  return PSGD_OK;
}

psgd_status take_event(psgd_clip_plan* plan, hipEvent_t* ev) {
  if (!plan->event_pool.empty()) {
    *ev = plan->event_pool.back();
    plan->event_pool.pop_back();
    return PSGD_OK;
  }
  const hipError_t e = hipEventCreate(ev);
  return e == hipSuccess ? PSGD_OK : hip_fail("hipEventCreate", e);
}

// Launch on `st`; with timing on, through hipExtLaunchKernelGGL with events the runtime
// records with the dispatch itself.
template <typename... KArgs, typename... Args>
psgd_status launch(psgd_clip_plan* plan, int kid, void (*kernel)(KArgs...), dim3 grid, dim3 block, hipStream_t st,
                   Args... args) {
  hipEvent_t a = nullptr, b = nullptr;
  if (plan->timing) {
    plan->pending.reserve(plan->pending.size() + 1);
    plan->event_pool.reserve(plan->event_pool.size() + 2);
    psgd_status s = take_event(plan, &a);
    if (s == PSGD_OK) s = take_event(plan, &b);
    if (s != PSGD_OK) {
      if (a) plan->event_pool.push_back(a);
      return s;
    }
    hipExtLaunchKernelGGL(kernel, grid, block, 0, st, a, b, 0, args...);
  } else {
    hipLaunchKernelGGL(kernel, grid, block, 0, st, args...);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) {
    if (plan->timing) {
      plan->event_pool.push_back(a);
      plan->event_pool.push_back(b);
    }
    return hip_fail((std::string("launch ") + kNames[kid]).c_str(), e);
  }
  if (plan->timing) plan->pending.push_back(PendingTiming{kid, a, b});
  return PSGD_OK;
}

struct Span {
  const char* name;
  const void* ptr;
  uint64_t bytes;
  unsigned align;
  bool nullable;
};

// Every pointer given, aligned, and no two ranges overlapping; `same` names the one pair
// (by index) that may be the same buffer.
psgd_status check_spans(const char* fn, const Span* spans, int n, int same_a = -1, int same_b = -1) {
  for (int i = 0; i < n; ++i) {
    const Span& a = spans[i];
    if (a.ptr == nullptr) {
      if (a.nullable) continue;
      return fail(PSGD_ERR_INVALID_ARG, std::string(fn) + ": " + a.name + " is NULL");
    }
    if (uintptr_t(a.ptr) % a.align != 0)
      return fail(PSGD_ERR_INVALID_ARG, std::string(fn) + ": " + a.name + " is not " + std::to_string(a.align) +
                                            "-byte aligned");
  }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      const Span &a = spans[i], &b = spans[j];
      if (a.ptr == nullptr || b.ptr == nullptr) continue;
      if (i == same_a && j == same_b && a.ptr == b.ptr) continue;
      const uintptr_t al = uintptr_t(a.ptr), bl = uintptr_t(b.ptr);
      if (al < bl + b.bytes && bl < al + a.bytes)
        return fail(PSGD_ERR_INVALID_ARG, std::string(fn) + ": " + a.name + " and " + b.name + " overlap");
    }
  return PSGD_OK;
}

psgd_status check_kind(const char* fn, int kind) {
  if (kind == PSGD_NORM_L2 || kind == PSGD_NORM_MAX) return PSGD_OK;
  return fail(PSGD_ERR_UNSUPPORTED, std::string(fn) + ": unknown norm kind");
}

// The norm of every slice, and what cl_final derives from it.
template <typename N>
psgd_status enqueue_norm(psgd_clip_plan* plan, const DevTables& dt, const void* grads, double max_norm, float* norms,
                         float* tensor_norms, float* coefs, char* ws, const AwArgs& aw, hipStream_t st) {
  typedef typename N::acc_t acc_t;
  acc_t* part = reinterpret_cast<acc_t*>(ws + plan->ws_part);
  const int n_tiles = int(plan->tiles.size());
  const dim3 grid(static_cast<unsigned>(n_tiles), static_cast<unsigned>(plan->n_slices));
  psgd_status s = PSGD_OK;
  if (aw.step == nullptr || aw.have_norm) {
    if (plan->dtype == PSGD_BF16)
      s = launch(plan, kNorm, cl_norm<uint16_t, N>, grid, dim3(kThreads), st, dt.tiles,
                 static_cast<const uint16_t*>(grads), part, plan->worker_stride);
    else
      s = launch(plan, kNorm, cl_norm<float, N>, grid, dim3(kThreads), st, dt.tiles, static_cast<const float*>(grads),
                 part, plan->worker_stride);
    if (s != PSGD_OK) return s;
  }
  return launch(plan, kFinal, cl_final<N>, dim3(static_cast<unsigned>(plan->n_slices)), dim3(kFinalThreads), st,
                dt.layers, int(plan->layers.size()), n_tiles, static_cast<const acc_t*>(part), max_norm, norms,
                tensor_norms, coefs, reinterpret_cast<float*>(ws + plan->ws_coef), aw);
}

psgd_status enqueue_norm(psgd_clip_plan* plan, int kind, const DevTables& dt, const void* grads, double max_norm,
                         float* norms, float* tensor_norms, float* coefs, char* ws, const AwArgs& aw, hipStream_t st) {
  if (kind == PSGD_NORM_MAX)
    return enqueue_norm<Max>(plan, dt, grads, max_norm, norms, tensor_norms, coefs, ws, aw, st);
  return enqueue_norm<L2>(plan, dt, grads, max_norm, norms, tensor_norms, coefs, ws, aw, st);
}

}  // namespace
}  // namespace clip
}  // namespace psgd

using namespace psgd;
using namespace psgd::clip;

extern "C" psgd_status psgd_clip_plan_create(const psgd_layer* layers, int32_t n_layers, int32_t n_slices,
                                             psgd_dtype grad_dtype, uint32_t flags, psgd_clip_plan** out) {
  if (out == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: out is NULL");
  *out = nullptr;
  if (layers == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: layers is NULL");
  if (n_layers < 1) return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: n_layers must be >= 1");
  if (n_slices < 1 || n_slices > 65535)
    return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: n_slices must be in 1..65535");
  if (grad_dtype != PSGD_F32 && grad_dtype != PSGD_BF16)
    return fail(PSGD_ERR_UNSUPPORTED, "psgd_clip_plan_create: unknown grad_dtype");
  if (flags != 0) return fail(PSGD_ERR_UNSUPPORTED, "psgd_clip_plan_create: unknown flag bits");
  psgd_clip_plan* plan = nullptr;
  try {
    plan = new psgd_clip_plan();
    plan->n_slices = n_slices;
    plan->dtype = grad_dtype;
    int64_t off = 0;
    for (int32_t i = 0; i < n_layers; ++i) {
      const int64_t rows = layers[i].rows, cols = layers[i].cols;
      if (rows < 1 || cols < 1 || rows > int64_t(0x7fffffff) / cols) {
        delete plan;
        return fail(PSGD_ERR_INVALID_ARG,
                    "psgd_clip_plan_create: layer " + std::to_string(i) + " needs 1 <= rows*cols < 2^31");
      }
      const int64_t numel = rows * cols;
      plan->info.push_back(psgd_clip_layer_info{rows, cols, numel, off});
      ClLayer L{};
      L.tile0 = int32_t(plan->tiles.size());
      L.ntiles = int32_t((numel + kTile - 1) / kTile);
      for (int32_t c = 0; c < L.ntiles; ++c) {
        ClTile t{};
        t.begin = off + int64_t(c) * kTile;
        t.len = int32_t(std::min<int64_t>(kTile, numel - int64_t(c) * kTile));
        t.matrix = rows > 1 && cols > 1 ? 1 : 0;
        plan->tiles.push_back(t);
      }
      if (plan->tiles.size() > size_t(0xffffffu)) {  // tiles * kThreads fits a launch's 32 bits
        delete plan;
        return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: too many tiles");
      }
      plan->layers.push_back(L);
      plan->numel += numel;
      off = (off + numel + kAlignElems - 1) / kAlignElems * kAlignElems;
    }
    plan->worker_stride = off;
    uint64_t ws = 0;
    plan->ws_part = ws;  // one partial per tile and slice
    ws = a256(ws + uint64_t(n_slices) * plan->tiles.size() * sizeof(double));
    plan->ws_coef = ws;
    ws = a256(ws + uint64_t(n_slices) * sizeof(float));
    plan->ws_aw = ws;
    ws = a256(ws + sizeof(AwState));
    plan->workspace_bytes = ws;
  } catch (...) {
    delete plan;
    return no_memory();
  }
  *out = plan;
  return PSGD_OK;
}

extern "C" psgd_status psgd_clip_plan_sizes(const psgd_clip_plan* plan, psgd_clip_sizes* out) {
  if (plan == nullptr || out == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_sizes: NULL argument");
  psgd_clip_sizes s{};
  s.n_layers = int32_t(plan->info.size());
  s.n_slices = plan->n_slices;
  s.grad_dtype = int32_t(plan->dtype);
  s.worker_stride = plan->worker_stride;
  s.numel = plan->numel;
  s.workspace_bytes = plan->workspace_bytes;
  const uint64_t gb = plan->dtype == PSGD_BF16 ? 2 : 4;
  const uint64_t n = uint64_t(plan->numel), S = uint64_t(plan->n_slices);
  s.norm_bytes = S * n * gb;
  s.clip_bytes = 2 * S * n * gb;
  s.adamw_bytes = n * (gb + 24);
  *out = s;
  return PSGD_OK;
}

extern "C" psgd_status psgd_clip_plan_layer_info(const psgd_clip_plan* plan, int32_t layer,
                                                 psgd_clip_layer_info* out) {
  if (plan == nullptr || out == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_layer_info: NULL argument");
  if (layer < 0 || size_t(layer) >= plan->info.size())
    return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_layer_info: layer index out of range");
  *out = plan->info[size_t(layer)];
  return PSGD_OK;
}

extern "C" psgd_status psgd_clip_plan_destroy(psgd_clip_plan* plan) {
  if (plan == nullptr) return PSGD_OK;
  psgd_status st = PSGD_OK;
  for (const PendingTiming& t : plan->pending) {
    (void)hipEventDestroy(t.start);
    (void)hipEventDestroy(t.stop);
  }
  for (hipEvent_t ev : plan->event_pool) (void)hipEventDestroy(ev);
  for (auto& kv : plan->dev) {
    int cur = 0;
    const bool have = hipGetDevice(&cur) == hipSuccess;
    if (have && cur != kv.first) (void)hipSetDevice(kv.first);
    if (hipFree(kv.second) != hipSuccess) {
      set_error("psgd_clip_plan_destroy: hipFree of the device tables failed");
      st = PSGD_ERR_HIP;
    }
    if (have && cur != kv.first) (void)hipSetDevice(cur);
  }
  delete plan;
  return st;
}

extern "C" psgd_status psgd_clip_plan_set_timing(psgd_clip_plan* plan, int32_t enable) {
  if (plan == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_set_timing: plan is NULL");
  plan->timing = enable != 0;
  return PSGD_OK;
}

extern "C" psgd_status psgd_clip_plan_kernel_stats(psgd_clip_plan* plan, psgd_kernel_stat* out, int32_t capacity,
                                                   int32_t* count, int32_t reset) {
  if (plan == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_kernel_stats: plan is NULL");
  if (capacity > 0 && out == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_kernel_stats: out is NULL");
  psgd_status st = PSGD_OK;
  try {
    plan->event_pool.reserve(plan->event_pool.size() + 2 * plan->pending.size());
    for (const PendingTiming& t : plan->pending) {
      float ms = 0.f;
      hipError_t e = hipEventSynchronize(t.stop);
      if (e == hipSuccess) e = hipEventElapsedTime(&ms, t.start, t.stop);
      if (e != hipSuccess) {
        st = hip_fail("psgd_clip_plan_kernel_stats", e);
      } else {
        plan->stats[t.kernel].launches += 1;
        plan->stats[t.kernel].total_ms += double(ms);
      }
      plan->event_pool.push_back(t.start);
      plan->event_pool.push_back(t.stop);
    }
  } catch (...) {
    return no_memory();
  }
  plan->pending.clear();
  int32_t n = 0;
  for (int k = 0; k < kNumK; ++k) {
    if (plan->stats[k].launches == 0) continue;
    if (n < capacity) {
      psgd_kernel_stat ks{};
      std::snprintf(ks.name, sizeof(ks.name), "%s", kNames[k]);
      ks.launches = plan->stats[k].launches;
      ks.total_ms = plan->stats[k].total_ms;
      out[n] = ks;
    }
    ++n;
  }
  if (count != nullptr) *count = std::min(n, std::max<int32_t>(capacity, 0));
  if (reset)
    for (auto& k : plan->stats) k = KernelStat{};
  return st;
}

extern "C" psgd_status psgd_grad_norm(psgd_clip_plan* plan, const void* grads, psgd_norm_kind kind, float* norms,
                                      float* tensor_norms, void* workspace, void* stream) {
  static const char* const fn = "psgd_grad_norm";
  try {
    if (plan == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_grad_norm: plan is NULL");
    psgd_status s = check_kind(fn, kind);
    if (s != PSGD_OK) return s;
    const uint64_t S = uint64_t(plan->n_slices), gb = plan->dtype == PSGD_BF16 ? 2 : 4;
    const Span spans[] = {
        {"grads", grads, S * uint64_t(plan->worker_stride) * gb, 16, false},
        {"norms", norms, S * 4, 4, false},
        {"tensor_norms", tensor_norms, S * plan->layers.size() * 4, 4, true},
        {"workspace", workspace, plan->workspace_bytes, 16, false},
    };
    if ((s = check_spans(fn, spans, 4)) != PSGD_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    DevTables dt{};
    if ((s = device_tables(fn, plan, st, &dt)) != PSGD_OK) return s;
    return enqueue_norm(plan, kind, dt, grads, double(INFINITY), norms, tensor_norms, nullptr,
                        static_cast<char*>(workspace), AwArgs{}, st);
  } catch (...) {
    return no_memory();
  }
}

extern "C" psgd_status psgd_grad_clip(psgd_clip_plan* plan, const void* grads, void* out, psgd_norm_kind kind,
                                      float max_norm, float* norms, float* coefs, void* workspace, void* stream) {
  static const char* const fn = "psgd_grad_clip";
  try {
    if (plan == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_grad_clip: plan is NULL");
    psgd_status s = check_kind(fn, kind);
    if (s != PSGD_OK) return s;
    if (!(max_norm > 0.0f)) return fail(PSGD_ERR_INVALID_ARG, "psgd_grad_clip: max_norm must be > 0");
    const uint64_t S = uint64_t(plan->n_slices), gb = plan->dtype == PSGD_BF16 ? 2 : 4;
    const uint64_t bytes = S * uint64_t(plan->worker_stride) * gb;
    const Span spans[] = {
        {"grads", grads, bytes, 16, false},
        {"out", out, bytes, 16, false},
        {"norms", norms, S * 4, 4, false},
        {"coefs", coefs, S * 4, 4, false},
        {"workspace", workspace, plan->workspace_bytes, 16, false},
    };
    if ((s = check_spans(fn, spans, 5, 0, 1)) != PSGD_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    DevTables dt{};
    if ((s = device_tables(fn, plan, st, &dt)) != PSGD_OK) return s;
    char* ws = static_cast<char*>(workspace);
    if ((s = enqueue_norm(plan, kind, dt, grads, double(max_norm), norms, nullptr, coefs, ws, AwArgs{}, st)) != PSGD_OK)
      return s;
    const dim3 grid(static_cast<unsigned>(plan->tiles.size()), static_cast<unsigned>(S));
    const float* c = reinterpret_cast<const float*>(ws + plan->ws_coef);
    if (plan->dtype == PSGD_BF16)
      return launch(plan, kScale, cl_scale<uint16_t>, grid, dim3(kThreads), st, dt.tiles,
                    static_cast<const uint16_t*>(grads), static_cast<uint16_t*>(out), c, plan->worker_stride);
    return launch(plan, kScale, cl_scale<float>, grid, dim3(kThreads), st, dt.tiles, static_cast<const float*>(grads),
                  static_cast<float*>(out), c, plan->worker_stride);
  } catch (...) {
    return no_memory();
  }
}

extern "C" psgd_status psgd_adamw_apply(psgd_clip_plan* plan, const psgd_adamw_config* config, const void* update,
                                        float* params, float* exp_avg, float* exp_avg_sq, void* params_bf16,
                                        int64_t* step, float* norm, void* workspace, void* stream) {
  static const char* const fn = "psgd_adamw_apply";
  try {
    if (plan == nullptr || config == nullptr)
      return fail(PSGD_ERR_INVALID_ARG, "psgd_adamw_apply: plan or config is NULL");
    const psgd_adamw_config cf = *config;
    if (plan->n_slices != 1) return fail(PSGD_ERR_INVALID_ARG, "psgd_adamw_apply: the plan must have one slice");
    if (cf.flags & ~uint32_t(PSGD_ADAMW_DECAY_MATRICES_ONLY | PSGD_ADAMW_SKIP_NONFINITE))
      return fail(PSGD_ERR_UNSUPPORTED, "psgd_adamw_apply: unknown flag bits");
    auto finite = [](double v) { return std::isfinite(v) && std::isfinite(float(v)); };
    if (!(finite(cf.lr) && cf.lr >= 0.0)) return fail(PSGD_ERR_INVALID_ARG, "psgd_adamw_apply: lr must be finite and >= 0");
    if (!(cf.beta1 >= 0.0 && cf.beta1 < 1.0 && cf.beta2 >= 0.0 && cf.beta2 < 1.0))
      return fail(PSGD_ERR_INVALID_ARG, "psgd_adamw_apply: beta1 and beta2 must be in [0, 1)");
    if (!(finite(cf.eps) && float(cf.eps) > 0.0f))
      return fail(PSGD_ERR_INVALID_ARG, "psgd_adamw_apply: eps must be finite and > 0 in float32");
    if (!(finite(cf.weight_decay) && cf.weight_decay >= 0.0 && finite(cf.lr * cf.weight_decay)))
      return fail(PSGD_ERR_INVALID_ARG, "psgd_adamw_apply: weight_decay must be finite and >= 0");
    if (!(cf.max_norm >= 0.0)) return fail(PSGD_ERR_INVALID_ARG, "psgd_adamw_apply: max_norm must be >= 0");
    const bool clipped = cf.max_norm > 0.0;
    if ((cf.flags & PSGD_ADAMW_SKIP_NONFINITE) && !clipped)
      return fail(PSGD_ERR_INVALID_ARG, "psgd_adamw_apply: PSGD_ADAMW_SKIP_NONFINITE needs max_norm > 0");
    psgd_status s = clipped ? check_kind(fn, cf.norm_kind) : PSGD_OK;
    if (s != PSGD_OK) return s;
    if (!clipped && norm != nullptr)
      return fail(PSGD_ERR_INVALID_ARG, "psgd_adamw_apply: norm must be NULL when max_norm is 0");
    const uint64_t n = uint64_t(plan->worker_stride), gb = plan->dtype == PSGD_BF16 ? 2 : 4;
    const Span spans[] = {
        {"update", update, n * gb, 16, false},
        {"params", params, n * 4, 16, false},
        {"exp_avg", exp_avg, n * 4, 16, false},
        {"exp_avg_sq", exp_avg_sq, n * 4, 16, false},
        {"params_bf16", params_bf16, n * 2, 16, true},
        {"step", step, 8, 8, false},
        {"norm", norm, 4, 4, !clipped},
        {"workspace", workspace, plan->workspace_bytes, 16, false},
    };
    if ((s = check_spans(fn, spans, 8)) != PSGD_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    DevTables dt{};
    if ((s = device_tables(fn, plan, st, &dt)) != PSGD_OK) return s;
    char* ws = static_cast<char*>(workspace);
    AwArgs aw{};
    aw.lr = cf.lr;
    aw.beta1 = cf.beta1;
    aw.beta2 = cf.beta2;
    aw.step = step;
    aw.state = reinterpret_cast<AwState*>(ws + plan->ws_aw);
    aw.have_norm = clipped ? 1 : 0;
    aw.skip_nonfinite = (cf.flags & PSGD_ADAMW_SKIP_NONFINITE) ? 1 : 0;
    if ((s = enqueue_norm(plan, clipped ? cf.norm_kind : int(PSGD_NORM_L2), dt, update, cf.max_norm, norm, nullptr,
                          nullptr, ws, aw, st)) != PSGD_OK)
      return s;
    const dim3 grid(static_cast<unsigned>(plan->tiles.size()));
    const int mo = (cf.flags & PSGD_ADAMW_DECAY_MATRICES_ONLY) ? 1 : 0;
    const float b1 = float(cf.beta1), o1 = float(1.0 - cf.beta1), b2 = float(cf.beta2), o2 = float(1.0 - cf.beta2);
    const float eps = float(cf.eps), decay = float(cf.lr * cf.weight_decay);
    uint16_t* copy = static_cast<uint16_t*>(params_bf16);
    const AwState* state = aw.state;
    if (plan->dtype == PSGD_BF16)
      return launch(plan, kAdamw, cl_adamw<uint16_t>, grid, dim3(kThreads), st, dt.tiles,
                    static_cast<const uint16_t*>(update), params, exp_avg, exp_avg_sq, copy, state, b1, o1, b2, o2,
                    eps, decay, mo);
    return launch(plan, kAdamw, cl_adamw<float>, grid, dim3(kThreads), st, dt.tiles, static_cast<const float*>(update),
                  params, exp_avg, exp_avg_sq, copy, state, b1, o1, b2, o2, eps, decay, mo);
  } catch (...) {
    return no_memory();
  }
}
