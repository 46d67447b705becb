// Gradient norms, clipping and AdamW over packed tensors: the gfx950 kernels and the host
// side of psgd_clip.h.
//
// A tile is at most kTile consecutive elements of one tensor, a run is a number of
// consecutive tiles.  Sums of squares are held in float64, and every reduction has a fixed
// order (another one in each variant: their float64 sums may differ in the last bits).
//
//   cl_norm    per (run, slice): the sum of squares, or the largest magnitude
//   cl_final   from these partials: the slices' norms and coefficients, the tensors' norms
//              if asked, and for AdamW the step's scalars
//   cl_scale   per (part of a tile, slice): out = c * g
//   cl_adamw   per part of a tile: the weight update
// Slices of a moderate size leave cl_final out: cl_scale and cl_adamw join the partials
// themselves (FOLD).  Small ones take a single launch, a workgroup per slice:
//   cl_small        norms, and clipping
//   cl_small_adamw  the AdamW step
//
// No kernel waits for another workgroup, and no state is kept between calls.

#include <hip/hip_runtime.h>
#include <hip/hip_ext.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <map>
#include <new>
#include <string>
#include <vector>

#include "plan.hpp"
#include "psgd_clip.h"

namespace psgd {
namespace clip {

// Elements per tile.  16384 ran alike on large plans; 8192 gives moderate ones more
// workgroups.
constexpr int kTile = 8192;
constexpr int kThreads = 256;
// cl_norm workgroups per slice: for a slice's norm cl_final's 256 threads then take at most
// 16 partials each (for a tensor's, one per tile).  Up to here there are about as many runs
// as tiles; the cut by cost lets short neighbours share one (119 odd tensors: 1155 tiles in
// 1114 runs).
constexpr int64_t kMaxRuns = 4096;
// What a tile costs cl_norm besides its elements, in elements: its loads start anew, so a
// run of tiny tensors takes their latencies one after the other (119 tensors of 1 to 2
// million elements: 17.8 us counted at 1024, 11.3 at 8192).
constexpr int64_t kTileCost = kTile;
// The norm pass leaves the last kKeepBytes it reads in the 256 MB memory-side cache
// (ordinary loads; the rest is read with non-temporal ones, which run at 7.2 instead of
// 6.4 TB/s), and the second pass goes backwards and finds them there.  Against no such
// part: AdamW on a 45 MB update 65.3 instead of 70.2 us, clipping 715 MB 327 instead of
// 332 us, 1.6 GB 732 instead of 740 us.  0, 64, 128, 160, 192, 224, 256 MB tried.
constexpr int64_t kKeepBytes = int64_t(224) << 20;
// Joining the partials in cl_scale / cl_adamw instead of a launch of cl_final (us a call in
// a graph, clipping float32): 1 slice of 2M elements 9.4 against 9.6, of 4M 16.1 against
// 12.7; 8 slices of 0.5M 12.0 against 12.8, of 1M 22.3 against 21.3.  Called one by one,
// the launch saved is worth 2 us more.
constexpr int64_t kFoldRuns = 256;   // per slice
constexpr int64_t kFoldTotal = 512;  // all slices together
// A single launch with a workgroup per slice, for plans of at most kMaxItems items, up to
// kSmallNorm, kSmallClip or kSmallAdamw elements per slice.  Against the two launches
// above (us a call in a graph): norm of 16384 4.4 against 5.2, of 32768 6.0 against 5.5;
// clip 5.8 / 5.9 and 8.3 / 5.8; AdamW of 4096 5.9 / 7.1, of 8192 7.7 / 7.1, of 16384
// 11.1 / 7.4.  Called one by one the smaller number of launches is worth 3.5 us.
constexpr int kItem = 512;      // elements per item
constexpr int kMaxItems = 128;
constexpr int kSmallThreads = 1024;
constexpr int64_t kSmallNorm = 32768, kSmallClip = 16384, kSmallAdamw = 8192;
// Parts a cl_scale workgroup takes when out is grads: 1, 2, 3, 4 of them let a call that has
// nothing to scale return after 39, 20, 13, 10 us (16 x 45 MB: 175 thousand workgroups
// for 1), and scale in 221, 216, 220, 233 us when it has.  With 2 the whole call takes 134
// us with nothing to scale (the norm alone 112) and 334 with every slice scaled.
constexpr int kInPlaceParts = 2;
constexpr int64_t kMaxTiles = 0x1fffff;  // tiles * (kTile / 4) threads fit a launch's 32 bits

struct ClTile {
  int64_t begin;   // element offset of the tile in a slice
  int32_t len;     // elements in the tile (kTile except at a tensor's end)
  int32_t matrix;  // 1: the tensor has more than one row and more than one column
};

struct ClLayer {
  int32_t tile0, ntiles;  // the tensor's tiles
};

struct ClRun {
  int32_t tile0, tile1;  // tiles [tile0, tile1)
};

// A part of a small plan's tensor, for one wave.
struct ClItem {
  int32_t begin, len;  // elements of the slice
  int32_t matrix;
  int32_t pad;
};

// The AdamW step's scalars, written by cl_final or cl_norm for cl_adamw.
struct AwState {
  float step_size;  // lr / (1 - beta1^t)
  float inv_sqrt;   // 1 / sqrt(1 - beta2^t)
  int64_t t;
};

struct AwArgs {
  double lr, beta1, beta2;
  const int64_t* step;
  AwState* state;
};

// What cl_adamw takes besides its buffers.  A beta is the sum of two float32: rounded to one,
// it and 1 - beta miss the sum 1, and the beta of the bias correction, by up to 2^-25 in
// every step (a second moment at beta2 = 0.99999 settled at 0.9986 of the squares' average).
struct AwConfig {
  float beta1, beta1_lo, om_beta1, beta2, beta2_lo, om_beta2, eps, decay;
  int32_t matrices_only, skip_nonfinite;
};

enum KernelId { kNorm = 0, kFinal, kScale, kAdamw, kSmall, kSmallAw, kNumK };
const char* const kNames[kNumK] = {"cl_norm", "cl_final", "cl_scale", "cl_adamw", "cl_small", "cl_small_adamw"};

}  // namespace clip
}  // namespace psgd

struct psgd_clip_plan {
  int32_t n_slices = 0;
  psgd_dtype dtype = PSGD_F32;
  std::vector<psgd_clip_layer_info> info;
  std::vector<psgd::clip::ClLayer> layers;
  std::vector<psgd::clip::ClTile> tiles;
  std::vector<psgd::clip::ClRun> runs;
  std::vector<psgd::clip::ClItem> items;        // of a small plan; empty otherwise
  std::vector<psgd::clip::ClLayer> item_layers;  // each tensor's items
  int64_t worker_stride = 0, numel = 0;
  uint64_t ws_tile = 0, ws_run = 0, ws_coef = 0, ws_aw = 0, workspace_bytes = 0;
  std::map<int, void*> dev;  // device copy of the layer, tile and run tables, per HIP device
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
typedef float v8f __attribute__((ext_vector_type(8)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

// Vectors of NE elements in memory and in registers (always float32 there).  bfloat16
// widens exactly and is rounded to nearest even by the hardware conversion, which keeps
// NaN.  cl_norm and cl_scale move 16 bytes per lane: 4 float32 or 8 bfloat16 (with 4,
// 8 bytes, scaling bfloat16 ran at 5.2 instead of 6.4 TB/s).
template <typename T, int NE> struct Vec;
template <> struct Vec<float, 4> { typedef v4f mem; typedef v4f reg; };
template <> struct Vec<uint16_t, 4> { typedef v4b mem; typedef v4f reg; };
template <> struct Vec<uint16_t, 8> { typedef v8b mem; typedef v8f reg; };
template <typename T> constexpr int kUnit = 16 / int(sizeof(T));

template <int NE, bool KEEP = false, typename T>
__device__ __forceinline__ typename Vec<T, NE>::reg load(const T* p) {
  const auto* q = reinterpret_cast<const typename Vec<T, NE>::mem*>(p);
  return __builtin_convertvector(KEEP ? *q : __builtin_nontemporal_load(q), typename Vec<T, NE>::reg);
}

// The first n of NE elements (n >= 1); what follows is padding.
template <int NE, typename T>
__device__ __forceinline__ void store(T* p, typename Vec<T, NE>::reg v, int n) {
  const auto m = __builtin_convertvector(v, typename Vec<T, NE>::mem);
  if (n >= NE) {
    __builtin_nontemporal_store(m, reinterpret_cast<typename Vec<T, NE>::mem*>(p));
    return;
  }
#pragma unroll
  for (int j = 0; j < NE - 1; ++j) {
    const auto x = m[j];
    if (j < n) p[j] = __builtin_bit_cast(T, x);
  }
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

__device__ __forceinline__ AwState step_scalars(const AwArgs& aw) {
  AwState s;
  s.t = *aw.step + 1;
  s.step_size = float(aw.lr / (1.0 - pow(aw.beta1, double(s.t))));
  s.inv_sqrt = float(1.0 / sqrt(1.0 - pow(aw.beta2, double(s.t))));
  return s;
}

// Part of a moment's decay that its beta's second float32 brings; an infinite moment has to
// stay one (lo * inf is NaN for lo = 0, and of the other sign for lo < 0).
__device__ __forceinline__ float low_part(float lo, float moment) {
  return lo * __builtin_amdgcn_fmed3f(moment, -FLT_MAX, FLT_MAX);
}

// Four elements' AdamW update: the new x, m and v in place of the old.  Both moments are
// float32 sums: float64 ones took the single launch (7 thousand elements, one compute unit)
// 7.1 instead of 6.9 us.  (1 - beta2) g comes before its product with g: g^2 alone is
// infinite from 1.8e19 on, where (1 - beta2) g^2 is not.
__device__ __forceinline__ void adamw4(v4f g, v4f& x, v4f& m, v4f& v, const AwState& s, const AwConfig& cf, float decay) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j] = cf.beta1 * m[j] + (low_part(cf.beta1_lo, m[j]) + cf.om_beta1 * g[j]);
    v[j] = cf.beta2 * v[j] + (low_part(cf.beta2_lo, v[j]) + (cf.om_beta2 * g[j]) * g[j]);
    const float den = sqrtf(v[j]) * s.inv_sqrt + cf.eps;
    x[j] = fmaf(-decay, x[j], x[j]) - s.step_size * (m[j] / den);
  }
}

// A slice's norm from its runs' partials, by one wave.
template <typename N>
__device__ __forceinline__ double fold_norm(const typename N::acc_t* __restrict__ part_run, int n_runs) {
  typename N::acc_t acc = N::zero();
  for (int i = int(threadIdx.x & 63); i < n_runs; i += 64) acc = N::join(acc, part_run[i]);
  return N::norm(wave_join<N>(acc));
}

// ------------------------------------------------------------------ kernels
// This thread's part of a tile's partial.
template <typename GT, typename N, bool KEEP>
__device__ __forceinline__ typename N::acc_t tile_sum(const GT* __restrict__ g, int len) {
  constexpr int NE = kUnit<GT>;
  constexpr int STEP = kThreads * NE;
  typename N::acc_t acc = N::zero();
  const int whole = len / STEP * STEP;
  int e = int(threadIdx.x) * NE;
#pragma unroll 4
  for (; e < whole; e += STEP) {
    const auto v = load<NE, KEEP>(g + e);
#pragma unroll
    for (int j = 0; j < NE; ++j) N::take(acc, v[j]);
  }
  if (e < len) {
    const auto v = load<NE, KEEP>(g + e);  // a tensor's padding reaches the next multiple of 64 elements
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (e + j < len) N::take(acc, v[j]);
  }
  return acc;
}

// A workgroup reads one run of one slice (grid.y).  Its partial goes to `part_run`, each
// tile's to `part_tile` if tensor norms are wanted.  Bound by HBM reads: 715 MB of float32
// in 106 us on average, 101 at best (6.7 and 7.1 TB/s; a bare reading loop reaches 7.2); 508
// MB of bfloat16 in 84 us, 76 at best (MAX: 74 and 70).  A workgroup to a tile keeps its
// loads (32 KB per 256 threads, 16 KB of bfloat16) short enough that the last ones end
// together; float64 costs nothing next to the loads, if whole steps go without bounds
// checks (with them bfloat16 took 83 us at best).
template <typename GT, typename N>
__global__ __launch_bounds__(kThreads) void cl_norm(const ClTile* __restrict__ tiles, const ClRun* __restrict__ runs,
                                                    int n_tiles, const GT* __restrict__ grads, int64_t stride,
                                                    int64_t keep_from, typename N::acc_t* __restrict__ part_tile,
                                                    typename N::acc_t* __restrict__ part_run, AwArgs aw) {
  typedef typename N::acc_t acc_t;
  __shared__ acc_t lds[kThreads / 64];
  const int64_t slice = blockIdx.y;
  const ClRun r = runs[blockIdx.x];
  if (aw.state != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *aw.state = step_scalars(aw);
  acc_t run = N::zero();
  for (int i = r.tile0; i < r.tile1; ++i) {
    const ClTile t = tiles[i];
    const GT* g = grads + slice * stride + t.begin;
    const acc_t acc = slice * stride + t.begin >= keep_from ? tile_sum<GT, N, true>(g, t.len)
                                                            : tile_sum<GT, N, false>(g, t.len);
    run = N::join(run, acc);
    if (part_tile != nullptr && r.tile1 - r.tile0 > 1) {
      const acc_t tile = block_join<N>(acc, lds);
      if (threadIdx.x == 0) part_tile[slice * n_tiles + i] = tile;
    }
  }
  run = block_join<N>(run, lds);
  if (threadIdx.x == 0) {
    part_run[slice * gridDim.x + blockIdx.x] = run;
    if (part_tile != nullptr && r.tile1 - r.tile0 == 1) part_tile[slice * n_tiles + r.tile0] = run;
  }
}

// Joined value of p[0..n) in every thread of the workgroup.
template <typename N>
__device__ __forceinline__ typename N::acc_t join_all(const typename N::acc_t* __restrict__ p, int n,
                                                      typename N::acc_t* lds) {
  typename N::acc_t acc = N::zero();
#pragma unroll 8
  for (int i = int(threadIdx.x); i < n; i += kThreads) acc = N::join(acc, p[i]);
  return block_join<N>(acc, lds);
}

// Bound by its launch (4 us).  Letting cl_norm's last workgroup to arrive do this instead
// costs as much (a store, two device-wide counts and a load one after the other) and needs
// counters that outlive the call.
// grid.x: workgroup 0 of a slice (grid.y) takes its norm and coefficient; the next n_layers
// ones a tensor's norm each (tensor_norms given); the last one the AdamW step's scalars
// (aw.state given).
template <typename N>
__global__ __launch_bounds__(kThreads) void cl_final(const ClLayer* __restrict__ layers, int n_layers, int n_tiles,
                                                     int n_runs, const typename N::acc_t* __restrict__ part_tile,
                                                     const typename N::acc_t* __restrict__ part_run, double max_norm,
                                                     float* __restrict__ norms, float* __restrict__ tensor_norms,
                                                     float* __restrict__ coefs, float* __restrict__ ws_coef,
                                                     AwArgs aw) {
  __shared__ typename N::acc_t lds[kThreads / 64];
  const int64_t slice = blockIdx.y;
  const int l = int(blockIdx.x) - 1;
  if (l < 0) {
    if (part_run == nullptr) return;
    const double norm = N::norm(join_all<N>(part_run + slice * n_runs, n_runs, lds));
    if (threadIdx.x != 0) return;
    const float c = clip_coef(norm, max_norm);
    norms[slice] = float(norm);
    ws_coef[slice] = c;
    if (coefs != nullptr) coefs[slice] = c;
  } else if (tensor_norms != nullptr && l < n_layers) {
    const ClLayer L = layers[l];
    const double norm = N::norm(join_all<N>(part_tile + slice * n_tiles + L.tile0, L.ntiles, lds));
    if (threadIdx.x == 0) tensor_norms[slice * n_layers + l] = float(norm);
  } else if (threadIdx.x == 0) {
    *aw.state = step_scalars(aw);
  }
}

// What cl_scale and cl_adamw take a coefficient from: cl_final's, or (FOLD) the partials.
template <typename N>
struct CoefArgs {
  const float* coef;
  const typename N::acc_t* part_run;
  int32_t n_runs;
  double max_norm;
  float *norms, *coefs;  // outputs, written with FOLD only
};

// Coefficient of a slice; *norm gets its norm (FOLD).
template <typename N, bool FOLD>
__device__ __forceinline__ float coefficient(const CoefArgs<N>& a, int64_t slice, float* norm) {
  if (!FOLD) return a.coef[slice];
  const double d = fold_norm<N>(a.part_run + slice * a.n_runs, a.n_runs);
  const float c = clip_coef(d, a.max_norm);
  *norm = float(d);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.norms[slice] = float(d);
    if (a.coefs != nullptr) a.coefs[slice] = c;
  }
  return c;
}

// One 16-byte unit per thread and 4 KB per workgroup: reads and writes then sweep the
// buffers in dispatch order, which HBM serves at the speed of a plain copy (16 x 45 MB in
// 222 us on average, 216 at best, 6.4 and 6.6 TB/s; 64 KB per workgroup took 262 us).
template <typename GT, typename N, bool FOLD>
__global__ __launch_bounds__(kThreads) void cl_scale(const ClTile* __restrict__ tiles, int n_parts,
                                                     const GT* grads, GT* out, int64_t stride, CoefArgs<N> ca) {
  constexpr int NE = kUnit<GT>, parts = kTile / (kThreads * NE);
  const int64_t slice = gridDim.y - 1 - blockIdx.y;  // last read, first rescaled
  float norm;
  const float c = coefficient<N, FOLD>(ca, slice, &norm);
  if (c == 1.0f && grads == out) return;
  for (int p = n_parts - 1 - int(blockIdx.x); p >= 0; p -= int(gridDim.x)) {
    const ClTile t = tiles[p / parts];
    const int e = (p % parts * kThreads + int(threadIdx.x)) * NE;
    if (e >= t.len) continue;
    const int64_t at = slice * stride + t.begin + e;
    store<NE>(out + at, load<NE>(grads + at) * c, t.len - e);
  }
}

// Four elements per thread, as in cl_scale: seven (eight) streams at 5.8 to 6.5 TB/s.  45 MB of
// update in 52 us, 1.6 GB in 1.72 to 1.95 ms from card to card (64 KB per workgroup: 67 us,
// 2.11 ms).
// CLIP: 0 no clipping (c = 1), 1 cl_final's coefficient, 2 from the partials.
template <typename GT, typename N, int CLIP>
__global__ __launch_bounds__(kThreads) void cl_adamw(const ClTile* __restrict__ tiles, const GT* __restrict__ update,
                                                     float* __restrict__ params, float* __restrict__ exp_avg,
                                                     float* __restrict__ exp_avg_sq, uint16_t* __restrict__ copy,
                                                     const AwState* __restrict__ state, AwConfig cf, CoefArgs<N> ca,
                                                     int64_t* step) {
  constexpr int parts = kTile / (kThreads * 4);
  const AwState s = *state;
  float c = 1.0f;
  if (CLIP) {
    float norm;
    c = coefficient<N, CLIP == 2>(ca, 0, &norm);
    if (CLIP == 1) norm = *ca.norms;
    if (cf.skip_nonfinite && !isfinite(norm)) return;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) step[0] = s.t;
  const unsigned p = gridDim.x - 1 - blockIdx.x;  // last read, first used
  const ClTile t = tiles[p / parts];
  const float d = cf.matrices_only && !t.matrix ? 0.0f : cf.decay;
  const int e = (int(p % parts) * kThreads + int(threadIdx.x)) * 4;
  if (e >= t.len) return;
  const int64_t at = t.begin + e;
  const v4f g = load<4>(update + at) * c;
  v4f x = load<4>(params + at), m = load<4>(exp_avg + at), v = load<4>(exp_avg_sq + at);
  adamw4(g, x, m, v, s, cf, d);
  const int n = t.len - e;
  store<4>(params + at, x, n);
  store<4>(exp_avg + at, m, n);
  store<4>(exp_avg_sq + at, v, n);
  if (copy != nullptr) store<4>(copy + at, x, n);
}

// The norm of one slice by one workgroup (every thread gets it): an item per wave at a
// time, its partial into `part`, which is whole after the barrier inside.
template <typename GT, typename N>
__device__ __forceinline__ double small_norm(const ClItem* items, int n_items, const GT* __restrict__ g,
                                             typename N::acc_t* part) {
  constexpr int NE = kUnit<GT>;
  const int lane = int(threadIdx.x & 63), wave = int(threadIdx.x >> 6);
  for (int i = wave; i < n_items; i += kSmallThreads / 64) {
    const ClItem it = items[i];
    typename N::acc_t acc = N::zero();
#pragma unroll
    for (int k = 0; k < kItem / (64 * NE); ++k) {
      const int e = (k * 64 + lane) * NE;
      if (e >= it.len) continue;
      const auto v = load<NE, true>(g + it.begin + e);
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if (e + j < it.len) N::take(acc, v[j]);
    }
    acc = wave_join<N>(acc);
    if (lane == 0) part[i] = acc;
  }
  __syncthreads();
  typename N::acc_t acc = lane < n_items ? part[lane] : N::zero();
  if (lane + 64 < n_items) acc = N::join(acc, part[lane + 64]);
  return N::norm(wave_join<N>(acc));
}

// Bound by latency: launch, table, loads, join, loads, stores (4 us for 7 thousand elements).
// One slice per workgroup: its norm, its tensors' (tensor_norms given), and out = c * g
// (out given).
template <typename GT, typename N>
__global__ __launch_bounds__(kSmallThreads) void cl_small(const ClItem* __restrict__ item_table, int n_items,
                                                          const ClLayer* __restrict__ item_layers, int n_layers,
                                                          const GT* grads, GT* out, int64_t stride, double max_norm,
                                                          float* __restrict__ norms, float* __restrict__ tensor_norms,
                                                          float* __restrict__ coefs) {
  constexpr int NE = kUnit<GT>;
  __shared__ typename N::acc_t part[kMaxItems];
  __shared__ ClItem items[kMaxItems];
  const int lane = int(threadIdx.x & 63), wave = int(threadIdx.x >> 6);
  const int64_t slice = blockIdx.x;
  if (int(threadIdx.x) < n_items) items[threadIdx.x] = item_table[threadIdx.x];
  __syncthreads();
  const GT* g = grads + slice * stride;
  const double norm = small_norm<GT, N>(items, n_items, g, part);
  if (tensor_norms != nullptr && int(threadIdx.x) < n_layers) {
    const ClLayer L = item_layers[threadIdx.x];
    typename N::acc_t acc = N::zero();
    for (int i = 0; i < L.ntiles; ++i) acc = N::join(acc, part[L.tile0 + i]);
    tensor_norms[slice * n_layers + int(threadIdx.x)] = float(N::norm(acc));
  }
  const float c = clip_coef(norm, max_norm);
  if (threadIdx.x == 0) {
    norms[slice] = float(norm);
    if (coefs != nullptr) coefs[slice] = c;
  }
  if (out == nullptr || (c == 1.0f && grads == out)) return;
  GT* o = out + slice * stride;
  for (int i = wave; i < n_items; i += kSmallThreads / 64) {
    const ClItem it = items[i];
#pragma unroll
    for (int k = 0; k < kItem / (64 * NE); ++k) {
      const int e = (k * 64 + lane) * NE;
      if (e < it.len) store<NE>(o + it.begin + e, load<NE, true>(g + it.begin + e) * c, it.len - e);
    }
  }
}

// The whole AdamW step in one workgroup; one wave forms the step's scalars (two float64
// powers) while the others take the norm.  6.9 us for 7 thousand elements.
template <typename GT, typename N, bool CLIP>
__global__ __launch_bounds__(kSmallThreads) void cl_small_adamw(const ClItem* __restrict__ item_table, int n_items,
                                                                const GT* __restrict__ update,
                                                                float* __restrict__ params,
                                                                float* __restrict__ exp_avg,
                                                                float* __restrict__ exp_avg_sq,
                                                                uint16_t* __restrict__ copy, AwConfig cf, AwArgs aw,
                                                                double max_norm, float* __restrict__ norm_out,
                                                                int64_t* step) {
  __shared__ typename N::acc_t part[kMaxItems];
  __shared__ ClItem items[kMaxItems];
  __shared__ AwState scalars;
  const int lane = int(threadIdx.x & 63), wave = int(threadIdx.x >> 6);
  if (int(threadIdx.x) < n_items) items[threadIdx.x] = item_table[threadIdx.x];
  __syncthreads();
  if (threadIdx.x == kSmallThreads - 1) scalars = step_scalars(aw);
  float c = 1.0f;
  if (!CLIP) __syncthreads();
  if (CLIP) {
    const double norm = small_norm<GT, N>(items, n_items, update, part);  // a barrier inside
    c = clip_coef(norm, max_norm);
    if (threadIdx.x == 0) norm_out[0] = float(norm);
    if (cf.skip_nonfinite && !isfinite(float(norm))) return;
  }
  const AwState s = scalars;
  if (threadIdx.x == 0) step[0] = s.t;  // read before the barrier
  for (int i = wave; i < n_items; i += kSmallThreads / 64) {
    const ClItem it = items[i];
    const float d = cf.matrices_only && !it.matrix ? 0.0f : cf.decay;
#pragma unroll
    for (int k = 0; k < kItem / 256; ++k) {
      const int e = (k * 64 + lane) * 4, at = it.begin + e, n = it.len - e;
      if (n <= 0) continue;
      const v4f g = load<4>(update + at) * c;
      v4f x = load<4>(params + at), m = load<4>(exp_avg + at), v = load<4>(exp_avg_sq + at);
      adamw4(g, x, m, v, s, cf, d);
      store<4>(params + at, x, n);
      store<4>(exp_avg + at, m, n);
      store<4>(exp_avg_sq + at, v, n);
      if (copy != nullptr) store<4>(copy + at, x, n);
    }
  }
}

// ------------------------------------------------------------------ host helpers
uint64_t a256(uint64_t x) { return (x + 255) / 256 * 256; }

struct DevTables {
  const ClLayer* layers;
  const ClTile* tiles;
  const ClRun* runs;
  const ClItem* items;
  const ClLayer* item_layers;
};

// The plan's tables one after the other, each at a multiple of 256 bytes.
struct Part {
  const void* src;
  uint64_t bytes, at;
};

constexpr int kParts = 5;

uint64_t lay_out(const psgd_clip_plan* plan, Part (&p)[kParts]) {
  p[0] = Part{plan->layers.data(), plan->layers.size() * sizeof(ClLayer), 0};
  p[1] = Part{plan->tiles.data(), plan->tiles.size() * sizeof(ClTile), 0};
  p[2] = Part{plan->runs.data(), plan->runs.size() * sizeof(ClRun), 0};
  p[3] = Part{plan->items.data(), plan->items.size() * sizeof(ClItem), 0};
  p[4] = Part{plan->item_layers.data(), plan->item_layers.size() * sizeof(ClLayer), 0};
  uint64_t at = 0;
  for (Part& x : p) {
    x.at = at;
    at = a256(at + x.bytes);
  }
  return at;
}

psgd_status device_tables(const char* fn, psgd_clip_plan* plan, hipStream_t st, DevTables* out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail("hipGetDevice", e);
  Part parts[kParts];
  const uint64_t total = lay_out(plan, parts);
  auto it = plan->dev.find(dev);
  if (it == plan->dev.end() || plan->timing) {
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    e = hipStreamIsCapturing(st, &cs);
    if (e != hipSuccess) return hip_fail("hipStreamIsCapturing", e);
    if (cs != hipStreamCaptureStatusNone)
      return fail(PSGD_ERR_INVALID_ARG, std::string(fn) + ": a plan can be captured into a graph only after an eager "
                                            "call of the plan on this device, and with kernel timing off");
  }
  if (it == plan->dev.end()) {
    std::vector<char> image(total);
    for (const Part& p : parts)
      if (p.bytes != 0) std::memcpy(image.data() + p.at, p.src, p.bytes);
    it = plan->dev.emplace(dev, nullptr).first;
    void* base = nullptr;
    e = hipMalloc(&base, total);
    if (e != hipSuccess) {
      plan->dev.erase(it);
      return fail(PSGD_ERR_NO_MEMORY, std::string("hipMalloc of the plan's device tables: ") + hipGetErrorString(e));
    }
    e = hipMemcpy(base, image.data(), total, hipMemcpyHostToDevice);
    if (e != hipSuccess) {
      (void)hipFree(base);
      plan->dev.erase(it);
      return hip_fail("upload of the plan's device tables", e);
    }
    it->second = base;
  }
  const char* b = static_cast<const char*>(it->second);
  out->layers = reinterpret_cast<const ClLayer*>(b + parts[0].at);
  out->tiles = reinterpret_cast<const ClTile*>(b + parts[1].at);
  out->runs = reinterpret_cast<const ClRun*>(b + parts[2].at);
  out->items = reinterpret_cast<const ClItem*>(b + parts[3].at);
  out->item_layers = reinterpret_cast<const ClLayer*>(b + parts[4].at);
  return PSGD_OK;
}

// Launch on `st`; with timing on, through hipExtLaunchKernelGGL with events the runtime
// records with the dispatch itself.
template <typename... KArgs, typename... Args>
psgd_status launch(psgd_clip_plan* plan, int kid, void (*kernel)(KArgs...), dim3 grid, dim3 block, hipStream_t st,
                   Args... args) {
  hipEvent_t a = nullptr, b = nullptr;
  if (plan->timing) {
    room_for_timing(plan);
    psgd_status s = take_event(plan->event_pool, &a);
    if (s == PSGD_OK) s = take_event(plan->event_pool, &b);
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

psgd_status check_kind(const char* fn, int kind) {
  if (kind == PSGD_NORM_L2 || kind == PSGD_NORM_MAX) return PSGD_OK;
  return fail(PSGD_ERR_UNSUPPORTED, std::string(fn) + ": unknown norm kind");
}

bool small(const psgd_clip_plan* plan, int64_t most) {
  return !plan->items.empty() && plan->worker_stride <= most;
}

bool fold(const psgd_clip_plan* plan) {
  const int64_t runs = int64_t(plan->runs.size());
  return runs <= kFoldRuns && runs * plan->n_slices <= kFoldTotal;
}

// The partials of every slice's norm.  `again`: the same call reads the gradients once more.
template <typename GT, typename N>
psgd_status enqueue_partials(psgd_clip_plan* plan, const DevTables& dt, const void* grads, bool tensors, bool again,
                             const AwArgs& aw, char* ws, hipStream_t st) {
  typedef typename N::acc_t acc_t;
  const int64_t total = int64_t(plan->n_slices) * plan->worker_stride;
  const int64_t keep_from = again ? total - kKeepBytes / int64_t(sizeof(GT)) : total;
  const dim3 grid(static_cast<unsigned>(plan->runs.size()), static_cast<unsigned>(plan->n_slices));
  return launch(plan, kNorm, cl_norm<GT, N>, grid, dim3(kThreads), st, dt.tiles, dt.runs, int(plan->tiles.size()),
                static_cast<const GT*>(grads), plan->worker_stride, keep_from,
                tensors ? reinterpret_cast<acc_t*>(ws + plan->ws_tile) : nullptr,
                reinterpret_cast<acc_t*>(ws + plan->ws_run), aw);
}

// What follows from the partials: see cl_final.
template <typename N>
psgd_status enqueue_final(psgd_clip_plan* plan, const DevTables& dt, double max_norm, float* norms,
                          float* tensor_norms, float* coefs, const AwArgs& aw, char* ws, hipStream_t st) {
  typedef typename N::acc_t acc_t;
  const int n_layers = tensor_norms != nullptr ? int(plan->layers.size()) : 0;
  const unsigned blocks = 1u + unsigned(n_layers) + (aw.state != nullptr ? 1u : 0u);
  return launch(plan, kFinal, cl_final<N>, dim3(blocks, static_cast<unsigned>(plan->n_slices)), dim3(kThreads), st,
                dt.layers, n_layers, int(plan->tiles.size()), int(plan->runs.size()),
                reinterpret_cast<const acc_t*>(ws + plan->ws_tile),
                norms != nullptr ? reinterpret_cast<const acc_t*>(ws + plan->ws_run) : nullptr, max_norm, norms,
                tensor_norms, coefs, reinterpret_cast<float*>(ws + plan->ws_coef), aw);
}

template <typename N>
CoefArgs<N> coef_args(const psgd_clip_plan* plan, double max_norm, float* norms, float* coefs, const char* ws) {
  return CoefArgs<N>{reinterpret_cast<const float*>(ws + plan->ws_coef),
                     reinterpret_cast<const typename N::acc_t*>(ws + plan->ws_run), int32_t(plan->runs.size()),
                     max_norm, norms, coefs};
}

template <typename GT, typename N>
psgd_status enqueue_small(psgd_clip_plan* plan, const DevTables& dt, const void* grads, void* out, double max_norm,
                          float* norms, float* tensor_norms, float* coefs, hipStream_t st) {
  return launch(plan, kSmall, cl_small<GT, N>, dim3(static_cast<unsigned>(plan->n_slices)), dim3(kSmallThreads), st,
                dt.items, int(plan->items.size()), dt.item_layers, int(plan->layers.size()),
                static_cast<const GT*>(grads), static_cast<GT*>(out), plan->worker_stride, max_norm, norms,
                tensor_norms, coefs);
}

struct Norm {
  const void* grads;
  float *norms, *tensor_norms;

  template <typename GT, typename N>
  psgd_status enqueue(psgd_clip_plan* plan, const DevTables& dt, char* ws, hipStream_t st) const {
    if (small(plan, kSmallNorm))
      return enqueue_small<GT, N>(plan, dt, grads, nullptr, INFINITY, norms, tensor_norms, nullptr, st);
    const psgd_status s =
        enqueue_partials<GT, N>(plan, dt, grads, tensor_norms != nullptr, false, AwArgs{}, ws, st);
    return s != PSGD_OK ? s
                        : enqueue_final<N>(plan, dt, INFINITY, norms, tensor_norms, nullptr, AwArgs{}, ws, st);
  }
};

struct Clip {
  const void* grads;
  void* out;
  double max_norm;
  float *norms, *coefs;

  template <typename GT, typename N>
  psgd_status enqueue(psgd_clip_plan* plan, const DevTables& dt, char* ws, hipStream_t st) const {
    if (small(plan, kSmallClip))
      return enqueue_small<GT, N>(plan, dt, grads, out, max_norm, norms, nullptr, coefs, st);
    psgd_status s = enqueue_partials<GT, N>(plan, dt, grads, false, true, AwArgs{}, ws, st);
    if (s == PSGD_OK && !fold(plan)) s = enqueue_final<N>(plan, dt, max_norm, norms, nullptr, coefs, AwArgs{}, ws, st);
    if (s != PSGD_OK) return s;
    const int n_parts = int(plan->tiles.size()) * (kTile / (kThreads * kUnit<GT>));
    const int per = grads == out ? kInPlaceParts : 1;
    const dim3 grid(static_cast<unsigned>((n_parts + per - 1) / per), static_cast<unsigned>(plan->n_slices));
    return launch(plan, kScale, fold(plan) ? cl_scale<GT, N, true> : cl_scale<GT, N, false>, grid, dim3(kThreads), st,
                  dt.tiles, n_parts, static_cast<const GT*>(grads), static_cast<GT*>(out), plan->worker_stride,
                  coef_args<N>(plan, max_norm, norms, coefs, ws));
  }
};

struct Adamw {
  const void* update;
  float *params, *exp_avg, *exp_avg_sq;
  uint16_t* copy;
  int64_t* step;
  float* norm;
  double max_norm;
  AwConfig cf;
  AwArgs aw;

  template <typename GT, typename N>
  psgd_status enqueue(psgd_clip_plan* plan, const DevTables& dt, char* ws, hipStream_t st) const {
    const bool clip = max_norm > 0.0, folded = clip && fold(plan);
    if (small(plan, kSmallAdamw))
      return clip ? launch_small<GT>(cl_small_adamw<GT, N, true>, plan, dt, st)
                  : launch_small<GT>(cl_small_adamw<GT, L2, false>, plan, dt, st);
    psgd_status s = PSGD_OK;
    if (clip) s = enqueue_partials<GT, N>(plan, dt, update, false, true, folded ? aw : AwArgs{}, ws, st);
    if (s == PSGD_OK && !folded) s = enqueue_final<N>(plan, dt, max_norm, norm, nullptr, nullptr, aw, ws, st);
    if (s != PSGD_OK) return s;
    if (!clip) return launch_parts<GT, L2>(cl_adamw<GT, L2, 0>, plan, dt, ws, st);
    return folded ? launch_parts<GT, N>(cl_adamw<GT, N, 2>, plan, dt, ws, st)
                  : launch_parts<GT, N>(cl_adamw<GT, N, 1>, plan, dt, ws, st);
  }

  template <typename GT, typename K>
  psgd_status launch_small(K kernel, psgd_clip_plan* plan, const DevTables& dt, hipStream_t st) const {
    return launch(plan, kSmallAw, kernel, dim3(1), dim3(kSmallThreads), st, dt.items, int(plan->items.size()),
                  static_cast<const GT*>(update), params, exp_avg, exp_avg_sq, copy, cf, aw, max_norm, norm, step);
  }

  template <typename GT, typename N, typename K>
  psgd_status launch_parts(K kernel, psgd_clip_plan* plan, const DevTables& dt, char* ws, hipStream_t st) const {
    const dim3 grid(static_cast<unsigned>(plan->tiles.size()) * (kTile / (kThreads * 4)));
    return launch(plan, kAdamw, kernel, grid, dim3(kThreads), st, dt.tiles, static_cast<const GT*>(update), params,
                  exp_avg, exp_avg_sq, copy, static_cast<const AwState*>(aw.state), cf,
                  coef_args<N>(plan, max_norm, norm, nullptr, ws), step);
  }
};

template <typename Call>
psgd_status enqueue(psgd_clip_plan* plan, int kind, const Call& call, const DevTables& dt, void* workspace,
                    hipStream_t st) {
  char* ws = static_cast<char*>(workspace);
  const bool bf = plan->dtype == PSGD_BF16;
  if (kind == PSGD_NORM_MAX)
    return bf ? call.template enqueue<uint16_t, Max>(plan, dt, ws, st)
              : call.template enqueue<float, Max>(plan, dt, ws, st);
  return bf ? call.template enqueue<uint16_t, L2>(plan, dt, ws, st) : call.template enqueue<float, L2>(plan, dt, ws, st);
}

}  // namespace
}  // namespace clip
}  // namespace psgd

using namespace psgd;
using namespace psgd::clip;

extern "C" psgd_status psgd_clip_plan_create(const psgd_layer* layers, int32_t n_layers, int32_t n_slices,
                                             psgd_dtype grad_dtype, uint32_t flags, psgd_clip_plan** out) {
  if (out == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: out is NULL");
  *out = nullptr;
  if (layers == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: layers is NULL");
  if (n_layers < 1) return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: n_layers must be >= 1");
  if (n_slices < 1 || n_slices > 65535)
    return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: n_slices must be in 1..65535");
  if (grad_dtype != PSGD_F32 && grad_dtype != PSGD_BF16)
    return refuse(PSGD_ERR_UNSUPPORTED, "psgd_clip_plan_create: unknown grad_dtype");
  if (flags != 0) return refuse(PSGD_ERR_UNSUPPORTED, "psgd_clip_plan_create: unknown flag bits");
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
        plan = nullptr;
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
      if (int64_t(plan->tiles.size()) > kMaxTiles) {
        delete plan;
        plan = nullptr;
        return fail(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_create: too many tiles");
      }
      plan->layers.push_back(L);
      plan->numel += numel;
      off = (off + numel + kAlignElems - 1) / kAlignElems * kAlignElems;
    }
    plan->worker_stride = off;
    // Runs of about equal cost, so that the workgroups of a launch end together.
    const int64_t n_tiles = int64_t(plan->tiles.size());
    const int64_t n_runs = std::min(n_tiles, kMaxRuns);
    int64_t cost = 0, done = 0;
    for (const ClTile& t : plan->tiles) cost += t.len + kTileCost;
    ClRun run{0, 0};
    for (int64_t i = 0; i < n_tiles; ++i) {
      done += plan->tiles[size_t(i)].len + kTileCost;
      run.tile1 = int32_t(i + 1);
      const int64_t made = int64_t(plan->runs.size()) + 1;
      if (i + 1 == n_tiles || (made < n_runs && done * n_runs >= cost * made)) {
        plan->runs.push_back(run);
        run.tile0 = run.tile1;
      }
    }
    // A small plan's tensors in items.
    int64_t n_items = 0;
    for (const psgd_clip_layer_info& li : plan->info) n_items += (li.numel + kItem - 1) / kItem;
    if (n_items <= kMaxItems)
      for (const psgd_clip_layer_info& li : plan->info) {
        const int32_t item0 = int32_t(plan->items.size());
        for (int64_t b = 0; b < li.numel; b += kItem)
          plan->items.push_back(ClItem{int32_t(li.offset + b), int32_t(std::min<int64_t>(kItem, li.numel - b)),
                                       li.rows > 1 && li.cols > 1 ? 1 : 0, 0});
        plan->item_layers.push_back(ClLayer{item0, int32_t(plan->items.size()) - item0});
      }
    uint64_t ws = 0;
    plan->ws_tile = ws;  // one partial per tile and slice
    ws = a256(ws + uint64_t(n_slices) * uint64_t(n_tiles) * sizeof(double));
    plan->ws_run = ws;  // one per run and slice
    ws = a256(ws + uint64_t(n_slices) * plan->runs.size() * sizeof(double));
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
  if (plan == nullptr || out == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_sizes: NULL argument");
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
  if (plan == nullptr || out == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_layer_info: NULL argument");
  if (layer < 0 || size_t(layer) >= plan->info.size())
    return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_layer_info: layer index out of range");
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
      st = refuse(PSGD_ERR_HIP, "psgd_clip_plan_destroy: hipFree of the device tables failed");
    }
    if (have && cur != kv.first) (void)hipSetDevice(cur);
  }
  delete plan;
  return st;
}

extern "C" psgd_status psgd_clip_plan_set_timing(psgd_clip_plan* plan, int32_t enable) {
  if (plan == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_set_timing: plan is NULL");
  plan->timing = enable != 0;
  return PSGD_OK;
}

extern "C" psgd_status psgd_clip_plan_kernel_stats(psgd_clip_plan* plan, psgd_kernel_stat* out, int32_t capacity,
                                                   int32_t* count, int32_t reset) {
  if (plan == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_kernel_stats: plan is NULL");
  if (capacity > 0 && out == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_clip_plan_kernel_stats: out is NULL");
  psgd_status st = PSGD_OK;
  try {
    st = collect_timings("psgd_clip_plan_kernel_stats", plan->pending, plan->event_pool, plan->stats);
  } catch (...) {
    return no_memory();
  }
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
    const ArgSpan spans[] = {
        {"grads", grads, S * uint64_t(plan->worker_stride) * gb, 16, false},
        {"norms", norms, S * 4, 4, false},
        {"tensor_norms", tensor_norms, S * plan->layers.size() * 4, 4, true},
        {"workspace", workspace, plan->workspace_bytes, 16, false},
    };
    if ((s = check_spans(fn, spans, 4)) != PSGD_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    DevTables dt{};
    if ((s = device_tables(fn, plan, st, &dt)) != PSGD_OK) return s;
    return enqueue(plan, kind, Norm{grads, norms, tensor_norms}, dt, workspace, st);
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
    const ArgSpan spans[] = {
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
    return enqueue(plan, kind, Clip{grads, out, double(max_norm), norms, coefs}, dt, workspace, st);
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
    const ArgSpan spans[] = {
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
    const AwArgs aw{cf.lr, cf.beta1, cf.beta2, step,
                    reinterpret_cast<AwState*>(static_cast<char*>(workspace) + plan->ws_aw)};
    const float beta1 = float(cf.beta1), beta2 = float(cf.beta2);
    const AwConfig ac{beta1, float(cf.beta1 - double(beta1)), float(1.0 - cf.beta1),
                      beta2, float(cf.beta2 - double(beta2)), float(1.0 - cf.beta2),
                      float(cf.eps), float(cf.lr * cf.weight_decay),
                      (cf.flags & PSGD_ADAMW_DECAY_MATRICES_ONLY) ? 1 : 0,
                      (cf.flags & PSGD_ADAMW_SKIP_NONFINITE) ? 1 : 0};
    const Adamw call{update, params, exp_avg, exp_avg_sq, static_cast<uint16_t*>(params_bf16), step, norm,
                     cf.max_norm, ac, aw};
    return enqueue(plan, clipped ? cf.norm_kind : int(PSGD_NORM_L2), call, dt, workspace, st);
  } catch (...) {
    return no_memory();
  }
}
