// Embedding, softmax cross entropy and dropout around a language model's table: the gfx950
// kernels and the host side of psgd_lm.h.
//
// Products run on 16-bit matrix cores from packed operands: 64 x 64 blocks of bf16 or fp16,
// 8 KB each and one after the other, so that a tile is a few contiguous runs of 16-byte loads,
// zero past a matrix's edges, so that no product loop has an edge of its own.  Operands in
// float32 are held in parts, and the loop over the contraction runs once per product of two
// parts:
// - for the scores every row, of x and of the table, is scaled by a power of two of its own,
//   which leaves the contraction, and held as two fp16 parts, x = h + l / 2048; a product of
//   two of them is h l' + l h' (divided by 2048) + h h';
// - for the products with g, whose contraction runs over rows, of any sizes, they and g are
//   three bf16 parts, x = h + m + l: every entry has its 24 bits, whatever the others are.  The
//   six products above 2^-24 take part.
//
//   lm_peak    the powers of two of float32 operands' rows
//   lm_pack    x (through dropout, zero where a row does not count) and the table, packed; the
//              counted rows of every worker
//   lm_scores  tiles of T drop(x)^T: their rows' maximum and sum (loss), or g of their entries,
//              packed (gradient)
//   lm_rows    lse and loss of every row from the tiles' maxima and sums
//   lm_mean    the workers' means
//   lm_products  g T, added up over the pieces of the vocabulary in float32, and g^T drop(x)
//              into the gradient slices
//   lm_dx_out  the sum of g T's splits, through dropout
//   lm_embed   rows of the table
//   lm_sort, lm_merge  every worker's (token, row) pairs in order; zeroes tables on the side
//   lm_sum, lm_join  the table gradient from runs of these pairs
//   lm_dropout
//
// No kernel waits for another workgroup, no atomics, no state is kept between calls.

#include <hip/hip_runtime.h>
#include <hip/hip_ext.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <string>
#include <type_traits>
#include <vector>

#include "plan.hpp"
#include "psgd_lm.h"

namespace psgd {
namespace lm {

constexpr int kBlk = 64;           // rows and columns of a packed block
constexpr int kBlkElems = kBlk * kBlk;
constexpr int64_t kMaxBlocks = int64_t(1) << 23;  // of x or the table: launches of 256 threads each stay below 2^32
constexpr int64_t kMaxDim = int64_t(1) << 23;     // strips of columns are a launch's second dimension
constexpr int kTile = 4;           // blocks per side of a workgroup's tile
constexpr int kThreads = 256;      // of the kernels around the products
constexpr int kGroup = 16;         // row blocks that take turns on one vocabulary tile (lm_scores)
constexpr int64_t kFewStats = 16384;  // maxima and sums of a worker that one workgroup takes in
constexpr int kSplitBlocks = 8;    // vocabulary blocks of a split of lm_products' dx, at least
// g of one piece of the vocabulary.  256, 512, 1024, 2048 MB: gradients of 33,278 x 650, 8 x 700
// rows float32 4.47, 4.39, 4.27, 4.35 ms; of 65,536 x 2048, 2 x 2048 rows bfloat16 3.22, 3.20,
// 3.21, 3.20 (64 MB: 3.65; each piece adds to all of dx, and the last tiles of a launch run alone).
constexpr int64_t kPieceBytes = int64_t(512) << 20;
constexpr int64_t kStatBytes = int64_t(64) << 20;    // maxima and sums of one chunk of rows
constexpr int kSortMax = 1024;     // pairs sorted by one workgroup
constexpr int kSortThreads = 512;
constexpr int kRun = 16;           // sorted pairs summed by one wave ...
constexpr int kRunLoads = 8;       // ... whose rows are loaded so many at a time
constexpr int kJoinWaves = 4;      // waves that join a token's runs
constexpr int kZeroUnits = 4;      // 16-byte stores of a thread that zeroes
constexpr int64_t kZeroGroups = 65536;  // workgroups that zero, at most: HIP takes below 2^32 threads a launch
constexpr int64_t kMostGroups = int64_t(1) << 23;  // workgroups of a launch of psgd_dropout: HIP takes below 2^32 threads
constexpr int64_t kMostEntries = int64_t(1) << 41;  // of psgd_dropout, below it: 256 launches at most

enum KernelId {
  kPeak = 0, kPack, kScores, kRows, kMean, kProducts, kDxOut, kEmbed, kSort, kMerge, kSum, kJoin, kNumK
};
const char* const kNames[kNumK] = {"lm_peak", "lm_pack", "lm_scores", "lm_rows", "lm_mean", "lm_products", "lm_dx_out", "lm_embed",
                                   "lm_sort", "lm_merge", "lm_sum", "lm_join"};

}  // namespace lm
}  // namespace psgd

struct psgd_lm_plan {
  int32_t n_layers = 0, n_workers = 0, table = 0;
  psgd_dtype act = PSGD_F32, grad = PSGD_F32;
  int64_t vocab = 0, dim = 0, rows = 0, worker_stride = 0, offset = 0;
  int32_t vb = 0, db = 0;        // blocks of the table
  int32_t tb = 0, tw = 0;        // blocks of all rows together, and of one worker's rows
  int32_t piece = 0, splits = 1;  // blocks of the vocabulary per piece, splits of dx's sum over one
  int32_t chunk = 0;             // row blocks per chunk in psgd_lm_loss
  bool direct = false;           // the table is read as it is
  bool loss_small = false, scores_small = false, grad_small = false;  // which tiles are the small ones
  uint64_t ws_x = 0, ws_w = 0, ws_x3 = 0, ws_w3 = 0, ws_x_exps = 0, ws_w_exps = 0, ws_info = 0, ws_count = 0;
  uint64_t ws_stat = 0, ws_hit = 0, ws_g = 0, ws_dx = 0;
  uint64_t ws_key = 0, ws_key2 = 0, ws_part = 0, workspace_bytes = 0;
  bool timing = false;
  std::vector<psgd::PendingTiming> pending;
  std::vector<hipEvent_t> event_pool;
  psgd::KernelStat stats[psgd::lm::kNumK];
};

namespace psgd {
namespace lm {
namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef int32_t i4v __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ numbers
__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ uint16_t narrow_bits(float x) { return __builtin_bit_cast(uint16_t, __bf16(x)); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = narrow_bits(x); }

// N elements from or to an address that is aligned to its type only.
template <int N, typename T>
__device__ __forceinline__ void load(const T* p, float (&x)[N]) {
  T v[N];
  __builtin_memcpy(v, p, sizeof(v));
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = widen(v[i]);
}
template <int N>
__device__ __forceinline__ void store(float* p, const float (&x)[N]) {
  __builtin_memcpy(p, x, sizeof(x));
}
template <int N>
__device__ __forceinline__ void store(uint16_t* p, const float (&x)[N]) {
  uint16_t v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = narrow_bits(x[i]);
  __builtin_memcpy(p, v, sizeof(v));
}

// x = h + m + l, bf16 each, every one the nearest to what is left.  A number past the largest
// bf16 takes that as its first part; infinities and NaN have one part.
__device__ __forceinline__ void split3(float x, uint16_t (&part)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint16_t b = narrow_bits(x);
    if ((b & 0x7fff) == 0x7f80 && (__float_as_uint(x) & 0x7fffffffu) < 0x7f800000u) b -= 1;
    part[i] = b;
    x = (b & 0x7f80) == 0x7f80 ? 0.f : x - widen(b);
  }
}

// The two fp16 parts of x, |x| < 2^15 or not finite: x = h + l / 2048.
__device__ __forceinline__ void split16(float x, uint16_t& h, uint16_t& l) {
  const _Float16 a = _Float16(x);
  const float rest = fabsf(x) < 65536.f ? (x - float(a)) * 2048.f : 0.f;
  h = __builtin_bit_cast(uint16_t, a);
  l = __builtin_bit_cast(uint16_t, _Float16(rest));
}

struct Drop {
  uint64_t keep_from;  // an entry is kept if its word is at least this; 0 with scale 1: no dropout
  uint32_t key0, key1;
  const int64_t* step;
  float scale;
  int32_t on;
};

// Philox4x32-10 with counter (i, step): the words of entries 4i to 4i + 3.
__device__ __forceinline__ void philox(uint64_t i, uint64_t step, uint32_t k0, uint32_t k1, uint32_t (&w)[4]) {
  uint32_t c0 = uint32_t(i), c1 = uint32_t(i >> 32), c2 = uint32_t(step), c3 = uint32_t(step >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
    c0 = uint32_t(b >> 32) ^ c1 ^ k0;
    c1 = uint32_t(b);
    c2 = uint32_t(a >> 32) ^ c3 ^ k1;
    c3 = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

__device__ __forceinline__ uint64_t step_of(const Drop& d) { return d.step != nullptr ? uint64_t(*d.step) : 0u; }

// Entries i to i + N - 1 through dropout, the kept ones times `scale`.
template <int N>
__device__ __forceinline__ void drop(const Drop& d, uint64_t step, uint64_t i, float scale, float (&x)[N]) {
  const int lead = int(i & 3);
#pragma unroll
  for (int g = 0; g < (N + 6) / 4; ++g) {
    if (4 * g >= N + lead) break;
    uint32_t w[4];
    philox(i / 4 + g, step, d.key0, d.key1, w);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int at = e + lead - 4 * g;  // its word, if in 0..3
      if (at >= 0 && at < 4) {
        const uint32_t v = at == 0 ? w[0] : at == 1 ? w[1] : at == 2 ? w[2] : w[3];
        x[e] = uint64_t(v) >= d.keep_from ? x[e] * scale : 0.f;
      }
    }
  }
}

// ------------------------------------------------------------------ packed operands
// A packed matrix: block (r, c) is 4096 elements at (r * cb + c) * 4096 of every part.
// Inside a block element (r, c) is at 64 r + 8 (c / 8 ^ turn(r)) + c % 8: the 16-byte pieces
// of a row are turned so that neither the reads along rows (16 rows, one piece each) nor the
// transposing ones (4 rows, two pieces each) meet on a bank.
//
// A bfloat16 table whose rows are whole blocks (dim a multiple of 64) needs no packing: its
// blocks are gathered, 16 bytes a lane, as they go into LDS.  Against packing it first,
// 131,072 x 2048 for 4096 rows: packing it took 228 of
// the loss's 2081 us.
struct Mat {
  const uint16_t* p;
  int64_t part;  // elements between parts
  int32_t rb, cb;
  int32_t last;  // not packed: its last row
};

__device__ __forceinline__ int turn(int r) { return ((r >> 1) & 1) << 2 | ((r >> 2) & 1) << 1 | ((r >> 3) & 1); }

// The part products of one contraction, one after the other: product i takes part
// a >> 4 i & 15 of one operand and b >> 4 i & 15 of the other.
struct Parts {
  uint32_t n, a, b;
};

typedef __attribute__((address_space(3))) uint16_t lds_t;

// C += A B over blocks [k0, k1) (at least one; of the last, `tail` steps of 16) for a tile of
// WM FM x WN FN pieces of 32 x 32, each wave FM x FN of them.  TA, TB: the operand's
// contraction runs along its blocks' rows instead of along their columns; it is then read
// from LDS with the transposing load.  RA, RB: the operand is not packed.  Two LDS stages: the
// blocks of the next step are on their way from memory straight into one while the matrix
// cores work on the other (three and four stages of small tiles ran alike).
template <int WM, int WN, int FM, int FN, bool TA, bool TB, bool F16, bool RA, bool RB>
struct Gemm {
  static_assert((FM == 4 && FN == 2) || (FM == 1 && FN == 1), "what the LDS reads are written out for");
  static constexpr int kWaves = WM * WN, kT = kWaves * 64;
  static constexpr int kA = WM * FM / 2, kB = WN * FN / 2;  // blocks of the tile's sides
  static constexpr int kPer = kBlkElems / 8 / kT;           // 16-byte pieces of a block per thread
  static constexpr int kStage = (kA + kB) * kBlkElems;
  static constexpr int kLds = 2 * kStage;
  // The small score tiles have registers for a sum of its own for each quarter of a block's
  // steps: shorter sums round less, and an error of a score of 40 reaches exp(s - lse) whole.
  // Distance of table gradients from float64, 1, 2 and 4 sums: 2 x 19 rows of 21,396 x 1532 8.0,
  // 4.7, 2.1e-6; 3 x 127 rows of 1429 x 1323 8.2, 4.1, 2.6e-6; 403 rows' loss over 14,070 x 259
  // in float32 takes 46, 46, 48 us.
  static constexpr int kSums = FM == 1 && !TA && !TB ? 4 : 1;
  static constexpr int kRowsA = FM * 32, kRowsB = FN * 32;  // of a wave
  typedef f16v Acc[FM][FN];
  static constexpr int kFM = FM, kFN = FN, kWN = WN, kWM = WM;
  static_assert(kPer * kT * 8 == kBlkElems, "a block is a whole number of pieces per thread");

  // Block (side, k) of an operand into LDS.
  template <bool T, bool R>
  static __device__ __forceinline__ void fetch(const Mat& m, int part, int side, int k, lds_t* s) {
    typedef __attribute__((address_space(1))) void from_t;
    typedef __attribute__((address_space(3))) void to_t;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = T ? k : min(side, m.rb - 1), c = T ? min(side, m.cb - 1) : k;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = j * kT + int(threadIdx.x);
      const uint16_t* g;
      if constexpr (R)
        g = m.p + int64_t(min(r * kBlk + i / 8, m.last)) * (m.cb * kBlk) + c * kBlk + ((i % 8 ^ turn(i / 8)) << 3);
      else
        g = m.p + part * m.part + (int64_t(r) * m.cb + c) * kBlkElems + i * 8;
      __builtin_amdgcn_global_load_lds((from_t*)g, (to_t*)(s + (j * kT + wave * 64) * 8), 16, 0, 0);
    }
  }

  // Operand pieces of step kk, 32 x 16 each: row (column) lane % 32, contraction 8 (lane / 32)
  // on.  at: a lane's byte address in every step.
  static __device__ __forceinline__ void rows_at(int f0, int lane, uint32_t (&at)[4]) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      at[kk] = 2 * ((f0 >> 1) * kBlkElems + ((f0 & 1) * 32 + (lane & 31)) * kBlk + (((kk * 2 + (lane >> 5)) ^ turn(lane)) << 3));
  }

  static __device__ __forceinline__ void rows_of(uint32_t a, bf8 (&x)[4]) {
    asm volatile(
        "ds_read_b128 %0, %4\n"
        "ds_read_b128 %1, %4 offset:4096\n"
        "ds_read_b128 %2, %4 offset:8192\n"
        "ds_read_b128 %3, %4 offset:12288\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
        : "v"(a)
        : "memory");
  }

  static __device__ __forceinline__ void rows_of(uint32_t a, bf8 (&x)[1]) {
    asm volatile(
        "ds_read_b128 %0, %1\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0])
        : "v"(a)
        : "memory");
  }

  static __device__ __forceinline__ void rows_of(uint32_t a, uint32_t b, bf8 (&x)[1], bf8 (&y)[1]) {
    asm volatile(
        "ds_read_b128 %0, %2\n"
        "ds_read_b128 %1, %3\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(y[0])
        : "v"(a), "v"(b)
        : "memory");
  }

  static __device__ __forceinline__ void rows_of(uint32_t a, uint32_t b, bf8 (&x)[4], bf8 (&y)[2]) {
    asm volatile(
        "ds_read_b128 %0, %6\n"
        "ds_read_b128 %1, %6 offset:4096\n"
        "ds_read_b128 %2, %6 offset:8192\n"
        "ds_read_b128 %3, %6 offset:12288\n"
        "ds_read_b128 %4, %7\n"
        "ds_read_b128 %5, %7 offset:4096\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(y[0]), "=&v"(y[1])
        : "v"(a), "v"(b)
        : "memory");
  }

  // The same from an operand whose contraction runs along the blocks' rows: a transposing read
  // takes 4 rows x 16 columns per 16 lanes.  at[p][j]: a lane's byte addresses for pieces
  // f0 + p of a block and for the two halves of its eight contraction slots.
  static __device__ __forceinline__ void columns_at(int f0, int lane, uint32_t (&at)[2][2]) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = (lane >> 5) * 8 + j * 4 + ((lane & 15) >> 2);
        const int c = ((f0 + p) & 1) * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
        at[p][j] = 2 * ((f0 >> 1) * kBlkElems + k * kBlk + ((c ^ turn(k)) << 3) + (lane & 1) * 4);
      }
  }

  static __device__ __forceinline__ bf8 join(const s4v& lo, const s4v& hi) {
    s8v v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
    return __builtin_bit_cast(bf8, v);
  }

  // The reads are written out because the compiler makes its own transposing reads wait for
  // every load into LDS that is under way; each block waits for its reads before it ends.
  template <int OFF>
  static __device__ __forceinline__ void columns_of(const uint32_t (&b)[2][2], bf8 (&y)[2]) {
    s4v v[4];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4 offset:%8\n"
        "ds_read_b64_tr_b16 %1, %5 offset:%8\n"
        "ds_read_b64_tr_b16 %2, %6 offset:%8\n"
        "ds_read_b64_tr_b16 %3, %7 offset:%8\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(b[0][0]), "v"(b[0][1]), "v"(b[1][0]), "v"(b[1][1]), "n"(OFF)
        : "memory");
    y[0] = join(v[0], v[1]);
    y[1] = join(v[2], v[3]);
  }

  template <int OFF>
  static __device__ __forceinline__ void columns_of(const uint32_t (&b)[2][2], bf8 (&y)[1]) {
    s4v v[2];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %2 offset:%4\n"
        "ds_read_b64_tr_b16 %1, %3 offset:%4\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1])
        : "v"(b[0][0]), "v"(b[0][1]), "n"(OFF)
        : "memory");
    y[0] = join(v[0], v[1]);
  }

  template <int OFF>
  static __device__ __forceinline__ void columns_of(const uint32_t (&a)[2][2], const uint32_t (&b)[2][2], bf8 (&x)[1],
                                                    bf8 (&y)[1]) {
    s4v v[4];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4 offset:%8\n"
        "ds_read_b64_tr_b16 %1, %5 offset:%8\n"
        "ds_read_b64_tr_b16 %2, %6 offset:%8\n"
        "ds_read_b64_tr_b16 %3, %7 offset:%8\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(a[0][0]), "v"(a[0][1]), "v"(b[0][0]), "v"(b[0][1]), "n"(OFF)
        : "memory");
    x[0] = join(v[0], v[1]);
    y[0] = join(v[2], v[3]);
  }

  template <int OFF>
  static __device__ __forceinline__ void columns_of(const uint32_t (&a)[2][2], const uint32_t (&b)[2][2], bf8 (&x)[4],
                                                    bf8 (&y)[2]) {
    s4v v[12];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %12 offset:%20\n"
        "ds_read_b64_tr_b16 %1, %13 offset:%20\n"
        "ds_read_b64_tr_b16 %2, %14 offset:%20\n"
        "ds_read_b64_tr_b16 %3, %15 offset:%20\n"
        "ds_read_b64_tr_b16 %4, %12 offset:%21\n"
        "ds_read_b64_tr_b16 %5, %13 offset:%21\n"
        "ds_read_b64_tr_b16 %6, %14 offset:%21\n"
        "ds_read_b64_tr_b16 %7, %15 offset:%21\n"
        "ds_read_b64_tr_b16 %8, %16 offset:%20\n"
        "ds_read_b64_tr_b16 %9, %17 offset:%20\n"
        "ds_read_b64_tr_b16 %10, %18 offset:%20\n"
        "ds_read_b64_tr_b16 %11, %19 offset:%20\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7]),
          "=&v"(v[8]), "=&v"(v[9]), "=&v"(v[10]), "=&v"(v[11])
        : "v"(a[0][0]), "v"(a[0][1]), "v"(a[1][0]), "v"(a[1][1]), "v"(b[0][0]), "v"(b[0][1]), "v"(b[1][0]), "v"(b[1][1]),
          "n"(OFF), "n"(OFF + 2 * kBlkElems)
        : "memory");
#pragma unroll
    for (int f = 0; f < 4; ++f) x[f] = join(v[2 * f], v[2 * f + 1]);
#pragma unroll
    for (int f = 0; f < 2; ++f) y[f] = join(v[8 + 2 * f], v[9 + 2 * f]);
  }

  static __device__ __forceinline__ void sweep(const Mat& a, int a0, const Mat& b, int b0, int k0, int k1, int tail, const Parts& parts,
                                               lds_t* sm, Acc& acc) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wa = (wave / WN) * FM, wb = (wave % WN) * FN;
    int k = k0;
    uint32_t pa = parts.a, pb = parts.b;
    auto stage = [&](lds_t* s) {
#pragma unroll
      for (int i = 0; i < kA; ++i) fetch<TA, RA>(a, pa & 15, a0 + i, k, s + i * kBlkElems);
#pragma unroll
      for (int i = 0; i < kB; ++i) fetch<TB, RB>(b, pb & 15, b0 + i, k, s + (kA + i) * kBlkElems);
      if (++k == k1) k = k0, pa >>= 4, pb >>= 4;
    };
    uint32_t at_a[2][2], at_b[2][2];
    columns_at(wa, lane, at_a);
    columns_at(wb, lane, at_b);
    uint32_t at_ra[4], at_rb[4];
    rows_at(wa, lane, at_ra);
    rows_at(wb, lane, at_rb);
    Acc sums[kSums] = {};
    auto multiply = [&](uint32_t base, const uint32_t (&ca)[2][2], const uint32_t (&cb)[2][2], auto kk) {
      constexpr int K = decltype(kk)::value;
      bf8 x[FM], y[FN];
      if constexpr (TA) {
        columns_of<K * 32 * kBlk>(ca, cb, x, y);
      } else if constexpr (TB) {
        rows_of(base + at_ra[K], x);
        columns_of<K * 32 * kBlk>(cb, y);
      } else {
        rows_of(base + at_ra[K], base + 2 * kA * kBlkElems + at_rb[K], x, y);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          f16v& a = kSums > 1 ? sums[K % kSums][i][j] : acc[i][j];
          if constexpr (F16)
            a = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, x[i]), __builtin_bit_cast(h8, y[j]), a, 0, 0, 0);
          else
            a = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[i], y[j], a, 0, 0, 0);
        }
    };
    const int steps = int(parts.n) * (k1 - k0);
    stage(sm);
    int at = k0;  // the block of the current step
    auto step = [&](const lds_t* cur, lds_t* next, bool more) {
      __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wave's part of `cur` is there
      // everybody's is, and nobody reads `next` any more: reads of LDS end with a wait of their own
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (more) stage(next);
      __builtin_amdgcn_sched_barrier(0);
      const uint32_t base = uint32_t(uintptr_t(cur));
      uint32_t ca[2][2], cb[2][2];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j) ca[p][j] = base + at_a[p][j], cb[p][j] = base + 2 * kA * kBlkElems + at_b[p][j];
      const int n = ++at == k1 ? tail : 4;
      if (at == k1) at = k0;
      multiply(base, ca, cb, std::integral_constant<int, 0>());
      if (n > 1) multiply(base, ca, cb, std::integral_constant<int, 1>());
      if (n > 2) multiply(base, ca, cb, std::integral_constant<int, 2>());
      if (n > 3) multiply(base, ca, cb, std::integral_constant<int, 3>());
      __builtin_amdgcn_sched_barrier(0);
    };
    for (int left = steps;;) {
      step(sm, sm + kStage, left > 1);
      if (--left == 0) break;
      step(sm + kStage, sm, left > 1);
      if (--left == 0) break;
    }
    __syncthreads();
    if constexpr (kSums > 1) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] += (sums[0][i][j] + sums[1][i][j]) + (sums[2][i][j] + sums[3][i][j]);
    }
  }

  // The whole product.  With fp16 parts the products with a low part come first and are
  // scaled back before the product of the high parts is added.
  static __device__ __forceinline__ void run(const Mat& a, int a0, const Mat& b, int b0, int k0, int k1, int tail,
                                             const Parts& parts, lds_t* sm, Acc& acc) {
    if constexpr (!F16) {
      sweep(a, a0, b, b0, k0, k1, tail, parts, sm, acc);
    } else {
      if (parts.n > 1) {
        sweep(a, a0, b, b0, k0, k1, tail, Parts{parts.n - 1, parts.a, parts.b}, sm, acc);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] *= 1.f / 2048.f;
      }
      sweep(a, a0, b, b0, k0, k1, tail, Parts{1, 0, 0}, sm, acc);
    }
  }
};

// Accumulator i of a 32 x 32 piece: its row for this lane; its column is lane % 32.
__device__ __forceinline__ int acc_row(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

// ------------------------------------------------------------------ rows and packing
// What the score tiles need of a packed row.
struct RowInfo {
  int32_t target;  // -1: the row does not count
  float lse;
  int32_t exp;     // float32: the row's power of two
};

constexpr float kLog2e = 1.44269504f;

constexpr int kPeakGroups = 2048;  // workgroups of lm_peak: all that fit the chip at once

template <typename F>
__device__ __forceinline__ F block_sum(F x, F* sm) {
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = x;
  __syncthreads();
  F t = 0;
  for (int i = 0; i < int(blockDim.x) / 64; ++i) t += sm[i];
  __syncthreads();
  return t;
}

__device__ __forceinline__ bool counts(int64_t target, int64_t vocab) { return uint64_t(target) < uint64_t(vocab); }

// Largest finite magnitude (as its bits) that dropout leaves of the n entries at p, the first of
// them entry `first`, by threads `id` of `of`.
__device__ __forceinline__ uint32_t peak_of(const float* p, int64_t n, int id, int of, bool dropped, const Drop& d,
                                            uint64_t step, uint64_t first) {
  uint32_t m = 0;
  for (int64_t i = id * 4; i < n; i += of * 16) {
    float v[4][4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = i + k * of * 4;
      if (at + 4 <= n) {
        load<4>(p + at, v[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at + e < n) v[k][e] = p[at + e];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (dropped && i + k * of * 4 < n) drop<4>(d, step, first + uint64_t(i + k * of * 4), 1.f, v[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t u = __float_as_uint(v[k][e]) & 0x7fffffffu;
        m = max(m, u < 0x7f800000u ? u : 0u);
      }
    }
  }
  return m;
}

// The power of two of every row of the table (0 past the vocabulary, up to `padded` words) and
// of every row of x that counts: it brings the largest finite entry that dropout leaves into
// [2^14, 2^15), so the row's fp16 parts hold 22 bits of entries down to 2^-28 of that one.  One
// power for a whole matrix would let the largest entry of one row, or one that is dropped, take
// bits from every other worker's rows.  `lanes` lanes (a power of two up to 64) take a row.
// Bound by memory: 87 MB of table and 15 MB of x in 23 us, 25 through dropout.
__global__ __launch_bounds__(kThreads) void lm_peak(const float* table, int64_t vocab, int64_t padded, const float* x,
                                                    int64_t rows, int64_t dim, const int64_t* targets, int32_t lanes,
                                                    int32_t* w_exps, int32_t* x_exps, Drop d) {
  const int id = threadIdx.x & (lanes - 1), per = kThreads / lanes;
  const uint64_t step = d.on ? step_of(d) : 0;
  for (int64_t job = int64_t(blockIdx.x) * per + threadIdx.x / lanes; job < padded + rows; job += int64_t(gridDim.x) * per) {
    const bool of_x = job < rows;  // first, as dropout makes them the longer ones
    const int64_t r = of_x ? job : job - rows;
    uint32_t m = 0;
    if (of_x ? counts(targets[r], vocab) : r < vocab)
      m = peak_of((of_x ? x : table) + r * dim, dim, id, lanes, of_x && d.on, d, step, uint64_t(r) * uint64_t(dim));
    for (int o = lanes >> 1; o > 0; o >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), o)));
    if (id == 0) (of_x ? x_exps : w_exps)[r] = m != 0 ? 14 - ilogbf(__uint_as_float(m)) : 0;
  }
}

// What every row of a worker's g is multiplied by.
__device__ __forceinline__ float coef_of(const float* scale, const int32_t* count, int64_t w) {
  return count[w] > 0 ? float((scale != nullptr ? double(scale[w]) : 1.0) / double(count[w])) : 0.f;
}

struct PackArgs {
  const void *x, *table;
  Mat x_to, w_to;        // packed (p is written); w_to.p NULL: the table is read as it is
  Mat x3_to, w3_to;      // float32: their three bf16 parts; p NULL: not wanted
  int64_t rows;          // of x in each group, which starts at a block of its own ...
  int32_t blocks;        // ... of `blocks`
  int64_t worker_rows;   // how the targets are counted
  int64_t vocab;
  int32_t dim;
  const int64_t* targets;
  const float* lse;      // NULL for the loss
  RowInfo* info;
  int32_t* count;        // counted rows of every worker, or NULL
  const int32_t *x_exps, *w_exps;  // float32 operands
};

// One block per workgroup: those of x (through dropout, but not scaled: the products' results
// are; zero where a row does not count), those of the table, and after them one workgroup per
// worker that counts its rows.  Bound by memory: 33,278 x 650 and 5600 rows in float32, 102 MB
// read and 108 MB written, in 40 us; with the bf16 parts, 270 MB, in 72.
template <typename T>
__global__ __launch_bounds__(kThreads) void lm_pack(PackArgs p, Drop d) {
  const int32_t cb = p.x_to.cb;
  const int64_t n_x = int64_t(p.x_to.rb) * cb, n_w = p.w_to.p != nullptr ? int64_t(p.w_to.rb) * cb : 0;
  const int64_t job = blockIdx.x;
  if (job >= n_x + n_w) {
    __shared__ int32_t sm[kThreads / 64];
    const int64_t w = job - n_x - n_w;
    int32_t n = 0;
    for (int64_t i = threadIdx.x; i < p.worker_rows; i += kThreads) n += counts(p.targets[w * p.worker_rows + i], p.vocab) ? 1 : 0;
    n = block_sum(n, sm);
    if (threadIdx.x == 0) p.count[w] = n;
    return;
  }
  const bool of_x = job < n_x;
  const int64_t block = of_x ? job : job - n_x, rb = block / cb, blocks = of_x ? p.blocks : p.w_to.rb;
  const int64_t rows = of_x ? p.rows : p.vocab, w = rb / blocks, t0 = (rb % blocks) * kBlk;
  const int32_t c0 = int32_t(block % cb) * kBlk;
  const T* src = static_cast<const T*>(of_x ? p.x : p.table);
  const Mat &to = of_x ? p.x_to : p.w_to, &to3 = of_x ? p.x3_to : p.w3_to;
  const bool dropped = of_x && d.on;
  const uint64_t step = dropped ? step_of(d) : 0;
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int r = it * 32 + int(threadIdx.x) / 8, c = c0 + int(threadIdx.x % 8) * 8;
    const int64_t t = t0 + r, row = w * rows + t;
    bool on = t < rows;
    int32_t exp = 0;
    if (of_x) {
      const int64_t target = on ? p.targets[row] : -1;
      on = counts(target, p.vocab);
      if (sizeof(T) == 4 && on) exp = p.x_exps[row];
      if (c == 0) {
        p.info[rb * kBlk + r] = RowInfo{on ? int32_t(target) : -1, on && p.lse != nullptr ? p.lse[row] : 0.f, exp};
      }
    } else if (sizeof(T) == 4 && on) {
      exp = p.w_exps[t];
    }
    float x[8] = {};
    if (on && c < p.dim) {
      const T* from = src + row * p.dim + c;
      if (c + 8 <= p.dim) {
        load<8>(from, x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < p.dim) x[e] = widen(from[e]);
      }
      if (dropped) drop<8>(d, step, uint64_t(row) * uint64_t(p.dim) + uint64_t(c), 1.f, x);
    }
    const int64_t at = block * kBlkElems + r * kBlk + ((int(threadIdx.x % 8) ^ turn(r)) << 3);
    uint16_t* o = const_cast<uint16_t*>(to.p) + at;
    s8v h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint16_t a = 0, b = 0;
      if constexpr (sizeof(T) == 2) a = narrow_bits(x[e]);
      else split16(ldexpf(x[e], exp), a, b);
      h[e] = short(a), l[e] = short(b);
    }
    *reinterpret_cast<s8v*>(o) = h;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<s8v*>(o + to.part) = l;
      if (to3.p == nullptr) continue;
      s8v v[3];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint16_t part[3];
        split3(x[e], part);
#pragma unroll
        for (int i = 0; i < 3; ++i) v[i][e] = short(part[i]);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) *reinterpret_cast<s8v*>(const_cast<uint16_t*>(to3.p) + i * to3.part + at) = v[i];
    }
  }
}

// ------------------------------------------------------------------ scores
// Tile sizes: 256 x 256 by eight waves where that gives at least kFewTiles tiles, and else
// 64 x 64 by four, so that small problems still spread over the chip.  us a call for bounds of
// 64, 128, 256 and 512 tiles: loss of 8000 x 512, 512 rows 86, 24, 24, 24; of 16,000 x 300, 1024
// rows 31, 30, 45, 46; of 32,000 x 1024, 1024 rows 74, 75, 76, 128; gradients of 4000 x 300, 1000
// rows float32 126, 100, 100, 100; of 32,000 x 1024, 512 rows 129, 129, 153, 203.
constexpr int64_t kFewTiles = 128;

template <bool SMALL, bool TA, bool TB, bool F16, bool RA, bool RB>
using Tile = Gemm<2, SMALL ? 2 : 4, SMALL ? 1 : 4, SMALL ? 1 : 2, TA, TB, F16, RA, RB>;

// Workgroups are dealt to the eight XCDs in turn: place `id` of a list of `total` such that
// every XCD gets a contiguous part of it and neighbours share its L2; -1 past the end.
__device__ __forceinline__ int64_t place_of(int64_t id, int64_t total) {
  const int64_t per = (total + 7) / 8, at = (id % 8) * per + id / 8;
  return at < total && id / 8 < per ? at : -1;
}

// In that list `group` row tiles take turns on each vocabulary tile.
__device__ __forceinline__ bool tile_at(int64_t id, int64_t n_v, int64_t n_t, int group, int& v, int& t) {
  const int64_t at = place_of(id, n_v * n_t);
  if (at < 0) return false;
  const int64_t g = at / (n_v * group), in = at % (n_v * group);
  const int64_t width = min(int64_t(group), n_t - g * group);
  v = int(in / width);
  t = int(g * group + in % width);
  return true;
}

struct ScoreArgs {
  Mat w, x;
  Parts parts;
  int32_t tail;          // steps of 16 in the last block of a row
  int32_t v0, v1;        // vocabulary blocks [v0, v1) of this launch
  int32_t t0, t1;        // row blocks
  int64_t vocab;
  const RowInfo* info;   // from row block 0 on
  const int32_t* w_exps;  // float32 operands
  float x_scale;         // dropout's
  float2* stat;          // loss: [vocabulary tile][row of the launch] maximum and sum
  float* hit;            // loss: [row] the target's score; as the maxima without x_scale
  uint16_t* g;           // gradient: blocks [t1 - t0][v1 - v0]
  int64_t g_part;
};

// A score as a float32 of its own: lse is one too, and where a row has one score that matters
// their difference has to be 0, however large they are.
__device__ __forceinline__ float score_of(float acc, float unit) {
#pragma clang fp contract(off)
  return acc * unit;
}

// What a launch of lm_scores leaves.  g lacks its row's factor scale / counted, which is one for
// all rows of a worker: the products' results are multiplied by it.
enum ScoreKind {
  kLossBf16, kLossF32,
  // g in bf16, the type that the caller chose for activations and gradients: an entry is off by up to
  // 2^-8 of itself, as much as dx's and the table gradient's own rounding.  More parts take more
  // products: with three for the table gradient, 65,536 x 2048, 2 x 2048 rows 3.05 -> 5.2 ms.
  kGradBf16,
  kGradBf16x3,  // in three bf16 parts, for a float32 table gradient (dx, in bfloat16, takes the first)
  kGradF32      // in three bf16 parts, of float32 operands
};

// Scores of a tile of words x rows: lane l of a wave holds words in its accumulators and row
// l mod 32 of each of its pieces, so a row's maximum and sum are taken within a lane, then
// over its two lane halves and the two waves that share the row: m the largest, and the sum of
// exp(s - m).  An exponent is always the difference of two scores, rounded once, times log2(e):
// multiplied first (one fused multiply-add an exponential), the rounding of m log2(e) reaches
// the sum whole, 2^-24 |m| of it, and past 2^31 a finite score gives an infinite one.
//
// Bound by the matrix cores and the card's power: 131,072 x 2048 for 4096 rows in bfloat16
// takes 1.83 to 1.95 ms (card to card), 1.2 PFLOP/s with the exponentials; the library's product
// alone, which keeps its scores, 1.65 (1.33 PFLOP/s).  The matrix cores are busy for 56% of
// the cycles at 1.7 GHz, there 75% at 1.5 GHz.  What got it here, in us: operands through
// registers 2113, straight into LDS 1907, LDS reads with one wait per 16 contraction steps
// 1798.  Four waves of 128 x 128: 2856.  The small tiles are held to the registers of three waves
// a SIMD: 403 rows' loss over 14,070 x 259 in float32 59 -> 48 us.
template <int KIND, bool SMALL, bool R>
__global__ __launch_bounds__(SMALL ? 256 : 512, SMALL ? 3 : 2) void lm_scores(ScoreArgs p) {
  constexpr bool kF16 = KIND == kLossF32 || KIND == kGradF32;
  typedef Tile<SMALL, false, false, kF16, R, false> G;
  constexpr int kRows = G::kB * kBlk;  // of the tile
  __shared__ __align__(16) uint16_t sm[G::kLds];
  int vt, tt;
  if (!tile_at(blockIdx.x, (p.v1 - p.v0 + G::kA - 1) / G::kA, (p.t1 - p.t0 + G::kB - 1) / G::kB, kGroup / G::kB, vt, tt)) return;
  const int v0 = p.v0 + vt * G::kA, t0 = p.t0 + tt * G::kB;
  typename G::Acc acc = {};
  G::run(p.w, v0, p.x, t0, 0, p.w.cb, p.tail, p.parts, (lds_t*)sm, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / G::kWN, wn = wave % G::kWN;
  const int64_t word0 = int64_t(v0) * kBlk + wm * G::kRowsA;  // of this wave
  const int n_words = int(min(int64_t(G::kRowsA), p.vocab - word0));  // may be negative
  const float unit = p.x_scale, c = kLog2e * unit;  // a score is an accumulator times this
  if constexpr (kF16) {  // after the powers of two of its row and its word, whose sum is taken first: neither overflows alone
    int32_t of_row[G::kFN];
#pragma unroll
    for (int j = 0; j < G::kFN; ++j) {
      const int at = wn * G::kRowsB + j * 32 + (lane & 31);
      of_row[j] = t0 + at / kBlk < p.t1 ? p.info[int64_t(t0) * kBlk + at].exp : 0;
    }
#pragma unroll
    for (int i = 0; i < G::kFM; ++i)
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const i4v of_word = *reinterpret_cast<const i4v*>(p.w_exps + word0 + i * 32 + e4 * 8 + (lane >> 5) * 4);
#pragma unroll
        for (int j = 0; j < G::kFN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e4 * 4 + e] = ldexpf(acc[i][j][e4 * 4 + e], -(of_word[e] + of_row[j]));
      }
  }
  if constexpr (KIND == kLossBf16 || KIND == kLossF32) {
    float2* joined = reinterpret_cast<float2*>(sm);  // the main loop ends in a barrier: its LDS is free
#pragma unroll
    for (int j = 0; j < G::kFN; ++j) {
      const int at = wn * G::kRowsB + j * 32 + (lane & 31);  // the row's place in the tile
      const int64_t row = int64_t(t0) * kBlk + at;
      const int64_t local = t0 + at / kBlk < p.t1 ? p.info[row].target - word0 : -1;
      const bool here = local >= 0 && local < n_words && (int(local) >> 2 & 1) == lane >> 5;
      if (__any(here)) {
        float hit = 0.f;
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (i * 32 + acc_row(e, lane) == int(local)) hit = acc[i][j][e];
        if (here) p.hit[row] = hit;
      }
      if (n_words < G::kRowsA) {
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (i * 32 + acc_row(e, lane) >= n_words) acc[i][j][e] = -INFINITY;
      }
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < G::kFM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, acc[i][j][e]);
      m = fmaxf(m, __shfl_xor(m, 32));
      const float base = m == -INFINITY ? 0.f : m;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < G::kFM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) s += __builtin_amdgcn_exp2f((acc[i][j][e] - base) * c);
      s += __shfl_xor(s, 32);
      if (lane < 32) joined[wm * kRows + at] = make_float2(m, s);
    }
    __syncthreads();
    const int r = threadIdx.x;
    if (r < kRows && t0 + r / kBlk < p.t1) {
      float2 a = joined[r];
#pragma unroll
      for (int k = 1; k < G::kWM; ++k) {
        const float2 b = joined[k * kRows + r];
        const float m = fmaxf(a.x, b.x), base = m == -INFINITY ? 0.f : m;
        a = make_float2(m, a.y * __builtin_amdgcn_exp2f((a.x - base) * c) + b.y * __builtin_amdgcn_exp2f((b.x - base) * c));
      }
      p.stat[int64_t(vt) * (p.t1 - p.t0) * kBlk + int64_t(tt) * kRows + r] = a;
    }
  } else {
    constexpr int kParts = KIND == kGradBf16 ? 1 : 3;
    static_assert(G::kLds >= G::kA * G::kB * kBlkElems, "the tile's blocks of g, one part of them, fit LDS");
    float g[G::kFM][G::kFN][16];
    auto place = [&](int block) { return sm + block * kBlkElems; };
#pragma unroll
    for (int j = 0; j < G::kFN; ++j) {
      const int at = wn * G::kRowsB + j * 32 + (lane & 31);
      RowInfo ri{-1, 0.f, 0};
      if (t0 + at / kBlk < p.t1) ri = p.info[int64_t(t0) * kBlk + at];
      const bool on = ri.target >= 0;
      const int64_t local = ri.target - word0;
      const bool here = on && local >= 0 && local < n_words;
#pragma unroll
      for (int i = 0; i < G::kFM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) g[i][j][e] = __builtin_amdgcn_exp2f((score_of(acc[i][j][e], unit) - ri.lse) * kLog2e);
      if (__any(here)) {
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (here && i * 32 + acc_row(e, lane) == int(local)) g[i][j][e] -= 1.f;
      }
      if (n_words < G::kRowsA || __any(!on)) {
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!on || i * 32 + acc_row(e, lane) >= n_words) g[i][j][e] = 0.f;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
#pragma unroll
      for (int j = 0; j < G::kFN; ++j)
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
#pragma unroll
          for (int e4 = 0; e4 < 4; ++e4) {
            s4v v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = g[i][j][e4 * 4 + e];
              const uint16_t h = narrow_bits(x);
              v[e] = short(h);
              if (part + 1 < kParts) g[i][j][e4 * 4 + e] = x - widen(h);
            }
            const int row = wn * G::kRowsB + j * 32 + (lane & 31), word = wm * G::kRowsA + i * 32 + e4 * 8;
            const int r = row % kBlk, c8 = word % kBlk / 8;
            *reinterpret_cast<s4v*>(place(row / kBlk * G::kA + word / kBlk) + r * kBlk + ((c8 ^ turn(r)) << 3) + (lane >> 5) * 4) = v;
            __builtin_amdgcn_sched_barrier(0);
          }
      __syncthreads();
      const int n_v = p.v1 - p.v0;
      constexpr int kPieces = G::kA * G::kB * 8 / G::kWaves;  // 1 KB each, per wave
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int at = wave * kPieces + k, block = at / 8, tb = t0 + block / G::kA, vb = v0 - p.v0 + block % G::kA;
        if (tb >= p.t1 || vb >= n_v) continue;
        uint16_t* o = p.g + part * p.g_part + (int64_t(tb - p.t0) * n_v + vb) * kBlkElems + (at % 8 * 64 + lane) * 8;
        *reinterpret_cast<u4v*>(o) = *reinterpret_cast<const u4v*>(place(block) + (at % 8 * 64 + lane) * 8);
      }
      __syncthreads();
    }
  }
}

struct RowsArgs {
  const float2* stat;
  int32_t tiles;
  int64_t ld;           // rows per tile in stat
  const RowInfo* info;
  const float* hit;
  float x_scale;
  int64_t rows;
  float *losses, *lse;
  float* mean;          // of each workgroup's rows, or NULL
  int32_t at;           // rows at a time: 256 or less, a power of two
};

// lse and loss of rows from their `tiles` maxima and sums: `at` rows at a time per workgroup,
// the threads `at` apart share a row's tiles.  With `mean`, a workgroup takes all of a
// worker's `rows` rows and leaves their mean.

__global__ __launch_bounds__(kThreads) void lm_rows(RowsArgs p) {
  __shared__ float2 sm[kThreads];
  __shared__ double sums[kThreads / 64];
  const int r = threadIdx.x % p.at, part = threadIdx.x / p.at, parts = kThreads / p.at;
  const int64_t first = p.mean != nullptr ? blockIdx.x * p.rows : int64_t(blockIdx.x) * p.at;
  const int64_t end = p.mean != nullptr ? first + p.rows : min(p.rows, first + p.at);
  const float c = kLog2e * p.x_scale;
  double sum = 0.0, n = 0.0;
  for (int64_t row0 = first; row0 < end; row0 += p.at) {
    const int64_t row = row0 + r;
    float m = -INFINITY, s = 0.f;
    auto join = [&](const float2& a) {
      const float top = fmaxf(m, a.x), base = top == -INFINITY ? 0.f : top;
      s = s * __builtin_amdgcn_exp2f((m - base) * c) + a.y * __builtin_amdgcn_exp2f((a.x - base) * c);
      m = top;
    };
    if (row < end) {
#pragma unroll 4
      for (int i = part; i < p.tiles; i += parts) join(p.stat[i * p.ld + row]);
    }
    sm[threadIdx.x] = make_float2(m, s);
    __syncthreads();
    if (part == 0 && row < end) {
      for (int i = 1; i < parts; ++i) join(sm[i * p.at + r]);
      const bool on = p.info[row].target >= 0;
      const double ln = double(logf(s));
      const float loss = on ? float((double(m) - double(p.hit[row])) * double(p.x_scale) + ln) : 0.f;  // not less than 0
      p.lse[row] = on ? float(double(m) * double(p.x_scale) + ln) : 0.f;
      p.losses[row] = loss;
      if (on) sum += double(loss), n += 1.0;
    }
    __syncthreads();
  }
  if (p.mean == nullptr) return;
  sum = block_sum(sum, sums);
  n = block_sum(n, sums);
  if (threadIdx.x == 0) p.mean[blockIdx.x] = n > 0.0 ? float(sum / n) : 0.f;
}

__global__ __launch_bounds__(kThreads) void lm_mean(const float* losses, const RowInfo* info, int64_t rows, float* mean) {
  __shared__ double sm[kThreads / 64];
  const int64_t at = blockIdx.x * rows;
  double s = 0.0, n = 0.0;
  for (int64_t i = threadIdx.x; i < rows; i += kThreads) {
    s += double(losses[at + i]);
    n += info[at + i].target >= 0 ? 1.0 : 0.0;
  }
  s = block_sum(s, sm);
  n = block_sum(n, sm);
  if (threadIdx.x == 0) mean[blockIdx.x] = n > 0.0 ? float(s / n) : 0.f;
}

// ------------------------------------------------------------------ products with g
struct ProductArgs {
  Mat g, w, x;        // of one piece of the vocabulary, w from its first block on; all rows
  Parts dx_parts, dw_parts;
  const float* scale;
  const int32_t* count;
  const RowInfo* info;
  int64_t dim;
  float x_scale;      // dropout's
  int32_t tw;         // row blocks per worker
  int64_t rows;       // per worker
  // dx = g T
  int32_t dx_jobs, splits, dx_tail;
  float* dx_part;     // [splits][packed row][ld], or NULL: straight into dx
  void* dx;
  int64_t ld;
  int32_t dx_add;
  // table gradient = g^T drop(x)
  int32_t dw_jobs, dw_tail;
  int32_t v0;         // first vocabulary block of the piece
  int64_t vocab, stride;
  int32_t dw_add;
};

// The two products with g.  The first dx_jobs workgroups take the tiles of dx and the splits of
// their sum over the piece, the others the tiles of every worker's table gradient; one launch, so
// that the chip does not run empty between them.
//
// Bound by the matrix cores as lm_scores where rows and dim are long: 65,536 x 2048 for 2 x 2048
// rows in bfloat16 2.0 ms, 1.1 PFLOP/s for both.  Tiles side by side on one XCD: 4.39 -> 4.22 ms
// for a call on 33,278 x 650, 8 x 700 rows in float32.  By memory where a worker has few rows:
// for 16 x 148 bfloat16 rows 55,650 x 292, 1.04 GB of float32 added to in 1.26 ms (a piece's old
// values loaded one after the other: 2.35; with float32 rows and their parts 2.22).
template <typename T, typename GT, bool SMALL, bool R>
__global__ __launch_bounds__(SMALL ? 256 : 512) void lm_products(ProductArgs p, GT* grads) {
  typedef Tile<SMALL, false, true, false, false, R> Gx;
  typedef Tile<SMALL, true, true, false, false, false> Gw;
  __shared__ __align__(16) uint16_t sm[Gx::kLds];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n_c = (p.x.cb + Gx::kB - 1) / Gx::kB;
  const int64_t in_r = (wave / Gx::kWN) * Gx::kRowsA, in_c = (wave % Gx::kWN) * Gx::kRowsB + (lane & 31);
  typename Gx::Acc acc = {};
  const int dx_grid = (p.dx_jobs + 7) / 8 * 8;
  if (int(blockIdx.x) < dx_grid) {
    const int job = int(place_of(blockIdx.x, p.dx_jobs));
    if (job < 0) return;
    // tiles side by side share g, those above each other the table
    const int kb = p.g.cb, n_r = (p.g.rb + Gx::kA - 1) / Gx::kA;
    const int c0 = job % n_c * Gx::kB, r0 = job / n_c % n_r * Gx::kA, split = job / n_c / n_r;
    const int k0 = int(int64_t(kb) * split / p.splits), k1 = int(int64_t(kb) * (split + 1) / p.splits);
    Gx::run(p.g, r0, p.w, c0, k0, k1, k1 == kb ? p.dx_tail : 4, p.dx_parts, (lds_t*)sm, acc);
    const int64_t packed = int64_t(p.g.rb) * kBlk, per = int64_t(p.tw) * kBlk;
#pragma unroll
    for (int i = 0; i < Gx::kFM; ++i)
#pragma unroll
      for (int j = 0; j < Gx::kFN; ++j) {
        const int64_t c = int64_t(c0) * kBlk + in_c + j * 32, r = int64_t(r0) * kBlk + in_r + i * 32;
        if (r >= packed || c >= p.ld) continue;  // packed rows and ld are whole pieces
        if (p.dx_part != nullptr) {
          float* o = p.dx_part + (split * packed + r) * p.ld + c;
          float old[16] = {};
          if (p.dx_add) {
#pragma unroll
            for (int e = 0; e < 16; ++e) old[e] = o[acc_row(e, lane) * p.ld];
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) o[acc_row(e, lane) * p.ld] = old[e] + acc[i][j][e];
          continue;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int64_t row = r + acc_row(e, lane), w = row / per;
          if (c < p.dim && row % per < p.rows)
            put(static_cast<T*>(p.dx) + (w * p.rows + row % per) * p.dim + c,
                p.info[row].target >= 0 ? acc[i][j][e] * coef_of(p.scale, p.count, w) : 0.f);
        }
      }
    return;
  }
  const int job = int(place_of(int(blockIdx.x) - dx_grid, p.dw_jobs));
  if (job < 0) return;
  const int per = (p.g.cb + Gw::kA - 1) / Gw::kA * n_c, w = job / per;
  const int c0 = job % per % n_c * Gw::kB, r0 = job % per / n_c * Gw::kA;
  Gw::run(p.g, r0, p.x, c0, w * p.tw, (w + 1) * p.tw, p.dw_tail, p.dw_parts, (lds_t*)sm, acc);
  const float coef = coef_of(p.scale, p.count, w) * p.x_scale;
  GT* out = grads + w * p.stride;
#pragma unroll
  for (int i = 0; i < Gw::kFM; ++i)
#pragma unroll
    for (int j = 0; j < Gw::kFN; ++j) {
      const int64_t c = int64_t(c0) * kBlk + in_c + j * 32, in = int64_t(r0) * kBlk + in_r + i * 32;
      const int64_t row = int64_t(p.v0) * kBlk + in, n = min(p.vocab - row, int64_t(p.g.cb) * kBlk - in);  // words left
      if (c >= p.dim || n <= 0) continue;
      GT* o = out + row * p.dim + c;
      // a whole piece's old values are loaded together
      float old[16] = {};
      if (p.dw_add) {
        if (n >= 32) {
#pragma unroll
          for (int e = 0; e < 16; ++e) old[e] = widen(o[acc_row(e, lane) * p.dim]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (acc_row(e, lane) < n) old[e] = widen(o[acc_row(e, lane) * p.dim]);
        }
      }
      if (n >= 32) {
#pragma unroll
        for (int e = 0; e < 16; ++e) put(o + acc_row(e, lane) * p.dim, old[e] + acc[i][j][e] * coef);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (acc_row(e, lane) < n) put(o + acc_row(e, lane) * p.dim, old[e] + acc[i][j][e] * coef);
      }
    }
}

// dx of every row from its splits, times scale / counted, through dropout: 5600 x 650
// float32 from three splits, 62 MB, in 16 us.
template <typename T>
__global__ __launch_bounds__(kThreads) void lm_dx_out(const float* part, int32_t splits, int64_t packed_rows, int64_t ld,
                                                      const RowInfo* info, const float* scale, const int32_t* count,
                                                      int64_t rows, int64_t packed, int32_t dim, T* out, Drop d) {
  const int64_t row = blockIdx.x, w = row / rows, r = w * packed + row % rows;
  const bool on = info[r].target >= 0;
  const uint64_t step = d.on ? step_of(d) : 0;
  const float coef = coef_of(scale, count, w);
  for (int32_t c = int32_t(threadIdx.x) * 4; c < dim; c += kThreads * 4) {
    float x[4] = {};
    if (on) {
      for (int s = 0; s < splits; ++s) {
        float y[4];
        load<4>(part + (s * packed_rows + r) * ld + c, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += y[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] *= coef;
      if (d.on) drop<4>(d, step, uint64_t(row) * uint64_t(dim) + uint64_t(c), d.scale, x);
    }
    T* o = out + row * dim + c;
    if (c + 4 <= dim) {
      store<4>(o, x);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < dim) put(o + e, x[e]);
    }
  }
}

// ------------------------------------------------------------------ embedding
// A wave takes 512 columns of a row.  8 x 700 rows of 650 in float32, dropped out: 9.2 us for
// 29 MB (one row: 2.8).
template <typename T>
__global__ __launch_bounds__(64) void lm_embed(const T* table, int64_t vocab, int32_t dim, const int64_t* tokens, T* out,
                                               Drop d) {
  const int64_t row = blockIdx.x;
  const int32_t c = (int32_t(blockIdx.y) * 64 + int32_t(threadIdx.x)) * 8;
  if (c >= dim) return;
  const int64_t t = tokens[row];
  const int n = min(8, dim - c);
  float x[8] = {};
  if (uint64_t(t) < uint64_t(vocab)) {
    const T* p = table + t * dim + c;
    if (n == 8) {
      load<8>(p, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) x[e] = widen(p[e]);
    }
    if (d.on) drop<8>(d, step_of(d), uint64_t(row) * uint64_t(dim) + uint64_t(c), d.scale, x);
  }
  T* o = out + row * dim + c;
  if (n == 8) {
    store<8>(o, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) put(o + e, x[e]);
  }
}

// A pair is token << 32 | row; pairs of tokens outside the vocabulary come last.
constexpr uint64_t kNoToken = 0xffffffffull;

// The first workgroups each sort one chunk of a worker's pairs (bitonic: a fixed network on
// distinct keys, 55 steps of a barrier each: 14 us for 1024 pairs, 50 for 4096); the others zero
// the tables that are not added to (537 MB in 98 us), 32 KB at a time in turn, which hides the sort.
template <typename GT>
__global__ __launch_bounds__(kSortThreads) void lm_sort(const int64_t* tokens, int64_t rows, int64_t vocab, int32_t size,
                                                        uint64_t* keys, int32_t chunks, int32_t workers, GT* table, int64_t n,
                                                        int64_t stride, int64_t zeros) {
  __shared__ uint64_t sm[kSortMax];
  if (int(blockIdx.x) >= chunks * workers) {
    constexpr int kV = 16 / sizeof(GT);
    const int64_t per = (n + kSortThreads * kZeroUnits * kV - 1) / (kSortThreads * kZeroUnits * kV);
    for (int64_t job = int64_t(blockIdx.x) - chunks * workers; job < zeros; job += int64_t(gridDim.x) - chunks * workers) {
      GT* t = table + job / per * stride;
#pragma unroll
      for (int u = 0; u < kZeroUnits; ++u) {
        const int64_t i = ((job % per * kZeroUnits + u) * kSortThreads + threadIdx.x) * kV;
        if (i + kV <= n) {
          __builtin_nontemporal_store(u4v{}, reinterpret_cast<u4v*>(t + i));
        } else {
          for (int64_t e = i; e < n; ++e) t[e] = GT(0);
        }
      }
    }
    return;
  }
  const int64_t at = int64_t(blockIdx.x) / chunks * rows, t0 = int64_t(blockIdx.x) % chunks * size;
  for (int i = threadIdx.x; i < size; i += kSortThreads) {
    uint64_t key = ~0ull;
    if (t0 + i < rows) {
      const uint64_t t = uint64_t(tokens[at + t0 + i]);
      key = (t < uint64_t(vocab) ? t : kNoToken) << 32 | uint64_t(t0 + i);
    }
    sm[i] = key;
  }
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kSortThreads) {
        const int lo = (i & ~(j - 1)) * 2 + (i & (j - 1)), hi = lo + j;
        const uint64_t a = sm[lo], b = sm[hi];
        if ((a > b) == ((lo & k) == 0)) sm[lo] = b, sm[hi] = a;
      }
      __syncthreads();
    }
  for (int i = threadIdx.x; i < size; i += kSortThreads)
    if (t0 + i < rows) keys[at + t0 + i] = sm[i];
}

// Sorted runs of `run` pairs into runs of twice that: a pair's place is its own plus the
// number of smaller ones in the other run.
__global__ __launch_bounds__(kThreads) void lm_merge(const uint64_t* src, uint64_t* dst, int64_t rows, int64_t run) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= rows) return;
  const uint64_t* s = src + int64_t(blockIdx.y) * rows;
  const int64_t pair = i / (2 * run) * (2 * run), mid = min(rows, pair + run), end = min(rows, pair + 2 * run);
  const bool right = i >= mid;
  const uint64_t key = s[i];
  int64_t lo = right ? pair : mid, hi = right ? mid : end;
  const int64_t from = lo;
  while (lo < hi) {
    const int64_t m = (lo + hi) / 2;
    if (s[m] < key) lo = m + 1;
    else hi = m;
  }
  dst[int64_t(blockIdx.y) * rows + (right ? i - mid : i - pair) + pair + (lo - from)] = key;
}

// Columns c to c + 3 of a row, without a branch around the load, so that the loads of several
// rows are under way together.  WIDE (dim >= 4): the last lane's columns come from the row's
// last four.
template <bool WIDE, typename T>
__device__ __forceinline__ void load_row(const T* row, int32_t c, int32_t dim, float (&x)[4]) {
  if constexpr (WIDE) {
    const int32_t from = min(c, dim - 4), skip = c - from;
    float v[4];
    load<4>(row + from, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = v[e];
#pragma unroll
      for (int k = 1; e + k < 4; ++k) x[e] = skip == k ? v[e + k] : x[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = widen(row[min(c + e, dim - 1)]);
  }
}

template <typename GT>
__device__ __forceinline__ void write_row(GT* o, int n, const float (&old)[4], const float (&x)[4]) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = old[e] + x[e];
  if (n == 4) {
    store<4>(o, y);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) put(o + e, y[e]);
  }
}

struct SumArgs {
  const uint64_t* keys;
  int64_t rows;  // per worker
  int32_t dim, dpad, n_runs, add;
  int64_t stride;
  float* part;  // [worker][run][2][dpad]: a token's sum from its earlier run on, and the start of one that goes on
};

// A pair that every lane reads, as a scalar.
__device__ __forceinline__ uint64_t pair_at(const uint64_t* keys, int64_t i) {
  const uint64_t k = keys[i];
  return uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(k >> 32)))) << 32 |
         uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(k))));
}

// kRun sorted pairs x 256 columns per wave, summed in their order.  A token whose pairs lie
// in one run is written here; the others leave a part per run for lm_join.  Bound by the
// latency of the loads, hence kRunLoads rows at once and no branch around them: 8 x 700 rows
// of 650 in float32, dropped out and added, 20 us (one row after the other, 32 per wave: 51).
template <typename T, typename GT, bool WIDE>
__global__ __launch_bounds__(64) void lm_sum(SumArgs p, const T* dout, GT* table, Drop d) {
  const int64_t w = blockIdx.z, run = blockIdx.x, i0 = run * kRun, i1 = min(p.rows, i0 + kRun);
  const int32_t c = (int32_t(blockIdx.y) * 64 + int32_t(threadIdx.x)) * 4;
  const uint64_t* keys = p.keys + w * p.rows;
  const int n = min(4, p.dim - c);
  if (n <= 0) return;
  const uint64_t step = d.on ? step_of(d) : 0;
  const uint64_t before = i0 > 0 ? pair_at(keys, i0 - 1) >> 32 : ~0ull, after = i1 < p.rows ? pair_at(keys, i1) >> 32 : ~0ull;
  float* part = p.part + (w * p.n_runs + run) * 2 * p.dpad + c;
  table += w * p.stride;
  float sum[4] = {};
  for (int64_t i = i0; i < i1; i += kRunLoads) {
    uint64_t key[kRunLoads + 1];
    float x[kRunLoads][4], old[kRunLoads][4] = {};
#pragma unroll
    for (int u = 0; u <= kRunLoads; ++u) key[u] = pair_at(keys, min(i + u, i1 - 1));
    // a token past the run or the vocabulary is loaded from the first row and left out below
    auto real = [&](int u) { return i + u < i1 && key[u] >> 32 != kNoToken; };
    auto row = [&](int u) { return table + (real(u) ? int64_t(key[u] >> 32) : 0) * p.dim; };
#pragma unroll
    for (int u = 0; u < kRunLoads; ++u)
      load_row<WIDE>(dout + (w * p.rows + int64_t(key[u] & 0xffffffffu)) * p.dim, c, p.dim, x[u]);
    if (p.add) {
#pragma unroll
      for (int u = 0; u < kRunLoads; ++u) load_row<WIDE>(row(u), c, p.dim, old[u]);
    }
#pragma unroll
    for (int u = 0; u < kRunLoads; ++u) {
      if (!real(u)) continue;
      const int64_t t = w * p.rows + int64_t(key[u] & 0xffffffffu);
      if (d.on) drop<4>(d, step, uint64_t(t) * uint64_t(p.dim) + uint64_t(c), d.scale, x[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += x[u][e];
      const uint64_t token = key[u] >> 32, next = i + u + 1 < i1 ? key[u + 1] >> 32 : ~0ull;
      if (token == next) continue;
      // the token's pairs of this run end here
      if (token == before || (i + u + 1 == i1 && token == after)) {
        store<4>(part + (token == before ? 0 : p.dpad), sum);
      } else {
        write_row(row(u) + c, n, old[u], sum);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = 0.f;
    }
  }
}

// The tokens whose pairs start in this run and go on after it: as far as the runs begin with
// them.  kRunLoads runs are looked at together, by one of kJoinWaves waves in turn, so that a word
// that fills many runs (a padding word) is no chain of one wave; the waves' sums are joined in
// their order.  The runs' parts are added up in float64: a token can fill 2^19 of them, and as
// many roundings to float32 of a sum that grows would be seen.  16,384 rows of 2048 bfloat16, words
// drawn as in text and one word in all: 10 and 60 us (one wave: 27 and 386; eight: 16 and 42).
template <typename GT, bool WIDE>
__global__ __launch_bounds__(64 * kJoinWaves) void lm_join(SumArgs p, GT* table) {
  __shared__ double sums[kJoinWaves][4][64];
  const int64_t w = blockIdx.z, run = blockIdx.x, i0 = run * kRun, i1 = i0 + kRun;
  const uint64_t* keys = p.keys + w * p.rows;
  if (i1 >= p.rows) return;
  const uint64_t token = pair_at(keys, i1 - 1) >> 32;
  if (token == kNoToken || pair_at(keys, i1) >> 32 != token || (i0 > 0 && pair_at(keys, i0 - 1) >> 32 == token)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t c = (int32_t(blockIdx.y) * 64 + lane) * 4;
  const int n = min(4, p.dim - c);
  const float* part = p.part + w * p.n_runs * 2 * p.dpad + (n > 0 ? c : 0);
  table += w * p.stride + int64_t(token) * p.dim;
  float first[4] = {}, old[4] = {};
  if (wave == 0) {
    load<4>(part + (run * 2 + 1) * p.dpad, first);
    if (p.add && n > 0) load_row<WIDE>(table, c, p.dim, old);
  }
  double sum[4] = {first[0], first[1], first[2], first[3]};
  auto begins = [&](int64_t r) { return pair_at(keys, min(r, int64_t(p.n_runs) - 1) * kRun) >> 32 == token && r < p.n_runs; };
  constexpr int kStep = kJoinWaves * kRunLoads;
  int64_t r = run + 1 + wave * kRunLoads;
  for (bool goes_on = begins(r); goes_on; r += kStep) {
    const bool more = begins(r + kStep);
    float x[kRunLoads][4];
    bool in[kRunLoads];
#pragma unroll
    for (int u = 0; u < kRunLoads; ++u) {
      in[u] = begins(r + u);
      load<4>(part + min(r + u, int64_t(p.n_runs) - 1) * 2 * p.dpad, x[u]);
    }
#pragma unroll
    for (int u = 0; u < kRunLoads; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += in[u] ? double(x[u][e]) : 0.0;
    goes_on = more;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sums[wave][e][lane] = sum[e];
  __syncthreads();
  if (wave > 0 || n <= 0) return;
  float all[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    for (int k = 1; k < kJoinWaves; ++k) sum[e] += sums[k][e][lane];
    all[e] = float(sum[e]);
  }
  write_row(table + c, n, old, all);
}

// ------------------------------------------------------------------ dropout
// n / d for 32-bit n: the multiplier and shifts of Granlund and Montgomery ("Division by
// invariant integers using multiplication", 1994).
struct Div {
  uint64_t d;
  uint32_t mul, s1, s2;
};

__device__ __forceinline__ uint64_t divide(uint64_t n, const Div& v) {
  if ((n | v.d) >> 32) return n / v.d;
  const uint32_t x = uint32_t(n), t = __umulhi(v.mul, x);
  return (t + ((x - t) >> v.s1)) >> v.s2;
}

struct DropArgs {
  const void *x, *residual;
  void* out;
  int64_t xs, rs, os;  // strides
  int64_t n, cols;
  int64_t first;  // the launch's first group of N entries
  Div groups;     // VEC: groups of N entries per row; otherwise cols
};

// N consecutive entries per thread.  VEC: they lie in one row (cols is a multiple of N); 16-byte
// loads at any alignment.  16,384 x 4096 bfloat16 with a residual: 71 us, 5.7 TB/s; element by
// element, with a 64-bit division per thread, 155.
template <typename T, int N, bool VEC>
__global__ __launch_bounds__(kThreads) void lm_dropout(DropArgs p, Drop d) {
  const int64_t group = p.first + int64_t(blockIdx.x) * kThreads + threadIdx.x, i = group * N;
  if (i >= p.n) return;
  const T* x = static_cast<const T*>(p.x);
  const T* residual = static_cast<const T*>(p.residual);
  T* out = static_cast<T*>(p.out);
  const uint64_t step = step_of(d);
  if constexpr (VEC) {
    const int64_t r = int64_t(divide(uint64_t(group), p.groups)), c = i - r * p.cols;
    float v[N], y[N] = {};
    load<N>(x + r * p.xs + c, v);
    if (residual != nullptr) load<N>(residual + r * p.rs + c, y);
    drop<N>(d, step, uint64_t(i), d.scale, v);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] += y[e];
    store<N>(out + r * p.os + c, v);
  } else {
    int64_t r = int64_t(divide(uint64_t(i), p.groups)), c = i - r * p.cols;
    int64_t rows[N], at[N];
    float v[N] = {}, y[N] = {};
#pragma unroll
    for (int e = 0; e < N; ++e) {
      rows[e] = r, at[e] = c;
      if (i + e < p.n) {
        v[e] = widen(x[r * p.xs + c]);
        if (residual != nullptr) y[e] = widen(residual[r * p.rs + c]);
      }
      if (++c == p.cols) c = 0, ++r;
    }
    drop<N>(d, step, uint64_t(i), d.scale, v);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (i + e < p.n) put(out + rows[e] * p.os + at[e], v[e] + y[e]);
  }
}

// ------------------------------------------------------------------ host helpers
uint64_t a256(uint64_t x) { return (x + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Launch on `st`; with timing on, through hipExtLaunchKernelGGL with events the runtime
// records with the dispatch itself.
template <typename... KArgs, typename... Args>
psgd_status launch(psgd_lm_plan* plan, int kid, void (*kernel)(KArgs...), dim3 grid, int threads, hipStream_t st, Args... args) {
  hipEvent_t a = nullptr, b = nullptr;
  if (plan->timing) {
    room_for_timing(plan);
    psgd_status s = take_event(plan->event_pool, &a);
    if (s == PSGD_OK) s = take_event(plan->event_pool, &b);
    if (s != PSGD_OK) {
      if (a) plan->event_pool.push_back(a);
      return s;
    }
    hipExtLaunchKernelGGL(kernel, grid, dim3(unsigned(threads)), 0, st, a, b, 0, args...);
  } else {
    hipLaunchKernelGGL(kernel, grid, dim3(unsigned(threads)), 0, st, args...);
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

// A graph must not hold the events of timed launches.
psgd_status check_capture(const char* fn, const psgd_lm_plan* plan, hipStream_t st) {
  if (!plan->timing) return PSGD_OK;
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  const hipError_t e = hipStreamIsCapturing(st, &cs);
  if (e != hipSuccess) return hip_fail("hipStreamIsCapturing", e);
  return cs == hipStreamCaptureStatusNone
             ? PSGD_OK
             : fail(PSGD_ERR_INVALID_ARG, std::string(fn) + ": a call can be captured into a graph only with kernel timing off");
}

psgd_status make_drop(const char* fn, const psgd_dropout_config* c, Drop* out) {
  *out = Drop{0, 0, 0, nullptr, 1.f, 0};
  if (c == nullptr) return PSGD_OK;
  if (!(c->p >= 0.0 && c->p <= 1.0)) return fail(PSGD_ERR_INVALID_ARG, std::string(fn) + ": dropout's p must be in [0, 1]");
  if (uintptr_t(c->step) % 8 != 0) return fail(PSGD_ERR_INVALID_ARG, std::string(fn) + ": dropout's step is not 8-byte aligned");
  out->keep_from = uint64_t(c->p * 4294967296.0);
  out->key0 = uint32_t(c->seed);
  out->key1 = uint32_t(c->seed >> 32);
  out->step = c->step;
  out->scale = c->p < 1.0 ? float(1.0 / (1.0 - c->p)) : 0.f;
  out->on = c->p > 0.0 ? 1 : 0;
  return PSGD_OK;
}

int parts_of(psgd_dtype t) { return t == PSGD_F32 ? 2 : 1; }
int g_parts(const psgd_lm_plan* plan) { return plan->act == PSGD_F32 || plan->grad == PSGD_F32 ? 3 : 1; }

constexpr Parts kOne{1, 0, 0};
constexpr Parts kF32{3, 0x001, 0x010};        // two fp16 parts each: high x low, low x high, high x high
// bf16 parts, the smallest products first
constexpr Parts kThreeByOne{3, 0x012, 0x000};
constexpr Parts kTwoByTwo{3, 0x010, 0x001};           // for a bf16 result: what is left out is 2^-16 of it
constexpr Parts kThreeByThree{6, 0x010120, 0x001102};  // all above 2^-24

int32_t steps_of_last(int64_t n) { return int32_t(ceil_div((n - 1) % kBlk + 1, 16)); }

struct Views {
  Mat x, w, x3, w3;
  uint16_t* g;
  RowInfo* info;
  int32_t* count;
  int32_t *x_exps, *w_exps;
  float2* stat;
  float *hit, *dx;
};

Views views(const psgd_lm_plan* plan, const void* params, void* workspace, int32_t tb) {
  char* ws = static_cast<char*>(workspace);
  Views v{};
  v.g = reinterpret_cast<uint16_t*>(ws + plan->ws_g);
  v.info = reinterpret_cast<RowInfo*>(ws + plan->ws_info);
  v.count = reinterpret_cast<int32_t*>(ws + plan->ws_count);
  v.x_exps = reinterpret_cast<int32_t*>(ws + plan->ws_x_exps);
  v.w_exps = reinterpret_cast<int32_t*>(ws + plan->ws_w_exps);
  v.stat = reinterpret_cast<float2*>(ws + plan->ws_stat);
  v.hit = reinterpret_cast<float*>(ws + plan->ws_hit);
  v.dx = reinterpret_cast<float*>(ws + plan->ws_dx);
  v.x = Mat{reinterpret_cast<uint16_t*>(ws + plan->ws_x), int64_t(tb) * plan->db * kBlkElems, tb, plan->db, 0};
  v.w = plan->direct ? Mat{static_cast<const uint16_t*>(params) + plan->offset, 0, plan->vb, plan->db, int32_t(plan->vocab - 1)}
                     : Mat{reinterpret_cast<uint16_t*>(ws + plan->ws_w), int64_t(plan->vb) * plan->db * kBlkElems, plan->vb,
                           plan->db, 0};
  v.x3 = v.x, v.w3 = v.w;
  if (plan->act == PSGD_F32) {
    v.x3.p = reinterpret_cast<uint16_t*>(ws + plan->ws_x3);
    v.w3.p = reinterpret_cast<uint16_t*>(ws + plan->ws_w3);
  }
  return v;
}

// Words of whole large tiles, as lm_scores reads their powers of two.
int64_t padded_words(int64_t vb) { return ceil_div(vb, kTile) * kTile * kBlk; }

const void* table_of(const psgd_lm_plan* plan, const void* params) {
  return static_cast<const char*>(params) + plan->offset * (plan->act == PSGD_F32 ? 4 : 2);
}

// The packed operands: x in groups of `rows` rows, and the table.  count: NULL for the loss.
// x3, w3: whether the products with g will read them.
psgd_status enqueue_pack(psgd_lm_plan* plan, const Views& v, const void* x, const void* params, int64_t rows, int32_t blocks,
                         const int64_t* targets, const float* lse, int32_t* count, bool x3, bool w3, const Drop& d,
                         hipStream_t st) {
  const bool f32 = plan->act == PSGD_F32;
  const void* table = table_of(plan, params);
  if (f32) {
    int32_t lanes = 1;
    while (lanes < 64 && lanes * 16 < plan->dim) lanes *= 2;
    const int64_t padded = padded_words(plan->vb), n = plan->rows * plan->n_workers;
    const int64_t groups = std::min<int64_t>(kPeakGroups, ceil_div((padded + n) * lanes, kThreads));
    const psgd_status s = launch(plan, kPeak, lm_peak, dim3(unsigned(groups)), kThreads, st, static_cast<const float*>(table),
                                 plan->vocab, padded, static_cast<const float*>(x), n, plan->dim, targets, lanes, v.w_exps,
                                 v.x_exps, d);
    if (s != PSGD_OK) return s;
  }
  PackArgs a{x, table, v.x, v.w, v.x3, v.w3, rows, blocks, plan->rows, plan->vocab, int32_t(plan->dim),
             targets, lse, v.info, count, v.x_exps, v.w_exps};
  if (plan->direct) a.w_to.p = nullptr;
  if (!x3) a.x3_to.p = nullptr;
  if (!w3) a.w3_to.p = nullptr;
  const int64_t jobs = int64_t(v.x.rb) * v.x.cb + (plan->direct ? 0 : int64_t(v.w.rb) * v.w.cb) +
                       (count != nullptr ? plan->n_workers : 0);
  return launch(plan, kPack, f32 ? lm_pack<float> : lm_pack<uint16_t>, dim3(unsigned(jobs)), kThreads, st, a, d);
}

unsigned score_grid(const ScoreArgs& a, int tile) {
  return unsigned(ceil_div(ceil_div(a.v1 - a.v0, tile) * ceil_div(a.t1 - a.t0, tile), 8) * 8);
}

// Whether the tiles of a v x t blocks problem are the small ones.
bool small_tiles(int64_t v, int64_t t) { return ceil_div(v, kTile) * ceil_div(t, kTile) < kFewTiles; }

template <int KIND, bool R>
psgd_status enqueue_scores(psgd_lm_plan* plan, const ScoreArgs& a, bool small, hipStream_t st) {
  return small ? launch(plan, kScores, lm_scores<KIND, true, R>, dim3(score_grid(a, 1)), 256, st, a)
               : launch(plan, kScores, lm_scores<KIND, false, R>, dim3(score_grid(a, kTile)), 512, st, a);
}

// What the products' results are multiplied by; with p = 1 they are zero.
float x_scale_of(const Drop& d) { return d.on && d.scale > 0.f ? d.scale : 1.f; }

psgd_status enqueue_loss(psgd_lm_plan* plan, const void* x, const void* params, const int64_t* targets, const Drop& d,
                         float* losses, float* lse, float* mean, void* workspace, hipStream_t st) {
  const int64_t rows = plan->rows * plan->n_workers;
  const Views v = views(plan, params, workspace, plan->tb);
  psgd_status s = enqueue_pack(plan, v, x, params, rows, plan->tb, targets, nullptr, nullptr, false, false, d, st);
  if (s != PSGD_OK) return s;
  const bool f32 = plan->act == PSGD_F32, small = plan->loss_small;
  const int32_t tiles = int32_t(ceil_div(plan->vb, small ? 1 : kTile));
  // a workgroup per worker does all its rows where that is little
  const bool one = plan->chunk >= plan->tb && plan->rows * tiles <= kFewStats;
  int32_t at = kThreads;  // 16 threads for a row's tiles, or as many as there are tiles
  while (at > 16 && kThreads / at < tiles) at /= 2;
  for (int32_t t0 = 0; t0 < plan->tb; t0 += plan->chunk) {
    const ScoreArgs a{v.w, v.x, f32 ? kF32 : kOne, steps_of_last(plan->dim), 0, plan->vb, t0, std::min(plan->tb, t0 + plan->chunk),
                      plan->vocab, v.info, v.w_exps, x_scale_of(d), v.stat, v.hit, nullptr, 0};
    s = f32 ? enqueue_scores<kLossF32, false>(plan, a, small, st)
            : plan->direct ? enqueue_scores<kLossBf16, true>(plan, a, small, st) : enqueue_scores<kLossBf16, false>(plan, a, small, st);
    if (s != PSGD_OK) return s;
    const int64_t r0 = int64_t(t0) * kBlk, n = one ? plan->rows : std::min(rows, int64_t(a.t1) * kBlk) - r0;
    const RowsArgs b{v.stat, tiles, int64_t(a.t1 - t0) * kBlk, v.info + r0, v.hit + r0, a.x_scale, n, losses + r0, lse + r0,
                     one ? mean : nullptr, at};
    s = launch(plan, kRows, lm_rows, dim3(unsigned(one ? plan->n_workers : ceil_div(n, at))), kThreads, st, b);
    if (s != PSGD_OK) return s;
  }
  if (one) return PSGD_OK;
  return launch(plan, kMean, lm_mean, dim3(unsigned(plan->n_workers)), kThreads, st, static_cast<const float*>(losses),
                static_cast<const RowInfo*>(v.info), plan->rows, mean);
}

template <typename T, typename GT, bool R>
psgd_status enqueue_products(psgd_lm_plan* plan, const ProductArgs& a, bool small, GT* grads, hipStream_t st) {
  const dim3 grid(unsigned(ceil_div(a.dx_jobs, 8) * 8 + ceil_div(a.dw_jobs, 8) * 8));
  return small ? launch(plan, kProducts, lm_products<T, GT, true, R>, grid, 256, st, a, grads)
               : launch(plan, kProducts, lm_products<T, GT, false, R>, grid, 512, st, a, grads);
}

psgd_status enqueue_grad(psgd_lm_plan* plan, const void* x, const void* params, const int64_t* targets, const float* lse,
                         const float* scale, const Drop& d, void* dx, void* grads, bool add, void* workspace, hipStream_t st) {
  const int32_t tb = plan->tw * plan->n_workers;
  const Views v = views(plan, params, workspace, tb);
  psgd_status s = enqueue_pack(plan, v, x, params, plan->rows, plan->tw, targets, lse, v.count, grads != nullptr, dx != nullptr,
                               d, st);
  if (s != PSGD_OK) return s;
  const bool f32 = plan->act == PSGD_F32, f32g = plan->grad == PSGD_F32, direct = plan->direct;
  const float x_scale = x_scale_of(d);
  // straight into dx: one piece, one split, and no mask to draw again
  const bool straight = plan->piece >= plan->vb && plan->splits == 1 && !d.on;
  const int tile = plan->grad_small ? 1 : kTile;
  const int64_t n_c = ceil_div(plan->db, tile);
  for (int32_t v0 = 0; v0 < plan->vb; v0 += plan->piece) {
    const int32_t v1 = std::min(plan->vb, v0 + plan->piece), n_v = v1 - v0;
    const int64_t g_part = int64_t(tb) * n_v * kBlkElems;
    const ScoreArgs a{v.w, v.x, f32 ? kF32 : kOne, steps_of_last(plan->dim), v0, v1, 0, tb, plan->vocab, v.info, v.w_exps, x_scale,
                      nullptr, nullptr, v.g, g_part};
    const bool small = plan->scores_small;
    if (f32)
      s = enqueue_scores<kGradF32, false>(plan, a, small, st);
    else if (f32g)
      s = direct ? enqueue_scores<kGradBf16x3, true>(plan, a, small, st) : enqueue_scores<kGradBf16x3, false>(plan, a, small, st);
    else
      s = direct ? enqueue_scores<kGradBf16, true>(plan, a, small, st) : enqueue_scores<kGradBf16, false>(plan, a, small, st);
    if (s != PSGD_OK) return s;
    Mat w = v.w3;
    w.p += int64_t(v0) * w.cb * kBlkElems;  // as many elements packed or not
    w.last -= v0 * kBlk;
    w.rb = n_v;
    ProductArgs b{};
    b.g = Mat{v.g, g_part, tb, n_v, 0};
    b.w = w;
    b.x = v.x3;
    b.dx_parts = f32 ? kThreeByThree : kOne;
    b.dw_parts = f32 ? (f32g ? kThreeByThree : kTwoByTwo) : f32g ? kThreeByOne : kOne;
    b.scale = scale;
    b.count = v.count;
    b.info = v.info;
    b.dim = plan->dim;
    b.x_scale = x_scale;
    b.tw = plan->tw;
    b.rows = plan->rows;
    b.splits = plan->splits;
    b.dx_jobs = dx != nullptr ? int32_t(ceil_div(tb, tile) * n_c * plan->splits) : 0;
    b.dx_tail = v1 == plan->vb ? steps_of_last(plan->vocab) : 4;
    b.dx_part = straight ? nullptr : v.dx;
    b.dx = dx;
    b.ld = int64_t(plan->db) * kBlk;
    b.dx_add = v0 > 0 ? 1 : 0;
    b.dw_jobs = grads != nullptr ? int32_t(ceil_div(n_v, tile) * n_c * plan->n_workers) : 0;
    b.dw_tail = steps_of_last(plan->rows);
    b.v0 = v0;
    b.vocab = plan->vocab;
    b.stride = plan->worker_stride;
    b.dw_add = add ? 1 : 0;
    float* gf = static_cast<float*>(grads) + plan->offset;
    uint16_t* gb = static_cast<uint16_t*>(grads) + plan->offset;
    const bool few = plan->grad_small;
    if (f32)
      s = f32g ? enqueue_products<float, float, false>(plan, b, few, gf, st) : enqueue_products<float, uint16_t, false>(plan, b, few, gb, st);
    else if (direct)
      s = f32g ? enqueue_products<uint16_t, float, true>(plan, b, few, gf, st) : enqueue_products<uint16_t, uint16_t, true>(plan, b, few, gb, st);
    else
      s = f32g ? enqueue_products<uint16_t, float, false>(plan, b, few, gf, st) : enqueue_products<uint16_t, uint16_t, false>(plan, b, few, gb, st);
    if (s != PSGD_OK) return s;
  }
  if (dx == nullptr || straight) return PSGD_OK;
  const dim3 grid(unsigned(plan->rows * plan->n_workers));
  const RowInfo* info = v.info;
  const float* part = v.dx;
  const int32_t* count = v.count;
  const int64_t packed = int64_t(tb) * kBlk, ld = int64_t(plan->db) * kBlk, per = int64_t(plan->tw) * kBlk;
  return f32 ? launch(plan, kDxOut, lm_dx_out<float>, grid, kThreads, st, part, plan->splits, packed, ld, info, scale, count,
                      plan->rows, per, int32_t(plan->dim), static_cast<float*>(dx), d)
             : launch(plan, kDxOut, lm_dx_out<uint16_t>, grid, kThreads, st, part, plan->splits, packed, ld, info, scale, count,
                      plan->rows, per, int32_t(plan->dim), static_cast<uint16_t*>(dx), d);
}

Div divide_by(uint64_t d) {
  Div v{d, 0, 0, 0};
  if (d >> 32) return v;
  uint32_t l = 0;
  while ((uint64_t(1) << l) < d) ++l;
  v.mul = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1);
  v.s1 = std::min<uint32_t>(l, 1);
  v.s2 = l > 1 ? l - 1 : 0;
  return v;
}

template <typename T, int N, bool VEC>
psgd_status enqueue_dropout(DropArgs a, const Drop& d, hipStream_t st) {
  a.groups = divide_by(uint64_t(VEC ? a.cols / N : a.cols));
  const int64_t all = ceil_div(a.n, kThreads * N);
  for (int64_t at = 0; at < all; at += kMostGroups) {
    a.first = at * kThreads;
    hipLaunchKernelGGL((lm_dropout<T, N, VEC>), dim3(unsigned(std::min(kMostGroups, all - at))), dim3(kThreads), 0, st, a, d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_fail("launch lm_dropout", e);
  }
  return PSGD_OK;
}

int32_t sort_size(int64_t rows) {
  int32_t n = 2;
  while (n < kSortMax && n < rows) n <<= 1;
  return n;
}

template <typename T, typename GT>
psgd_status enqueue_embed_grad(psgd_lm_plan* plan, const int64_t* tokens, const T* dout, const Drop& d, GT* table, bool add,
                               void* workspace, hipStream_t st) {
  char* ws = static_cast<char*>(workspace);
  uint64_t* keys = reinterpret_cast<uint64_t*>(ws + plan->ws_key);
  uint64_t* other = reinterpret_cast<uint64_t*>(ws + plan->ws_key2);
  const unsigned W = unsigned(plan->n_workers);
  const int32_t size = sort_size(plan->rows);
  const int64_t n = plan->vocab * plan->dim, chunks = ceil_div(plan->rows, size);
  const int64_t zeros = add ? 0 : ceil_div(n, kSortThreads * kZeroUnits * (16 / int64_t(sizeof(GT)))) * plan->n_workers;
  psgd_status s = launch(plan, kSort, lm_sort<GT>, dim3(unsigned(chunks * plan->n_workers + std::min(zeros, kZeroGroups))),
                         kSortThreads, st, tokens, plan->rows, plan->vocab, size, keys, int32_t(chunks), plan->n_workers, table, n,
                         plan->worker_stride, zeros);
  for (int64_t run = size; s == PSGD_OK && run < plan->rows; run *= 2) {
    s = launch(plan, kMerge, lm_merge, dim3(unsigned(ceil_div(plan->rows, kThreads)), W), kThreads, st,
               static_cast<const uint64_t*>(keys), other, plan->rows, run);
    std::swap(keys, other);
  }
  if (s != PSGD_OK) return s;
  const int32_t runs = int32_t(ceil_div(plan->rows, kRun)), dpad = int32_t(ceil_div(plan->dim, 4) * 4);
  const SumArgs a{keys, plan->rows, int32_t(plan->dim), dpad, runs, add ? 1 : 0, plan->worker_stride,
                  reinterpret_cast<float*>(ws + plan->ws_part)};
  const dim3 grid(unsigned(runs), unsigned(ceil_div(plan->dim, 256)), W);
  const bool wide = plan->dim >= 4;
  s = launch(plan, kSum, wide ? lm_sum<T, GT, true> : lm_sum<T, GT, false>, grid, 64, st, a, dout, table, d);
  if (s != PSGD_OK || runs == 1) return s;
  return launch(plan, kJoin, wide ? lm_join<GT, true> : lm_join<GT, false>, grid, 64 * kJoinWaves, st, a, table);
}

}  // namespace
}  // namespace lm
}  // namespace psgd

using namespace psgd;
using namespace psgd::lm;

extern "C" psgd_status psgd_lm_plan_create(const psgd_layer* layers, int32_t n_layers, int32_t table, int32_t n_workers,
                                           int64_t rows, psgd_dtype act_dtype, psgd_dtype grad_dtype, uint32_t flags,
                                           psgd_lm_plan** out) {
  if (out == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_create: out is NULL");
  *out = nullptr;
  if (layers == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_create: layers is NULL");
  if (n_layers < 1) return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_create: n_layers must be >= 1");
  if (table < 0 || table >= n_layers) return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_create: table is no tensor of the list");
  if (n_workers < 1 || n_workers > 65535)
    return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_create: n_workers must be in 1..65535");
  if (rows < 1 || rows > (int64_t(1) << 23) / n_workers)
    return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_create: n_workers * rows must be in 1..2^23");
  for (const psgd_dtype t : {act_dtype, grad_dtype})
    if (t != PSGD_F32 && t != PSGD_BF16) return refuse(PSGD_ERR_UNSUPPORTED, "psgd_lm_plan_create: unknown dtype");
  if (flags != 0) return refuse(PSGD_ERR_UNSUPPORTED, "psgd_lm_plan_create: unknown flag bits");
  psgd_lm_plan* plan = nullptr;
  try {
    plan = new psgd_lm_plan();
    int64_t off = 0;
    for (int32_t i = 0; i < n_layers; ++i) {
      const int64_t r = layers[i].rows, c = layers[i].cols;
      if (r < 1 || c < 1 || r > int64_t(0x7fffffff) / c) {
        delete plan;
        plan = nullptr;
        return fail(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_create: layer " + std::to_string(i) + " needs 1 <= rows*cols < 2^31");
      }
      if (i == table) plan->offset = off, plan->vocab = r, plan->dim = c;
      off = (off + r * c + kAlignElems - 1) / kAlignElems * kAlignElems;
    }
    plan->n_layers = n_layers;
    plan->n_workers = n_workers;
    plan->table = table;
    plan->rows = rows;
    plan->act = act_dtype;
    plan->grad = grad_dtype;
    plan->worker_stride = off;
    const int64_t n = rows * n_workers;
    plan->vb = int32_t(ceil_div(plan->vocab, kBlk));
    plan->db = int32_t(ceil_div(plan->dim, kBlk));
    plan->tb = int32_t(ceil_div(n, kBlk));
    plan->tw = int32_t(ceil_div(rows, kBlk));
    const int64_t tbp = int64_t(plan->tw) * n_workers;  // >= tb
    if (plan->dim > kMaxDim || std::max<int64_t>(tbp, plan->vb) * plan->db > kMaxBlocks) {
      delete plan;
      plan = nullptr;
      return fail(PSGD_ERR_INVALID_ARG,
                  "psgd_lm_plan_create: dim is over 2^23, or the table or the workers' rows have over 2^23 blocks of 64 x 64");
    }
    const uint64_t blk = kBlkElems * 2, p = uint64_t(parts_of(act_dtype)), gp = uint64_t(g_parts(plan));
    // pieces of about equal size, whole tiles each
    const int64_t most = std::max<int64_t>(1, kPieceBytes / int64_t(gp * blk) / tbp / kTile) * kTile;
    plan->piece = int32_t(ceil_div(ceil_div(plan->vb, ceil_div(plan->vb, most)), kTile) * kTile);
    const int64_t piece = std::min(plan->piece, plan->vb), last = plan->vb - (plan->vb - 1) / plan->piece * plan->piece;
    plan->direct = act_dtype == PSGD_BF16 && plan->dim % kBlk == 0;
    plan->loss_small = small_tiles(plan->vb, plan->tb);
    plan->scores_small = small_tiles(piece, tbp);
    // the products' tiles: of dx (rows x dim) and of the table gradients (vocabulary x dim)
    const int64_t cols = ceil_div(plan->db, kTile);
    plan->grad_small = cols * (ceil_div(tbp, kTile) + n_workers * ceil_div(piece, kTile)) < kFewTiles;
    // dx's sum over a piece is split where its tiles leave most of the chip idle, kSplitBlocks at least each
    const int64_t side = plan->grad_small ? 1 : kTile, dx_tiles = ceil_div(tbp, side) * ceil_div(plan->db, side);
    plan->splits = int32_t(std::max<int64_t>(1, std::min<int64_t>({256 / dx_tiles, 16, last / kSplitBlocks})));
    const int64_t v_tiles = ceil_div(plan->vb, plan->loss_small ? 1 : kTile);
    plan->chunk = plan->loss_small ? plan->tb : int32_t(std::max<int64_t>(1, kStatBytes / (v_tiles * kTile * kBlk * 8)) * kTile);
    uint64_t ws = 0;
    auto take = [&](uint64_t bytes) {
      const uint64_t at = ws;
      ws = a256(ws + bytes);
      return at;
    };
    plan->ws_x = take(p * uint64_t(tbp) * uint64_t(plan->db) * blk);
    if (act_dtype == PSGD_F32) {
      plan->ws_x_exps = take(uint64_t(n) * 4);
      plan->ws_w_exps = take(uint64_t(padded_words(plan->vb)) * 4);
    }
    plan->ws_w = take(plan->direct ? 0 : p * uint64_t(plan->vb) * uint64_t(plan->db) * blk);
    plan->ws_info = take(uint64_t(tbp) * kBlk * sizeof(RowInfo));
    plan->ws_count = take(uint64_t(n_workers) * 4);
    const uint64_t common = ws;
    plan->ws_stat = take(uint64_t(v_tiles) * uint64_t(std::min(plan->chunk, plan->tb)) * kBlk * 8);
    plan->ws_hit = take(uint64_t(plan->tb) * kBlk * 4);
    const uint64_t loss_end = ws;
    ws = common;
    if (act_dtype == PSGD_F32) {
      plan->ws_x3 = take(3 * uint64_t(tbp) * uint64_t(plan->db) * blk);
      plan->ws_w3 = take(3 * uint64_t(plan->vb) * uint64_t(plan->db) * blk);
    }
    plan->ws_g = take(gp * uint64_t(tbp) * uint64_t(std::min(plan->piece, plan->vb)) * blk);
    plan->ws_dx = take(uint64_t(plan->splits) * uint64_t(tbp) * kBlk * uint64_t(plan->db) * kBlk * 4);
    const uint64_t grad_end = ws;
    ws = 0;
    plan->ws_key = take(uint64_t(n) * 8);
    plan->ws_key2 = take(uint64_t(n) * 8);
    plan->ws_part = take(uint64_t(n_workers) * uint64_t(ceil_div(rows, kRun)) * 2 * uint64_t(ceil_div(plan->dim, 4)) * 16);
    plan->workspace_bytes = std::max({loss_end, grad_end, ws});
  } catch (...) {
    delete plan;
    return no_memory();
  }
  *out = plan;
  return PSGD_OK;
}

extern "C" psgd_status psgd_lm_plan_sizes(const psgd_lm_plan* plan, psgd_lm_sizes* out) {
  if (plan == nullptr || out == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_sizes: NULL argument");
  psgd_lm_sizes s{};
  s.n_layers = plan->n_layers;
  s.n_workers = plan->n_workers;
  s.table = plan->table;
  s.act_dtype = int32_t(plan->act);
  s.grad_dtype = int32_t(plan->grad);
  s.vocab = plan->vocab;
  s.dim = plan->dim;
  s.rows = plan->rows;
  s.worker_stride = plan->worker_stride;
  s.table_offset = plan->offset;
  s.workspace_bytes = plan->workspace_bytes;
  *out = s;
  return PSGD_OK;
}

extern "C" psgd_status psgd_lm_plan_destroy(psgd_lm_plan* plan) {
  if (plan == nullptr) return PSGD_OK;
  for (const PendingTiming& t : plan->pending) {
    (void)hipEventDestroy(t.start);
    (void)hipEventDestroy(t.stop);
  }
  for (hipEvent_t ev : plan->event_pool) (void)hipEventDestroy(ev);
  delete plan;
  return PSGD_OK;
}

extern "C" psgd_status psgd_lm_plan_set_timing(psgd_lm_plan* plan, int32_t enable) {
  if (plan == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_set_timing: plan is NULL");
  plan->timing = enable != 0;
  return PSGD_OK;
}

extern "C" psgd_status psgd_lm_plan_kernel_stats(psgd_lm_plan* plan, psgd_kernel_stat* out, int32_t capacity, int32_t* count,
                                                 int32_t reset) {
  if (plan == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_kernel_stats: plan is NULL");
  if (capacity > 0 && out == nullptr) return refuse(PSGD_ERR_INVALID_ARG, "psgd_lm_plan_kernel_stats: out is NULL");
  psgd_status st = PSGD_OK;
  try {
    st = collect_timings("psgd_lm_plan_kernel_stats", plan->pending, plan->event_pool, plan->stats);
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

namespace {

uint64_t size_of(psgd_dtype t) { return t == PSGD_BF16 ? 2 : 4; }

uint64_t act_bytes(const psgd_lm_plan* plan) {
  return uint64_t(plan->rows) * uint64_t(plan->n_workers) * uint64_t(plan->dim) * size_of(plan->act);
}

ArgSpan act_span(const psgd_lm_plan* plan, const char* name, const void* p, bool nullable) {
  return ArgSpan{name, p, act_bytes(plan), unsigned(size_of(plan->act)), nullable};
}

ArgSpan row_span(const psgd_lm_plan* plan, const char* name, const void* p, unsigned bytes) {
  return ArgSpan{name, p, uint64_t(plan->rows) * uint64_t(plan->n_workers) * bytes, bytes, false};
}

ArgSpan params_span(const psgd_lm_plan* plan, const void* p) {
  return ArgSpan{"params", p, uint64_t(plan->worker_stride) * size_of(plan->act), 16, false};
}

ArgSpan grads_span(const psgd_lm_plan* plan, const void* p, bool nullable) {
  return ArgSpan{"grads", p, uint64_t(plan->n_workers) * uint64_t(plan->worker_stride) * size_of(plan->grad), 16, nullable};
}

ArgSpan step_span(const psgd_dropout_config* d) { return ArgSpan{"dropout's step", d != nullptr ? d->step : nullptr, 8, 8, true}; }

}  // namespace

extern "C" psgd_status psgd_lm_embed(psgd_lm_plan* plan, const void* params, const int64_t* tokens,
                                     const psgd_dropout_config* dropout, void* out, void* stream) {
  static const char* const fn = "psgd_lm_embed";
  try {
    if (plan == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_lm_embed: plan is NULL");
    Drop d;
    psgd_status s = make_drop(fn, dropout, &d);
    if (s != PSGD_OK) return s;
    const ArgSpan spans[] = {params_span(plan, params), row_span(plan, "tokens", tokens, 8), act_span(plan, "out", out, false),
                          step_span(dropout)};
    if ((s = check_spans(fn, spans, 4)) != PSGD_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if ((s = check_capture(fn, plan, st)) != PSGD_OK) return s;
    const dim3 grid(unsigned(plan->rows * plan->n_workers), unsigned(ceil_div(plan->dim, 512)));
    const int32_t dim = int32_t(plan->dim);
    return plan->act == PSGD_F32
               ? launch(plan, kEmbed, lm_embed<float>, grid, 64, st, static_cast<const float*>(params) + plan->offset,
                        plan->vocab, dim, tokens, static_cast<float*>(out), d)
               : launch(plan, kEmbed, lm_embed<uint16_t>, grid, 64, st, static_cast<const uint16_t*>(params) + plan->offset,
                        plan->vocab, dim, tokens, static_cast<uint16_t*>(out), d);
  } catch (...) {
    return no_memory();
  }
}

extern "C" psgd_status psgd_lm_embed_grad(psgd_lm_plan* plan, const int64_t* tokens, const void* dout,
                                          const psgd_dropout_config* dropout, void* grads, uint32_t flags, void* workspace,
                                          void* stream) {
  static const char* const fn = "psgd_lm_embed_grad";
  try {
    if (plan == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_lm_embed_grad: plan is NULL");
    if (flags & ~PSGD_LM_ACCUMULATE) return fail(PSGD_ERR_UNSUPPORTED, "psgd_lm_embed_grad: unknown flag bits");
    Drop d;
    psgd_status s = make_drop(fn, dropout, &d);
    if (s != PSGD_OK) return s;
    const ArgSpan spans[] = {row_span(plan, "tokens", tokens, 8), act_span(plan, "dout", dout, false),
                          grads_span(plan, grads, false), {"workspace", workspace, plan->workspace_bytes, 16, false},
                          step_span(dropout)};
    if ((s = check_spans(fn, spans, 5)) != PSGD_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if ((s = check_capture(fn, plan, st)) != PSGD_OK) return s;
    const bool add = flags & PSGD_LM_ACCUMULATE;
    auto with = [&](auto* dy) {
      return plan->grad == PSGD_F32
                 ? enqueue_embed_grad(plan, tokens, dy, d, static_cast<float*>(grads) + plan->offset, add, workspace, st)
                 : enqueue_embed_grad(plan, tokens, dy, d, static_cast<uint16_t*>(grads) + plan->offset, add, workspace, st);
    };
    return plan->act == PSGD_F32 ? with(static_cast<const float*>(dout)) : with(static_cast<const uint16_t*>(dout));
  } catch (...) {
    return no_memory();
  }
}

extern "C" psgd_status psgd_lm_loss(psgd_lm_plan* plan, const void* x, const void* params, const int64_t* targets,
                                    const psgd_dropout_config* dropout, float* losses, float* lse, float* mean,
                                    void* workspace, void* stream) {
  static const char* const fn = "psgd_lm_loss";
  try {
    if (plan == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_lm_loss: plan is NULL");
    Drop d;
    psgd_status s = make_drop(fn, dropout, &d);
    if (s != PSGD_OK) return s;
    const ArgSpan spans[] = {act_span(plan, "x", x, false), params_span(plan, params), row_span(plan, "targets", targets, 8),
                          row_span(plan, "losses", losses, 4), row_span(plan, "lse", lse, 4),
                          {"mean", mean, uint64_t(plan->n_workers) * 4, 4, false},
                          {"workspace", workspace, plan->workspace_bytes, 16, false}, step_span(dropout)};
    if ((s = check_spans(fn, spans, 8)) != PSGD_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if ((s = check_capture(fn, plan, st)) != PSGD_OK) return s;
    return enqueue_loss(plan, x, params, targets, d, losses, lse, mean, workspace, st);
  } catch (...) {
    return no_memory();
  }
}

extern "C" psgd_status psgd_lm_loss_grad(psgd_lm_plan* plan, const void* x, const void* params, const int64_t* targets,
                                         const float* lse, const float* scale, const psgd_dropout_config* dropout, void* dx,
                                         void* grads, uint32_t flags, void* workspace, void* stream) {
  static const char* const fn = "psgd_lm_loss_grad";
  try {
    if (plan == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_lm_loss_grad: plan is NULL");
    if (flags & ~PSGD_LM_ACCUMULATE) return fail(PSGD_ERR_UNSUPPORTED, "psgd_lm_loss_grad: unknown flag bits");
    if (dx == nullptr && grads == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_lm_loss_grad: dx and grads are both NULL");
    Drop d;
    psgd_status s = make_drop(fn, dropout, &d);
    if (s != PSGD_OK) return s;
    const ArgSpan spans[] = {act_span(plan, "x", x, false), params_span(plan, params), row_span(plan, "targets", targets, 8),
                          row_span(plan, "lse", lse, 4), {"scale", scale, uint64_t(plan->n_workers) * 4, 4, true},
                          act_span(plan, "dx", dx, true), grads_span(plan, grads, true),
                          {"workspace", workspace, plan->workspace_bytes, 16, false}, step_span(dropout)};
    if ((s = check_spans(fn, spans, 9)) != PSGD_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if ((s = check_capture(fn, plan, st)) != PSGD_OK) return s;
    return enqueue_grad(plan, x, params, targets, lse, scale, d, dx, grads, (flags & PSGD_LM_ACCUMULATE) != 0, workspace, st);
  } catch (...) {
    return no_memory();
  }
}

extern "C" psgd_status psgd_dropout(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, void* out,
                                    int64_t out_stride, int64_t rows, int64_t cols, psgd_dtype dtype,
                                    const psgd_dropout_config* config, void* stream) {
  static const char* const fn = "psgd_dropout";
  try {
    if (config == nullptr) return fail(PSGD_ERR_INVALID_ARG, "psgd_dropout: config is NULL");
    if (dtype != PSGD_F32 && dtype != PSGD_BF16) return fail(PSGD_ERR_UNSUPPORTED, "psgd_dropout: unknown dtype");
    if (rows < 0 || cols < 0 || (cols > 0 && rows > (int64_t(1) << 62) / cols))
      return fail(PSGD_ERR_INVALID_ARG, "psgd_dropout: rows and cols must be >= 0, rows * cols at most 2^62");
    Drop d;
    psgd_status s = make_drop(fn, config, &d);
    if (s != PSGD_OK) return s;
    if (rows == 0 || cols == 0) return PSGD_OK;
    if (rows == 1) x_stride = residual_stride = out_stride = cols;
    if (residual == nullptr) residual_stride = cols;
    const int64_t far = std::max({x_stride, residual_stride, out_stride});
    if (std::min({x_stride, residual_stride, out_stride}) < cols || far > (int64_t(1) << 60) / rows)
      return fail(PSGD_ERR_INVALID_ARG, "psgd_dropout: a stride is less than cols, or its rows span over 2^60 elements");
    if (rows * cols >= kMostEntries) return fail(PSGD_ERR_INVALID_ARG, "psgd_dropout: rows * cols must be below 2^41");
    const unsigned e = unsigned(size_of(dtype));
    auto span = [&](const char* name, const void* p, int64_t stride, bool nullable) {
      return ArgSpan{name, p, (uint64_t(rows - 1) * uint64_t(stride) + uint64_t(cols)) * e, e, nullable};
    };
    const ArgSpan spans[] = {span("x", x, x_stride, false), span("residual", residual, residual_stride, true),
                          span("out", out, out_stride, false), step_span(config)};
    // in place: out over x, or over residual; x and residual may be one buffer (they are read)
    const bool over_x = out == x && out_stride == x_stride, over_r = out == residual && out_stride == residual_stride;
    for (int skip = 0; skip < 2; ++skip) {
      const ArgSpan three[] = {spans[skip], spans[2], spans[3]};
      const bool same = skip == 0 ? over_x : over_r;
      if ((s = check_spans(fn, three, 3, same ? 0 : -1, same ? 1 : -1)) != PSGD_OK) return s;
    }
    const hipStream_t st = static_cast<hipStream_t>(stream);
    DropArgs a{x, residual, out, x_stride, residual_stride, out_stride, rows * cols, cols, 0, Div{}};
    if (dtype == PSGD_F32) return cols % 4 == 0 ? enqueue_dropout<float, 4, true>(a, d, st) : enqueue_dropout<float, 4, false>(a, d, st);
    return cols % 8 == 0 ? enqueue_dropout<uint16_t, 8, true>(a, d, st) : enqueue_dropout<uint16_t, 4, false>(a, d, st);
  } catch (...) {
    return no_memory();
  }
}
