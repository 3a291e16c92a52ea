// train_muon.cu -- orthogonalised updates: the Newton-Schulz iteration on the tensor cores,
// and the step of momentum, iteration and weights that follows the combine.
//
// With X = G / |G| (m x n, m <= n; a taller matrix is laid out transposed) every step is
//     A = X X',   B = b A + c A A,   X <- a X + B X,
// three products, the first two of which are symmetric: only tiles that touch the lower
// triangle are computed, and written to both places.
//
// Precision.  Operands are fp16, kept times a power of two so that what is far below a
// matrix's largest values stays in the normal range; products accumulate in fp32.
// Each step multiplies small singular values by a (3.4 in the usual iteration), and with them
// the rounding errors of X that point into their directions: after five steps one rounding of
// X to bf16 is 1e-2 to 1e-1 of the result's norm, to fp16 2e-3 to 2e-2 (random, power-law and
// low-rank spectra).
// The diagonals of A and B, which dominate once the singular values are near 1, are kept apart in
// fp32, the rest of the two being fp16:
//     A A = E E + (d_i + d_j) E + d^2  with A = E + diag(d),   B X = F X + d_i X.
//   bf16 results: products of X and of A and B off their diagonals as single fp16 numbers, but X
//     itself as the sum of two for the terms a X and d_i X, where the growing errors would come from; the
//     last two steps, whose errors no longer grow, take the rounded X there too.  Off by 2e-4 to
//     1.1e-3, less than the result's rounding to bf16 (1.7e-3).  (Random, falling and equal singular
//     values, 64 x 64 to 4096 x 4096.  With the diagonals in fp16 4e-4 to 2.8e-3, in 1 to 4% less time; with both
//     parts of X in the last two steps too 1.1e-4 to 1.0e-3, in 6% more.)
//   fp32 results: X, E and F are sums of two fp16 numbers (22 bits), a product is three products
//     of them (the fourth, of the low parts, is below 2^-22); the rest is added to the product in fp32.
//     The tensor cores cut every partial sum off towards zero: 64 cut-offs along a depth of 1024 lose
//     1.4e-6 of a sum that grows evenly, which is made good by a factor (kCutOff), but up to twice that
//     where one term outweighs the others, so that sums come in runs.  Off by 2e-7 to 7e-6, fp32
//     throughout by 5e-7 to 1.1e-5: 0.2 to 1.5 times that, 2.3 times for some of a few rows in seven
//     steps.  (1024 x 4096 after five steps: 1.5e-5 without factor and diagonals apart, 1.2e-5 with the
//     factor alone, now 0.8e-6.)
#include <cuda.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "adasum_host.h"
#include "adasum_launch.h"
#include "adasum_train.cuh"
#include "adasum_umma.cuh"

namespace adasum {
namespace {

constexpr int kMaxBatch = 256;                    // matrices of one launch
constexpr int64_t kChunkBytes = int64_t(1) << 30;  // scratch of a chunk of equal matrices, about
// X and A are kept times these, B times kScaleB or less, and X times another power of two where its
// norm is far below 1 (plan_scales).
constexpr float kScaleX = 8192.f, kScaleA = 8192.f, kScaleB = 4096.f;

// What a wait that ran out leaves (adasum_get_last_error).
__device__ int g_error;
// Devices on which the iteration has been launched or captured, so that g_error may be set (of
// those beyond the last: any of them).
std::atomic<bool> g_launched[65];
int launched_index(int device) { return device >= 0 && device < 64 ? device : 64; }
constexpr long long kWaitCycles = 4000000000ll;  // a wait's limit, about two seconds
constexpr long long kSettleCycles = 4000000ll;     // what copies or products take at the very most

// ------------------------------------------------------------------ momentum and norms

// Where a matrix's elements are: 2 * start + (1: transposed).
struct Places {
  int64_t at[kMaxBatch];
};

struct SourceArgs {
  const void* x;       // the matrices, or the gradient
  float* momentum;     // null: no momentum
  int dtype;
  int64_t rows, cols, ld;  // of a matrix as the caller has it, if not transposed
  float mu;
  int nesterov;
  float* partials;     // [matrix][chunk][3]
  int* ready;          // per matrix, to be zeroed
  int* shift;          // per matrix, see FlowGroup
  int first;           // the first matrix' place among all
  int chunks;
  int64_t per_chunk;
  float eps;
  bool vec;            // x and momentum lie on 16-byte boundaries
  __half *hi, *lo;     // the first X
  int64_t m, n, ldx;
};

// Sums of squares in three ranges, so that no magnitude that fp32 holds is lost: of the
// values, of the values times 2^-64, and times 2^96.
struct Squares {
  F2 mid = f2(0.f), big = f2(0.f), small = f2(0.f);
  __device__ __forceinline__ void add(float x, float y) {
    const F2 v = f2(x, y), b = mul2(v, f2(0x1p-64f)), s = mul2(v, f2(0x1p96f));
    mid = fma2(v, v, mid);
    big = fma2(b, b, big);
    small = fma2(s, s, small);
  }
  static __device__ __forceinline__ float of_warp(F2 x) {
    const float2 p = parts(x);
    return warp_sum(p.x + p.y);
  }
};

// Eight neighbouring elements from element `at` on, of which `count` exist (others 0); vec: they
// lie on a 16-byte boundary (and are all there).
__device__ __forceinline__ void load_eight(const void* p, int dtype, int64_t at, int count, bool vec, float (&v)[8]) {
  if (vec) {
    if (dtype == kBF16) {
      const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const bf16*>(p) + at));
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    } else {
      const float4 x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at));
      const float4 y = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at) + 1);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < count ? load_any(p, dtype, at + e) : 0.f;
  }
}
// Of floats that this kernel may have written.
__device__ __forceinline__ void load_eight_own(const float* p, int count, bool vec, float (&v)[8]) {
  if (vec) {
    const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < count ? p[e] : 0.f;
  }
}
__device__ __forceinline__ void store_eight(float* p, int count, bool vec, const float (&v)[8]) {
  if (vec) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < count) p[e] = v[e];
  }
}
__device__ __forceinline__ uint32_t pack2_half(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// The high parts of eight values as fp16, and what is left of them.
__device__ __forceinline__ void split_eight(const float (&x)[8], uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 p = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
    const float2 w = __half22float2(p);
    const __half2 rest = __floats2half2_rn(x[2 * e] - w.x, x[2 * e + 1] - w.y);
    h[e] = *reinterpret_cast<const uint32_t*>(&p);
    l[e] = *reinterpret_cast<const uint32_t*>(&rest);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// v <- mu v + g (with momentum), and the sums of squares of the update, per chunk.  Bound by
// bytes: with momentum 5.9 TB/s (24 layers of 12 x 1024^2); alone, 24 x (4096 x 1024) bf16, 49 us, 4.1 TB/s,
// with four pieces a thread on their way and pairs of operations (65 piece by piece).
__global__ void __launch_bounds__(256) squares_kernel(const SourceArgs a, const __grid_constant__ Places places) {
  pdl_enter();
  __shared__ float red[3][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t start = places.at[a.first + blockIdx.y] >> 1, size = a.rows * a.cols;
  const int64_t lo = blockIdx.x * a.per_chunk, hi = min(lo + a.per_chunk, size);
  const bool dense = a.ld == a.cols, vec = a.vec && start % 8 == 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.ready[blockIdx.y] = 0;
  Squares s;
  if (dense) {
    int64_t i = lo + threadIdx.x * 8;
    if (vec && a.momentum == nullptr) {
      for (; i + 3 * 2048 + 8 <= hi; i += 4 * 2048) {
        float u[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) load_eight(a.x, a.dtype, start + i + j * 2048, 8, true, u[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 8; e += 2) s.add(u[j][e], u[j][e + 1]);
      }
    }
#pragma unroll 2
    for (; i < hi; i += 2048) {
      const int count = static_cast<int>(min(hi - i, static_cast<int64_t>(8)));
      const bool whole = vec && count == 8;
      float u[8];
      load_eight(a.x, a.dtype, start + i, count, whole, u);
      if (a.momentum) {
        float v[8];
        load_eight_own(a.momentum + start + i, count, whole, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = __fmaf_rn(a.mu, v[e], u[e]);
          u[e] = a.nesterov ? __fmaf_rn(a.mu, v[e], u[e]) : v[e];
        }
        store_eight(a.momentum + start + i, count, whole, v);
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) s.add(u[e], u[e + 1]);  // (0 where there is none)
    }
  } else {
    for (int64_t i = lo + threadIdx.x; i < hi; i += 256) s.add(load_any(a.x, a.dtype, start + i / a.cols * a.ld + i % a.cols), 0.f);
  }
  const float mid = Squares::of_warp(s.mid), big = Squares::of_warp(s.big), small = Squares::of_warp(s.small);
  if (lane == 0) red[0][warp] = mid, red[1][warp] = big, red[2][warp] = small;
  __syncthreads();
  if (threadIdx.x < 3) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[threadIdx.x][i];
    a.partials[(static_cast<int64_t>(blockIdx.y) * a.chunks + blockIdx.x) * 3 + threadIdx.x] = t;
  }
}

// X = update / (|update| + eps), times kScaleX and 2^shift, in its parts; 64 x 64 tiles, eight
// neighbours a thread on both sides.  Bound by bytes.
__global__ void __launch_bounds__(256) normalize_kernel(const SourceArgs a, const __grid_constant__ Places places) {
  pdl_enter();
  __shared__ float tile[64][65];
  __shared__ float factors[2];
  const int64_t place = places.at[a.first + blockIdx.z], start = place >> 1;
  const bool transposed = place & 1;
  if (threadIdx.x < 32) {
    const float* p = a.partials + static_cast<int64_t>(blockIdx.z) * a.chunks * 3;
    float s[3] = {0.f, 0.f, 0.f};
    for (int i = threadIdx.x; i < a.chunks; i += 32)
      for (int j = 0; j < 3; ++j) s[j] += p[i * 3 + j];
    for (int j = 0; j < 3; ++j) s[j] = warp_sum(s[j]);
    if (threadIdx.x == 0) {
      // (the middle range between 2^-80 and 2^100; NaN takes the last branch)
      float pre = 1.f, own;
      if (s[0] > 0x1p100f) pre = 0x1p-64f, own = sqrtf(s[1]);
      else if (s[0] < 0x1p-80f) pre = 0x1p96f, own = sqrtf(s[2]);
      else own = sqrtf(s[0]);
      const float norm = own + a.eps * pre;
      // X's norm is from 2^-(shift + 1) up to below 2^-shift (zeros, NaN, a norm of 1: 0)
      const int shift = own > 0.f ? max(0, 126 - static_cast<int>(__float_as_uint(own / norm) >> 23 & 255)) : 0;
      if (blockIdx.x == 0 && blockIdx.y == 0) a.shift[blockIdx.z] = shift;
      factors[0] = pre;
      factors[1] = norm > 0.f || norm != norm ? kScaleX / norm * __uint_as_float(static_cast<uint32_t>(127 + shift) << 23) : 0.f;
    }
  }
  __syncthreads();
  const float pre = factors[0], factor = factors[1];
  const int at8 = (threadIdx.x & 7) * 8, line = threadIdx.x >> 3;
  // rows and columns as the caller has them
  const int64_t rows = transposed ? a.n : a.m, cols = transposed ? a.m : a.n;
  const int64_t ld = a.momentum || a.ld == a.cols ? cols : a.ld;
  const int64_t r0 = static_cast<int64_t>(transposed ? blockIdx.x : blockIdx.y) * 64;
  const int64_t c0 = static_cast<int64_t>(transposed ? blockIdx.y : blockIdx.x) * 64;
  const bool vec = a.vec && start % 8 == 0 && ld % 8 == 0;
  auto put = [&](int64_t i, int64_t j, const float (&x)[8]) {  // (a row's last eight may reach into its padding)
    const int64_t to = (static_cast<int64_t>(blockIdx.z) * a.m + i) * a.ldx + j;
    uint4 h, l;
    split_eight(x, h, l);
    *reinterpret_cast<uint4*>(a.hi + to) = h;
    *reinterpret_cast<uint4*>(a.lo + to) = l;
  };
#pragma unroll
  for (int r = line; r < 64; r += 32) {
    if (r0 + r >= rows || c0 + at8 >= cols) continue;
    const int count = static_cast<int>(min(cols - c0 - at8, static_cast<int64_t>(8)));
    const int64_t at = start + (r0 + r) * ld + c0 + at8;
    const bool whole = vec && count == 8;
    float u[8];
    if (a.momentum) {
      load_eight_own(a.momentum + at, count, whole, u);
      if (a.nesterov) {
        float g[8];
        load_eight(a.x, a.dtype, at, count, whole, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = __fmaf_rn(a.mu, u[e], g[e]);
      }
    } else {
      load_eight(a.x, a.dtype, at, count, whole, u);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = u[e] * pre * factor;
    if (transposed) {
#pragma unroll
      for (int e = 0; e < 8; ++e) tile[r][at8 + e] = u[e];
    } else {
      put(r0 + r, c0 + at8, u);
    }
  }
  if (!transposed) return;
  __syncthreads();
#pragma unroll
  for (int c = line; c < 64; c += 32) {
    if (c0 + c >= cols || r0 + at8 >= rows) continue;
    float u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = tile[at8 + e][c];
    put(c0 + c, r0 + at8, u);
  }
}

// ------------------------------------------------------------------------- products

// The warps that take results out of TMEM and write them, in blocks of 32 rows and kCols columns.
// TERMS = 1: eight with blocks of 32 columns, which have the next block's inputs on their way (16
// warps with 16 columns: 24 x (4096 x 1024) in 2.47 ms against 1.69).  TERMS = 3: sixteen with 16
// columns, since a tile's sums are in registers for a while (eight: 8.4 ms against 4.6).
template <int TERMS>
struct Epilogue {
  static constexpr int kWarps = TERMS == 1 ? 8 : 16, kCols = TERMS == 1 ? 32 : 16;
  static constexpr int kThreads = 96 + 32 * kWarps;
  static constexpr int kGroups = kWarps / 4;               // of warps that share 32 rows
  static constexpr int kOcts = kCols / 8, kRows = 32 / kOcts, kPasses = kOcts;  // lanes a row, rows at a time
  static constexpr int kFloats = TERMS == 1 ? 32 * 33 : 32 * 16;  // of a block in shared memory
  // Place of element (r, c) of the block: no two of a row-wise or column-wise access of a warp
  // meet a bank (kCols = 16: two of the transposed one).
  static __device__ __forceinline__ int place(int r, int c) { return TERMS == 1 ? r * 33 + c : r * 16 + (c ^ ((r >> 1) & 15)); }
};

// Equal matrices that are iterated: the operands' maps (boxes of 64 x 128 and 64 x 64) and places,
// the tiles of a product.
struct FlowGroup {
  CUtensorMap x_tall[2][2], x_square[2][2], a_tall[2], a_square[2], b_tall[2];  // [buffer][part], [part]
  __half *x[2][2], *a[2], *b[2];
  float *da, *db;              // A's and B's diagonals, times kScaleA and the step's scale_b
  int64_t ldx, lda;
  int m, n, batch, first;      // the first matrix' place among all
  int col_tiles[2], tiles[2];  // of A and B (lower triangle), of X
  int* ready;                  // per matrix: warps that have written their part of a tile
  const int* shift;            // per matrix: X is first kept times 2^shift, in step k times 2^max(0, shift - growth[k])
  float step[2];               // weights: w <- keep w - step x (of a matrix as it is, transposed)
};
constexpr int kMaxGroups = 4;  // of one launch
// And where the results go.
struct FlowArgs {
  FlowGroup group[kMaxGroups];
  int groups, steps, per_step;  // tiles of a step
  int last;                     // 1: results to `dest`, 2: weights there are moved
  void* dest;
  int dest_dtype, dest_vec;     // on a 16-byte boundary
  float keep;
  float coefficients[3 * ADASUM_NEWTON_SCHULZ_MAX_STEPS];
  float scale_b[ADASUM_NEWTON_SCHULZ_MAX_STEPS];
  int growth[ADASUM_NEWTON_SCHULZ_MAX_STEPS];  // X's norm is below 2^growth times the first one's
  long long wait_cycles;
#ifdef ADASUM_TEST_HOOKS
  int held_step;                // from this one on no product is ever found written
#endif
};

enum Kind : int { kGram = 0, kPoly = 1, kApply = 2 };

// Tiles are 128 * CTAS x NT: CTAS = 2 CTAs (a cluster) share one, each with 128 of its rows, and
// each copies its rows of the left operand and its half of the columns of the right one.
// TERMS = 3: products of sums of two parts.  Their sums come in runs along the depth, each drained
// and added in fp32 registers; shorter ones for A = X X', which has squares on its diagonal and whose
// errors every later step sees: 16 cut-offs a sum.  (4096 x 4096 in one run: 9.5e-6 off after five
// steps.  A of 257 x 513 in runs of 32 cut-offs: 3.7e-6 off, of 16 1.7e-6, fp32 throughout 1.7e-6; 24 x
// (1024 x 4096) takes 1.4% more for it, its step no more.  Runs half as long for the other products too: half
// the error where the singular values fall off, 4 to 12% more time.)
template <int CTAS, int NT, int TERMS>
struct FlowShape {
  static constexpr int kHeight = 128 * CTAS;
  static constexpr int kParts = TERMS == 3 ? 2 : 1;
  static constexpr int kQRows = NT / CTAS;                           // of the right operand, of one CTA
  static constexpr int kPBytes = 128 * 128, kQBytes = kQRows * 128;  // of one part: 64 along the depth
  static constexpr int kStageBytes = kParts * (kPBytes + kQBytes);
  static constexpr int kStages = 196608 / kStageBytes < 6 ? 196608 / kStageBytes : 6;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes + Epilogue<TERMS>::kWarps * Epilogue<TERMS>::kFloats * 4;
  static_assert(kSmem + 1024 <= 232448, "with the barriers, a CTA's shared memory");
  // Two sets of 256 columns, one filled while the other is read.  TERMS = 3: half of a set for the
  // high parts' product, half for the two others.  A narrower tile's sums take turns: a product
  // waits for the one before it on the same sums.
  static constexpr int kSet = 256, kHigh = TERMS == 3 ? 128 : 256, kChains = kHigh / NT, kCols = 512;
  static_assert(NT <= kHigh, "a set holds a tile");
  // stages of 64 along the depth in a run
  __device__ static int run(int kind) { return TERMS == 1 ? 1 << 30 : kind == kGram ? 4 * kChains : 16; }
  static constexpr int kBlocks = NT / 64;  // of an epilogue warp
};

// Row tile r of a symmetric product has the column tiles up to the diagonal.
__host__ __device__ constexpr int sym_tiles(int r, int height, int nt) { return (r * height + height - 1) / nt + 1; }

// Average loss of a sum to one cut-off at fp32's 24 bits: half a unit of the last place, which is
// 2^-23 / x of a value x in [1, 2), and that 0.72 * 2^-23 on average over the logarithm of x.
// Sums grow in proportion to their terms so far, so k cut-offs take (k + 1) / 2 of them; 4 of
// products of depth 16 make a stage.
constexpr float kCutOff = 4.3e-8f;
template <int CHAINS>
__device__ __forceinline__ float cut_off(int stages) {
  return 1.f + kCutOff * (2.f / CHAINS * static_cast<float>(stages) + 0.5f);
}

struct Tile {
  int step, kind, group, matrix, row, col;  // row and column of the result where it starts
};

// All steps of the iteration in one launch of co-resident CTAs.  The tiles (128 CTAS x NT of one
// product of one matrix) of all products lie in one sequence, product after product, and CTAs
// take them in turn.  A tile needs its matrix's previous product whole, and nothing else: a
// count per matrix of what has been written tells.  Every tile waits only for tiles before it
// in the sequence, which CTAs take in order, so all waits end; and where there are several
// matrices the products of one fill the SMs while another's last tiles finish.  (One launch a
// product: 24 x (4096 x 1024) bf16 5.3 ms at the time against 2.8, one of 256 x 1024 137 us against 119.)
// Two warps copy (TMA), a thread issues the products, the others take finished sums out of TMEM.
// What bounds it: with many large matrices the results, of which a tile of 256 columns takes as long
// as its products of depth 1024, and what they and the operands move between L2 and the SMs (43 bytes a cycle
// and SM, as bytes over time): 24 x (1024 x 4096) bf16 1.75 ms (when it was 1.62 ms, 1.1 without the results'
// reads and writes, at 1.7 PFLOP/s then); fp32 4.4 ms, three times the products.  One matrix of 4096 x 4096 bf16
// in 0.96 ms, 1.4 PFLOP/s of the products that count.  Small matrices: the latency of 15 products in series, each
// about 2.5 thousand cycles until the first operands are there, 2 to 13 thousand of products, 3 of
// results and 2 until others may read them: one of 256 x 1024 in 93 us, fp32 134.
template <int CTAS, int NT, int TERMS>
__global__ void __launch_bounds__(Epilogue<TERMS>::kThreads, 1) flow_kernel(const __grid_constant__ FlowArgs a, const __grid_constant__ Places places) {
  using S = FlowShape<CTAS, NT, TERMS>;
  using E = Epilogue<TERMS>;
  extern __shared__ uint8_t raw[];
  uint8_t* stages = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  __shared__ uint64_t full[S::kStages], empty[S::kStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int stop;
  __shared__ int copied;  // tiles whose operands this CTA has found ready
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(&full[i], 2), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], E::kWarps * CTAS);
    mbar_fence_init();
    stop = 0;
    copied = 0;
  }
  if (warp == 1) tmem_alloc<S::kCols, CTAS>(&tmem_slot);
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS > 1) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int rank = CTAS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = blockIdx.x / CTAS, stride = gridDim.x / CTAS;  // of this cluster's tiles
  const int total = a.steps * a.per_step;
  auto give_up = [&] {
    if (!stop) atomicOr(&g_error, 2);
    stop = 1;
    return false;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait_pair<CTAS>(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait_pair<CTAS>(bar, parity))
      if (stop || clock64() - t0 > a.wait_cycles) return give_up();
    return true;
  };
  // The same by a whole warp, which goes on or gives up together.
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
  // until the products of its matrix before this tile's are written
  auto wait_ready = [&](const Tile& t) {
    const FlowGroup& g = a.group[t.group];
    const int need = E::kWarps * CTAS * (t.step * (2 * g.tiles[0] + g.tiles[1]) + t.kind * g.tiles[0])
#ifdef ADASUM_TEST_HOOKS
                     + (t.step >= a.held_step ? 1 << 30 : 0)
#endif
        ;
    if (load_acquire(g.ready + t.matrix) >= need) return true;
    const long long t0 = clock64();
    while (load_acquire(g.ready + t.matrix) < need) {
      if (stop || clock64() - t0 > a.wait_cycles) return give_up();
      __nanosleep(32);
    }
    return true;
  };
  auto locate = [&](int t) {
    Tile w;
    w.step = t / a.per_step;
    int r = t - w.step * a.per_step;
    w.kind = kGram;
    w.group = 0;
    for (int n; r >= (n = a.group[w.group].batch * a.group[w.group].tiles[w.kind == kApply]);) {
      r -= n;
      if (++w.group == a.groups) w.group = 0, ++w.kind;
    }
    const FlowGroup& g = a.group[w.group];
    const int tiles = g.tiles[w.kind == kApply], columns = g.col_tiles[w.kind == kApply];
    w.matrix = r / tiles;
    r -= w.matrix * tiles;
    int i = 0;
    if (w.kind == kApply) {
      i = r / columns;
      r -= i * columns;
    } else {
      for (int n; r >= (n = min(sym_tiles(i, S::kHeight, NT), columns)); ++i) r -= n;
    }
    w.row = i * S::kHeight;
    w.col = r * NT;
    return w;
  };
  auto depth = [&](const Tile& t) { return ((t.kind == kGram ? a.group[t.group].n : a.group[t.group].m) + 63) / 64; };
  // Two warps copy, the left operand's tiles and the right one's: an instruction takes its thread
  // about 100 cycles, which for both operands was more than narrow tiles' products take.
  constexpr int kCopyQ = 2 + E::kWarps;
  int issued = 0;  // whole stages whose copies this thread began
  if (warp == 0 || warp == kCopyQ) {
    if (elect_one()) {
      const bool right = warp == kCopyQ;
      const uint32_t bytes = CTAS * S::kParts * (right ? S::kQBytes : S::kPBytes);
      bool ok = true;
      int tiles = 0, s = 0;
      uint32_t phase = 1;
      for (int at = first; ok && at < total; at += stride) {
        const Tile t = locate(at);
        if (!(ok = wait_ready(t))) break;
        if (!right) store_release_cta(&copied, ++tiles);
        fence_proxy_async();
        const FlowGroup& g = a.group[t.group];
        const int ks = depth(t), b = t.step & 1;
        // (the right operand of kApply has the depth along its rows)
        const CUtensorMap* map = !right ? (t.kind == kGram ? g.x_tall[b] : t.kind == kPoly ? g.a_tall : g.b_tall)
                                 : t.kind == kApply ? g.x_square[b]
                                 : S::kQRows == 128 ? (t.kind == kGram ? g.x_tall[b] : g.a_tall)
                                                    : (t.kind == kGram ? g.x_square[b] : g.a_square);
        const int line = right ? t.col + rank * S::kQRows : t.row + rank * 128;
        for (int k = 0; k < ks; ++k, ++issued) {
          if (!(ok = wait(&empty[s], phase))) break;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          const uint32_t bar = first_of_pair<CTAS>(smem_addr(&full[s]));
          uint32_t to = smem_addr(stages) + s * S::kStageBytes + (right ? S::kParts * S::kPBytes : 0);
          if (!right || (t.kind != kApply && S::kQRows <= 128)) {
#pragma unroll
            for (int part = 0; part < S::kParts; ++part, to += right ? S::kQBytes : S::kPBytes)
              tma_load3<CTAS>(to, map + part, bar, k * 64, line, t.matrix);
          } else {
#pragma unroll
            for (int part = 0; part < S::kParts; ++part)
#pragma unroll
              for (int h = 0; h < S::kQRows / 64; ++h, to += 8192) tma_load3<CTAS>(to, map + part, bar, line + h * 64, k * 64, t.matrix);
          }
          if (++s == S::kStages) s = 0, phase ^= 1;
        }
      }
      // every stage consumed: no arrival is on its way to a CTA that has left, and no product still
      // reads shared memory or writes TMEM when they are given back
      for (int i = max(0, issued - S::kStages); ok && i < issued; ++i) ok = wait(&empty[i % S::kStages], (i / S::kStages) & 1);
      if (!ok) {
        const long long t0 = clock64();
        // Copies still in flight.  A stage whose copies have all begun tells; one that another copying
        // thread has not come to, or one of a pair's second CTA, which cannot see its copies' barrier,
        // does not, but then time has passed, for products of stages that were full too, after which
        // their thread begins no other; and a pair's CTAs leave together.
        for (int i = max(0, issued - S::kStages); rank == 0 && i < issued; ++i)
          while (!mbar_try_wait(&full[i % S::kStages], (i / S::kStages) & 1) && clock64() - t0 < kSettleCycles) {
          }
        while (clock64() - t0 < kSettleCycles) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      int acc = 0, s = 0;
      uint32_t phase = 0;
      bool ok = tmem_slot == 0;  // (all of TMEM is this CTA's, so it begins at 0, which the compiler may know)
      for (int at = first; ok && at < total; at += stride) {
        const Tile t = locate(at);
        const int ks = depth(t);
        const bool mn = t.kind == kApply;
        const int run = S::run(t.kind);
        const uint32_t idesc = mn ? umma_idesc(CTAS, NT, true) : umma_idesc(CTAS, NT, false);
        const uint32_t q_block = mn ? 8192 : 16, q_step = mn ? 128 : 2;
        int in_run = 0;
        for (int k = 0; k < ks; ++k) {
          if (in_run == 0) {
            if (!(ok = wait(&acc_empty[acc & 1], ((acc >> 1) & 1) ^ 1))) break;
            tc_fence_after();
          }
          if (!(ok = wait(&full[s], phase))) break;
          tc_fence_after();
          const uint32_t base = smem_addr(stages) + s * S::kStageBytes, qbase = base + S::kParts * S::kPBytes;
          auto multiply = [&](int p_part, int q_part, uint32_t d, bool clear) {
            const uint32_t p = umma_low(base + p_part * S::kPBytes, 16), q = umma_low(qbase + q_part * S::kQBytes, q_block);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              umma_f16<CTAS>(d + e % S::kChains * NT, p + e * 2, q + e * q_step, idesc, !clear || e >= S::kChains);
          };
          const uint32_t set = (acc & 1) * S::kSet;
          multiply(0, 0, set, in_run == 0);
          if constexpr (TERMS == 3) {
            multiply(0, 1, set + S::kHigh, in_run == 0);
            multiply(1, 0, set + S::kHigh, false);
          }
          umma_commit<CTAS>(&empty[s]);
          if (++in_run == run || k + 1 == ks) {
            umma_commit<CTAS>(&acc_full[acc & 1]);
            ++acc;
            in_run = 0;
          }
          if (++s == S::kStages) s = 0, phase ^= 1;
        }
      }
      if (!ok) give_up();
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, group = (warp - 2) >> 2;
    float* block = reinterpret_cast<float*>(stages + S::kStages * S::kStageBytes) + (warp - 2) * E::kFloats;
    const int sub = lane / E::kOcts, oct = lane % E::kOcts * 8;  // row, of kRows, and the first of eight columns
    int acc = 0, tiles = 0;
    for (int at = first; at < total; at += stride, ++tiles) {
      const Tile t = locate(at);
      const FlowGroup& g = a.group[t.group];
      const bool apply = t.kind == kApply, last_step = t.step + 1 == a.steps;
      // (TERMS = 1) parts of X in the linear term of this step and of the next
      const int in_parts = TERMS == 3 || (apply && t.step + 2 < a.steps) ? 2 : 1;
      const int out_parts = TERMS == 3 || (apply && t.step + 3 < a.steps) ? 2 : 1;
      const float c_a = a.coefficients[3 * t.step], c_b = a.coefficients[3 * t.step + 1], c_c = a.coefficients[3 * t.step + 2];
      const float scale_b = a.scale_b[t.step];
      // X's further power of two, and the next X's (the result has none)
      const int shift = __ldg(g.shift + t.matrix), here = max(0, shift - a.growth[t.step]);
      const int next_shift = last_step ? 0 : max(0, shift - a.growth[t.step + 1]);
      auto power = [](int n) { return n < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + n) << 23); };
      const float moved = apply ? power(next_shift - here) : 1.f;
      const float scale = t.kind == kGram   ? kScaleA / (kScaleX * kScaleX) * power(-2 * here)
                          : t.kind == kPoly ? c_c * (scale_b / (kScaleA * kScaleA))
                                            : moved / scale_b;
      const bool even = (t.step & 1) == 0;
      const __half *in0 = apply ? (even ? g.x[0][0] : g.x[1][0]) : g.a[0], *in1 = apply ? (even ? g.x[0][1] : g.x[1][1]) : g.a[1];
      __half *out0 = apply ? (even ? g.x[1][0] : g.x[0][0]) : t.kind == kGram ? g.a[0] : g.b[0];
      __half *out1 = apply ? (even ? g.x[1][1] : g.x[0][1]) : t.kind == kGram ? g.a[1] : g.b[1];
      const int64_t ld = apply ? g.ldx : g.lda, base = static_cast<int64_t>(t.matrix) * g.m * ld;
      const int cols = apply ? g.n : g.m, i0 = t.row + rank * 128 + quarter * 32;
      const float* diagonal_a = g.da + static_cast<int64_t>(t.matrix) * g.lda;
      auto column = [&](int k) { return t.col + (group + E::kGroups * k) * E::kCols; };
      // (of a symmetric result: the lower triangle in squares of 32 x 32)
      auto there = [&](int k) { return k < S::kBlocks && i0 < g.m && column(k) < cols && (apply || column(k) < i0 + 32); };
      // What X's row is multiplied with beside the product (kApply), or A's (kPoly: with more for
      // the column).  A's and B's diagonals are kept apart (the file's comment).
      float of_row[E::kPasses];
      // What is added, of block k: some rows' eight columns of each lane.
      struct Added {
        uint4 part[2][E::kPasses];
        float diagonal;  // kPoly: of A, the lane's column of the block
      };
      auto fetch = [&](int k, Added& f) {
        if (t.kind == kGram || !there(k)) return;
        const int c = column(k);
        if (!apply) f.diagonal = c + lane % E::kCols < cols ? __ldcg(diagonal_a + c + lane % E::kCols) : 0.f;
#pragma unroll
        for (int r = 0; r < E::kPasses; ++r) {
          const int i = i0 + r * E::kRows + sub;
          const int64_t from = base + i * ld + c + oct;
          const bool on = i < g.m && c + oct < cols;
          const uint4 none = make_uint4(0, 0, 0, 0);
          f.part[0][r] = on ? __ldcg(reinterpret_cast<const uint4*>(in0 + from)) : none;
          f.part[1][r] = on && in_parts == 2 ? __ldcg(reinterpret_cast<const uint4*>(in1 + from)) : none;
        }
      };
      auto put = [&](int64_t to, const float (&x)[8]) {
        uint4 h, l;
        if (TERMS == 3 || out_parts == 2) {
          split_eight(x, h, l);
          *reinterpret_cast<uint4*>(out1 + to) = l;
        } else {
          h = make_uint4(pack2_half(x[0], x[1]), pack2_half(x[2], x[3]), pack2_half(x[4], x[5]), pack2_half(x[6], x[7]));
        }
        *reinterpret_cast<uint4*>(out0 + to) = h;
      };
      // Eight neighbours of row `line` of the result (or column, if it is stored transposed).
      auto put_last = [&](int line, int from, int lines, int length, const float (&x)[8]) {
        if (line >= lines || from >= length) return;
        const int64_t place = places.at[g.first + t.matrix], to = (place >> 1) + static_cast<int64_t>(line) * length + from;
        const int count = min(8, length - from);
        const bool whole = a.dest_vec && length % 8 == 0 && (place >> 1) % 8 == 0;
        float y[8];
        if (a.last == 2) {
          float* w = static_cast<float*>(a.dest) + to;
          const float step = g.step[place & 1] * (1.f / kScaleX);
          load_eight_own(w, count, whole, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __fmaf_rn(-step, x[e], a.keep * y[e]);
          store_eight(w, count, whole, y);
          return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e] * (1.f / kScaleX);
        if (a.dest_dtype == kF32) {
          store_eight(static_cast<float*>(a.dest) + to, count, whole, y);
        } else if (whole) {
          *reinterpret_cast<uint4*>(static_cast<bf16*>(a.dest) + to) =
              make_uint4(pack2_bf16(y[0], y[1]), pack2_bf16(y[2], y[3]), pack2_bf16(y[4], y[5]), pack2_bf16(y[6], y[7]));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < count) static_cast<bf16*>(a.dest)[to + e] = narrow<bf16>(y[e]);
        }
      };
      const bool final = apply && last_step, transposed = final && (places.at[g.first + t.matrix] & 1);
      // Block k, whose rows' products the lanes hold.
      auto finish = [&](int k, const float (&v)[E::kCols], const Added& f) {
        const int j0 = column(k);
        const bool mirror = !apply && j0 < i0;
        __syncwarp();  // the last block has been read
#pragma unroll
        for (int c = 0; c < E::kCols; ++c) block[E::place(lane, c)] = v[c];
        __syncwarp();
        float of_column[8];  // (TERMS = 3: in every pass, for want of registers)
        auto columns = [&] {
#pragma unroll
          for (int e = 0; e < 8; ++e) of_column[e] = __shfl_sync(0xFFFFFFFFu, f.diagonal, oct + e);
        };
        if (TERMS == 1 && t.kind == kPoly) columns();
        if (!apply && !mirror) {  // a block on the diagonal: a lane has one of its elements, and leaves 0
          const int i = j0 + lane;
          if (lane < E::kCols) {
            float& at = block[E::place(i - i0, lane)];
            const float d = at * scale;
            at = 0.f;
            const int64_t to = static_cast<int64_t>(t.matrix) * g.lda + i;
            if (i < g.m && t.kind == kGram) g.da[to] = d;
            if (i < g.m && t.kind == kPoly) g.db[to] = __fmaf_rn(__fmaf_rn(scale, f.diagonal, c_b * (scale_b / kScaleA)), f.diagonal, d);
          }
          __syncwarp();
        }
        // (a row's last eight columns may reach into its padding)
#pragma unroll
        for (int r = 0; r < E::kPasses; ++r) {
          const int row = r * E::kRows + sub, i = i0 + row;
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = block[E::place(row, oct + e)] * scale;
          if (t.kind != kGram) {
            float factor[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) factor[e] = of_row[r];
            if (!apply) {
              if constexpr (TERMS == 3) columns();
#pragma unroll
              for (int e = 0; e < 8; ++e) factor[e] = __fmaf_rn(scale, of_column[e], factor[e]);
            }
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              const uint32_t w[4] = {f.part[part][r].x, f.part[part][r].y, f.part[part][r].z, f.part[part][r].w};
              if (part == 1 && in_parts == 1) break;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 y = __half22float2(*reinterpret_cast<const __half2*>(w + e));
                x[2 * e] = __fmaf_rn(factor[2 * e], y.x, x[2 * e]);
                x[2 * e + 1] = __fmaf_rn(factor[2 * e + 1], y.y, x[2 * e + 1]);
              }
            }
          }
          if (mirror || transposed) {
#pragma unroll
            for (int e = 0; e < 8; ++e) block[E::place(row, oct + e)] = x[e];
          }
          if (final) {
            if (!transposed) put_last(i, j0 + oct, g.m, cols, x);
          } else if (i < g.m && j0 + oct < cols) {
            put(base + i * ld + j0 + oct, x);
          }
        }
        if (mirror || transposed) {
          __syncwarp();
          const int row = (lane & 3) * 8;
#pragma unroll
          for (int r = 0; r < E::kCols / 8; ++r) {
            const int c = r * 8 + (lane >> 2), j = j0 + c;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = block[E::place(row + e, c)];
            if (transposed) put_last(j, i0 + row, cols, g.m, x);
            else if (j < cols && i0 + row < g.m) put(base + j * ld + i0 + row, x);
          }
        }
      };
      // (the copying warp has seen this tile's matrix ready; what it saw is visible after that)
      bool ok = true;
      const long long t0 = clock64();
      while (load_acquire_cta(&copied) <= tiles)
        if (stop || clock64() - t0 > a.wait_cycles) {
          ok = give_up();
          break;
        }
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      Added next;
      fetch(0, next);
      // (a lane's row of the diagonal)
      const float on_diagonal = t.kind == kGram || i0 + lane >= g.m ? 0.f : __ldcg((apply ? g.db : g.da) + static_cast<int64_t>(t.matrix) * g.lda + i0 + lane);
#pragma unroll
      for (int r = 0; r < E::kPasses; ++r)
        of_row[r] = __fmaf_rn(scale, __shfl_sync(0xFFFFFFFFu, on_diagonal, r * E::kRows + sub), apply ? c_a * moved : c_b * (scale_b / kScaleA));
      const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + group * E::kCols;
      auto release = [&](uint64_t* bar) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at<CTAS>(first_of_pair<CTAS>(smem_addr(bar)));
      };
      const int ks = depth(t);
      constexpr int kStep = E::kGroups * E::kCols;  // columns between a warp's blocks
      if (TERMS == 3 && ks > S::run(t.kind)) {
        float v[S::kBlocks][E::kCols];
#pragma unroll
        for (int k = 0; k < S::kBlocks; ++k)
#pragma unroll
          for (int c = 0; c < E::kCols; ++c) v[k][c] = 0.f;
        const int length = S::run(t.kind);
        for (int run = 0; ok && run < ks; run += length, ++acc) {
          if (!(ok = wait_warp(&acc_full[acc & 1], (acc >> 1) & 1))) break;
          tc_fence_after();
          const float gain = cut_off<S::kChains>(min(ks - run, length));
          const uint32_t set = from + (acc & 1) * S::kSet;
#pragma unroll
          for (int k = 0; k < S::kBlocks; ++k)
            if (there(k)) {
#pragma unroll
              for (int c = 0; c < S::kChains; ++c) {
                tmem_add<E::kCols>(set + c * NT + k * kStep, v[k], gain);
                tmem_add<E::kCols>(set + S::kHigh + c * NT + k * kStep, v[k], 1.f);
              }
            }
          release(&acc_empty[acc & 1]);
        }
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < S::kBlocks; ++k) {
          if (there(k)) finish(k, v[k], next);
          if (t.kind != kGram) fetch(k + 1, next);
        }
      } else {
        if (!wait_warp(&acc_full[acc & 1], (acc >> 1) & 1)) break;
        tc_fence_after();
        const float gain = TERMS == 3 ? cut_off<S::kChains>(ks) : 1.f;
        const uint32_t set = from + (acc & 1) * S::kSet;
#pragma unroll 1
        for (int k = 0; k < S::kBlocks; ++k) {
          const Added now = next;
          fetch(k + 1, next);
          if (!there(k)) continue;
          float v[E::kCols];
          tmem_load<E::kCols>(set + k * kStep, v);
          if constexpr (TERMS == 3) {
#pragma unroll
            for (int c = 0; c < E::kCols; ++c) v[c] *= gain;
          }
#pragma unroll
          for (int c = 1; c < S::kChains; ++c) tmem_add<E::kCols>(set + c * NT + k * kStep, v, gain);
          if constexpr (TERMS == 3) {
#pragma unroll
            for (int c = 0; c < S::kChains; ++c) tmem_add<E::kCols>(set + S::kHigh + c * NT + k * kStep, v, 1.f);
          }
          finish(k, v, now);
        }
        release(&acc_empty[acc & 1]);
        ++acc;
      }
      // what this warp wrote is there, for others' copies too
      if (!final) {
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) add_release(g.ready + t.matrix, 1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS > 1) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_free<S::kCols, CTAS>(tmem);
}

// ----------------------------------------------------------------------- host side

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

// Boxes of 64 x `box_rows` of `batch` matrices of rows x cols fp16, their rows ld apart.
bool make_map(CUtensorMap* map, const __half* p, int64_t rows, int64_t cols, int64_t ld, int64_t batch, cuuint32_t box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * static_cast<cuuint64_t>(rows) * 2};
  const cuuint32_t box[3] = {64, box_rows, 1}, ones[3] = {1, 1, 1};
  return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(p), dims, strides, box, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether results of `dtype` of matrices m x n are computed as fp32 ones are.  Of bf16 results the smallest
// are: few elements' errors do not average out, and a step's slope at a singular value may be 3.9 (16 x 16 off
// by up to 1.6e-3, 2 x 3 by 5e-3, 8 x 64 by 0.7e-3 besides the result's rounding, and two steps more by three
// times that).  One of 31 x 31 takes 72 us for it (54), 48 of 16 x 16 68 (62).
constexpr int64_t kFewElements = 1024;
bool fine_for(int dtype, int64_t m, int64_t n) { return dtype == kF32 || m * n < kFewElements; }

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Matrices of one shape m x n (m <= n) that are iterated together, and where their parts lie
// in the scratch memory.
struct ScratchMap {
  int64_t m, n, ldx, lda;
  int64_t x[2][2], a[2], b[2], da, db, partials, ready, shift, bytes;
  int chunks;
  int64_t per_chunk;
  ScratchMap(int64_t m_, int64_t n_, int64_t batch, bool fine) : m(m_), n(n_), ldx(round_up(n_, 8)), lda(round_up(m_, 8)) {
    int64_t at = 0;
    auto take = [&](int64_t count) {
      const int64_t here = at;
      at += round_up(count, 256);
      return here;
    };
    for (int i = 0; i < 2; ++i)
      for (int part = 0; part < 2; ++part) x[i][part] = take(batch * m * ldx * 2);
    for (int part = 0; part < 2; ++part) {
      a[part] = part == 0 || fine ? take(batch * m * lda * 2) : 0;
      b[part] = part == 0 || fine ? take(batch * m * lda * 2) : 0;
    }
    per_chunk = 16384;
    while ((m * n + per_chunk - 1) / per_chunk > 1024) per_chunk *= 2;
    chunks = static_cast<int>((m * n + per_chunk - 1) / per_chunk);
    partials = take(batch * chunks * 3 * 4);
    da = take(batch * lda * 4);
    db = take(batch * lda * 4);
    ready = take(batch * 4);
    shift = take(batch * 4);
    bytes = at;
  }
};
// Equal matrices, m x n once the taller ones are transposed, that are iterated in one launch, on
// their own or with others.
struct Piece {
  int64_t m, n;
  int batch;
  float step[2];  // as in FlowGroup
};
// Matrices of a piece: what about a gigabyte of scratch holds, as even as possible.
int64_t chunk_of(int64_t m, int64_t n, int64_t count, bool fine) {
  const int64_t one = ScratchMap(m, n, 1, fine).bytes;
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kMaxBatch, kChunkBytes / one));
  const int64_t chunks = (count + most - 1) / most;
  return (count + chunks - 1) / chunks;
}
// How many of the pieces from `p` on, up to `end`, one launch takes, and the scratch they need.
int take_pieces(const Piece* p, const Piece* end, bool fine, int64_t& bytes) {
  int count = 0, matrices = 0;
  bytes = 0;
  for (; p + count < end && count < kMaxGroups; ++count) {
    const int64_t more = ScratchMap(p[count].m, p[count].n, p[count].batch, fine).bytes;
    if (count > 0 && (bytes + more > kChunkBytes || matrices + p[count].batch > kMaxBatch)) break;
    bytes += more;
    matrices += p[count].batch;
  }
  return count;
}

struct Iteration {
  int steps;
  const float* coefficients;
  float eps;
};
struct Result {
  int last;  // as in FlowArgs
  void* dest;
  int dtype;
  float keep;
};

int64_t count_tiles(int64_t rows, int64_t cols, int height, int nt, bool sym) {
  const int64_t row_tiles = (rows + height - 1) / height, col_tiles = (cols + nt - 1) / nt;
  if (!sym) return row_tiles * col_tiles;
  int64_t tiles = 0;
  for (int64_t r = 0; r < row_tiles; ++r) tiles += std::min<int64_t>(sym_tiles(static_cast<int>(r), height, nt), col_tiles);
  return tiles;
}
// CTAs and columns of a tile: those for which the products of a step, one after the other, take
// least.  Wide tiles copy less for a product, narrow ones give more CTAs something to do: in
// cycles, about as measured, a tile takes `deep` for 64 along the depth and `end` for its
// results.  (us of all five steps by 2 x 256, 128 and 64 columns, bf16: 24 x (1024 x 4096) 1731,
// 2394, 3134, one of 2048 x 2048 311, 273, 372, one of 256 x 1024 187, 132, 96; by 2 x 128, 128 and 64,
// fp32: 4532, 4615, 5756; 494, 519, 665; 189, 190, 135.)
struct TileSize {
  int ctas, nt, deep, end;
};
TileSize tile_size(const Piece* p, int pieces, bool fine) {
  constexpr TileSize kBf16[3] = {{2, 256, 640, 11000}, {1, 128, 480, 7800}, {1, 64, 400, 3400}};
  constexpr TileSize kFp32[3] = {{2, 128, 850, 14000}, {1, 128, 1000, 12000}, {1, 64, 620, 6600}};
  const TileSize* const kSizes = fine ? kFp32 : kBf16;
#ifdef ADASUM_TEST_HOOKS
  if (const char* v = std::getenv("ADASUM_UPDATE_TILE"))
    if (*v >= '0' && *v <= '2' && v[1] == '\0') return kSizes[*v - '0'];
#endif
  TileSize best = kSizes[0];
  double least = 1e300;
  for (int which = 0; which < 3; ++which) {
    const TileSize& s = kSizes[which];
    const int64_t units = sm_count() / s.ctas;
    int64_t sym = 0, gen = 0, deep = 0, low = 0;  // (the deepest of the pieces' products)
    for (int i = 0; i < pieces; ++i) {
      sym += p[i].batch * count_tiles(p[i].m, p[i].m, 128 * s.ctas, s.nt, true);
      gen += p[i].batch * count_tiles(p[i].m, p[i].n, 128 * s.ctas, s.nt, false);
      deep = std::max(deep, (p[i].n + 63) / 64);
      low = std::max(low, (p[i].m + 63) / 64);
    }
    auto waves = [&](int64_t tiles) { return static_cast<double>((tiles + units - 1) / units); };
    auto tile = [&](int64_t stages) { return static_cast<double>(stages) * s.deep + s.end; };
    const double cost = waves(sym) * (tile(deep) + tile(low)) + waves(gen) * tile(low);
    if (cost < least) least = cost, best = s;
  }
  return best;
}

template <int CTAS, int NT, int TERMS>
int launch_flow_as(FlowArgs& a, const Places& places, cudaStream_t stream) {
  using S = FlowShape<CTAS, NT, TERMS>;
  static SmemAllowed allowed;
  if (int rc = allow_smem(flow_kernel<CTAS, NT, TERMS>, S::kSmem, allowed)) return rc;
  int64_t sym = 0, gen = 0;
  for (int i = 0; i < a.groups; ++i) {
    FlowGroup& g = a.group[i];
    g.col_tiles[0] = (g.m + NT - 1) / NT;
    g.col_tiles[1] = (g.n + NT - 1) / NT;
    g.tiles[0] = static_cast<int>(count_tiles(g.m, g.m, S::kHeight, NT, true));
    g.tiles[1] = static_cast<int>(count_tiles(g.m, g.n, S::kHeight, NT, false));
    sym += static_cast<int64_t>(g.batch) * g.tiles[0];
    gen += static_cast<int64_t>(g.batch) * g.tiles[1];
  }
  const int64_t most = std::max(sym, gen);
  a.per_step = static_cast<int>(2 * sym + gen);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(most, sm_count() / CTAS) * CTAS));
  cfg.blockDim = dim3(Epilogue<TERMS>::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;  // (all CTAs resident, as they wait for each other)
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CTAS > 1 ? 2 : 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, flow_kernel<CTAS, NT, TERMS>, static_cast<const FlowArgs&>(a), places));
}
template <int TERMS>
int launch_flow(FlowArgs& a, const Places& places, TileSize s, cudaStream_t stream) {
  if (s.ctas == 2) return launch_flow_as<2, TERMS == 3 ? 128 : 256, TERMS>(a, places, stream);
  if (s.nt == 128) return launch_flow_as<1, 128, TERMS>(a, places, stream);
  return launch_flow_as<1, 64, TERMS>(a, places, stream);
}

// The powers of two of every step that follow from the coefficients.  The singular values s of X are
// 1 at most at first, then what the steps so far can have made of those, and below 2.8 (the caller's
// part).
//   scale: B = b A + c A A is kept times it.  B's elements are at most its largest singular value,
// |b t + c t^2| for some t = s^2, and have to stay below fp16's 65504.  With the usual coefficients that is
// 2.8 at most, and the scale kScaleB.
//   growth: a step multiplies X's norm by |a + b t + c t^2| at most.  Where the first X is small, since
// its matrix is far below eps, it is kept times as much more (FlowGroup's shift), which later steps take back as it
// grows; else its elements would be below what fp16 holds (norms of 2^-19 off by 2e-4, of 2^-29 by 0.2).
void plan_scales(const float* coefficients, int steps, float* scale, int* growth) {
  double most = 1.01;  // singular value (roundings added)
  for (int k = 0, grown = 0; k < steps; ++k) {
    const double a = coefficients[3 * k], b = coefficients[3 * k + 1], c = coefficients[3 * k + 2], end = most * most;
    double of_b = 0.0, of_x = 0.0, gain = std::fabs(a);
    auto at = [&](double t) {  // an end or an extreme value inside
      if (!(t >= 0.0 && t <= end)) return;
      const double q = t * (b + c * t);
      of_b = std::max(of_b, std::fabs(q));
      of_x = std::max(of_x, std::sqrt(t) * std::fabs(a + q));
      gain = std::max(gain, std::fabs(a + q));
    };
    at(end);
    if (c != 0.0) {
      at(-b / (2.0 * c));
      const double root = std::sqrt(9.0 * b * b - 20.0 * a * c);  // (NaN: no extreme value)
      at((-3.0 * b + root) / (10.0 * c));
      at((-3.0 * b - root) / (10.0 * c));
    } else if (b != 0.0) {
      at(-a / (3.0 * b));
    }
    scale[k] = kScaleB;
    while (of_b * scale[k] > 65000.0) scale[k] *= 0.5f;
    growth[k] = grown;
    for (double g = 1.01 * gain; g > 1.0; g *= 0.5) ++grown;
    most = std::min(1.01 * of_x, 2.8);
  }
}

// Iterates the pieces' matrices, which are at `from`, all in one launch; the results go to `places`.
adasum_status_t iterate(SourceArgs src, const Places& from, const Places& places, const Piece* pieces, int count, bool fine,
                        const Iteration& it, const Result& res, char* scratch, cudaStream_t stream) {
  FlowArgs f = {};
  f.groups = count;
  f.steps = it.steps;
  f.last = res.last;
  f.dest = res.dest;
  f.dest_dtype = res.dtype;
  f.dest_vec = is_aligned(res.dest, 16);
  f.keep = res.keep;
  std::copy(it.coefficients, it.coefficients + 3 * it.steps, f.coefficients);
  plan_scales(it.coefficients, it.steps, f.scale_b, f.growth);
  f.wait_cycles = kWaitCycles;
#ifdef ADASUM_TEST_HOOKS
  f.held_step = it.steps;
  const char* inject = std::getenv("ADASUM_FAULT_INJECT");
  if (inject != nullptr && std::strcmp(inject, "timeout") == 0) {
    f.wait_cycles = 2000000;  // about a millisecond
    f.held_step = std::min(1, it.steps - 1);
  }
#endif
  src.eps = it.eps;
  src.vec = is_aligned(src.x, 16) && is_aligned(src.momentum, 16);
  int first = 0;
  for (int i = 0; i < count; ++i) {
    const int64_t m = pieces[i].m, n = pieces[i].n;
    const int batch = pieces[i].batch;
    const ScratchMap l(m, n, batch, fine);
    FlowGroup& g = f.group[i];
    bool ok = true;
    for (int part = 0; part < 2; ++part) {
      for (int j = 0; j < 2; ++j) {
        g.x[j][part] = reinterpret_cast<__half*>(scratch + l.x[j][part]);
        if (part > 0 && !fine) continue;
        ok = ok && make_map(&g.x_tall[j][part], g.x[j][part], m, n, l.ldx, batch, 128) &&
             make_map(&g.x_square[j][part], g.x[j][part], m, n, l.ldx, batch, 64);
      }
      if (part > 0 && !fine) continue;
      g.a[part] = reinterpret_cast<__half*>(scratch + l.a[part]);
      g.b[part] = reinterpret_cast<__half*>(scratch + l.b[part]);
      ok = ok && make_map(&g.a_tall[part], g.a[part], m, m, l.lda, batch, 128) &&
           make_map(&g.a_square[part], g.a[part], m, m, l.lda, batch, 64) && make_map(&g.b_tall[part], g.b[part], m, m, l.lda, batch, 128);
    }
    if (!ok) return ADASUM_ERR_CUDA;
    g.da = reinterpret_cast<float*>(scratch + l.da);
    g.db = reinterpret_cast<float*>(scratch + l.db);
    g.ldx = l.ldx;
    g.lda = l.lda;
    g.m = static_cast<int>(m);
    g.n = static_cast<int>(n);
    g.batch = batch;
    g.first = src.first = first;
    g.ready = src.ready = reinterpret_cast<int*>(scratch + l.ready);
    g.shift = src.shift = reinterpret_cast<int*>(scratch + l.shift);
    std::copy(pieces[i].step, pieces[i].step + 2, g.step);
    src.partials = reinterpret_cast<float*>(scratch + l.partials);
    src.chunks = l.chunks;
    src.per_chunk = l.per_chunk;
    src.hi = g.x[0][0];
    src.lo = g.x[0][1];
    src.m = m;
    src.n = n;
    src.ldx = l.ldx;
    if (src.momentum) {  // (dense)
      src.rows = m;
      src.cols = src.ld = n;
    }
    const double elements = static_cast<double>(m) * n * batch, e = dtype_bytes(src.dtype);
    adasum_status_t st = counted_launch(stream, "update_squares", elements * (e + (src.momentum ? 8 : 0)), [&] {
      return launch_pdl(squares_kernel, dim3(l.chunks, batch), dim3(256), 0, stream, src, from);
    });
    if (st) return st;
    st = counted_launch(stream, "update_normalize", elements * (e + (src.momentum ? 4 : 0) + 4), [&] {
      return launch_pdl(normalize_kernel, dim3(static_cast<unsigned>((n + 63) / 64), static_cast<unsigned>((m + 63) / 64), batch),
                        dim3(256), 0, stream, src, from);
    });
    if (st) return st;
    first += batch;
    scratch += l.bytes;
  }
  const TileSize size = tile_size(pieces, count, fine);
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return ADASUM_ERR_CUDA;
  g_launched[launched_index(device)].store(true, std::memory_order_relaxed);
  return counted_launch(stream, fine ? "update_iterate3" : "update_iterate", 0.0, [&] {
    return fine ? launch_flow<3>(f, places, size, stream) : launch_flow<1>(f, places, size, stream);
  });
}

adasum_status_t check_iteration(int steps, const float* coefficients, float eps) {
  if (steps < 1 || coefficients == nullptr || !(eps >= 0.f)) return ADASUM_ERR_INVALID_ARG;
  if (steps > ADASUM_NEWTON_SCHULZ_MAX_STEPS) return ADASUM_ERR_UNSUPPORTED;
  for (int i = 0; i < 3 * steps; ++i)
    if (!std::isfinite(coefficients[i])) return ADASUM_ERR_INVALID_ARG;
  return ADASUM_OK;
}

// The matrices of a step, equal shapes together and large ones first, and their pieces.
struct StepPlan {
  std::vector<int> order;  // segments
  std::vector<Piece> pieces;
};
StepPlan plan_step(const int64_t* rows, const int64_t* cols, int L) {
  StepPlan plan;
  for (int s = 0; s < L; ++s)
    if (rows[s] > 0 && cols[s] > 0) plan.order.push_back(s);
  auto m = [&](int s) { return std::min(rows[s], cols[s]); };
  auto n = [&](int s) { return std::max(rows[s], cols[s]); };
  std::stable_sort(plan.order.begin(), plan.order.end(), [&](int a, int b) { return m(a) != m(b) ? m(a) > m(b) : n(a) > n(b); });
  for (size_t i = 0, j; i < plan.order.size(); i = j) {
    const int s = plan.order[i];
    for (j = i + 1; j < plan.order.size() && m(plan.order[j]) == m(s) && n(plan.order[j]) == n(s);) ++j;
    const int64_t all = static_cast<int64_t>(j - i), chunk = chunk_of(m(s), n(s), all, true);
    for (int64_t done = 0; done < all; done += chunk)
      plan.pieces.push_back(Piece{m(s), n(s), static_cast<int>(std::min(chunk, all - done)), {0.f, 0.f}});
  }
  return plan;
}

bool fits(int64_t rows, int64_t cols) { return rows <= ADASUM_NEWTON_SCHULZ_MAX_DIM && cols <= ADASUM_NEWTON_SCHULZ_MAX_DIM; }

}  // namespace

int take_update_error(int device) {
  if (!g_launched[launched_index(device)].load(std::memory_order_relaxed)) return 0;
  int h = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&h, g_error, sizeof h) != cudaSuccess) return -1;
  if (h != 0 && cudaMemcpyToSymbol(g_error, &zero, sizeof zero) != cudaSuccess) return -1;
  return h;
}

}  // namespace adasum

using namespace adasum;

extern "C" {

int64_t adasum_orthogonalize_scratch_bytes(int64_t batch, int64_t rows, int64_t cols, adasum_dtype_t dtype) {
  if (batch < 1 || rows < 1 || cols < 1 || !fits(rows, cols)) return 0;
  const int64_t m = std::min(rows, cols), n = std::max(rows, cols);
  const bool fine = fine_for(dtype, m, n);
  return ScratchMap(m, n, chunk_of(m, n, batch, fine), fine).bytes;
}

adasum_status_t adasum_orthogonalize(const void* x, int64_t batch, int64_t rows, int64_t cols, int64_t batch_stride, int64_t ld,
                                     adasum_dtype_t dtype, int steps, const float* coefficients, float eps, void* out,
                                     void* scratch, int64_t scratch_bytes, adasum_stream_t stream_) {
  EntryScope scope("adasum_orthogonalize");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (batch < 0 || rows < 0 || cols < 0 || !valid_dtype(dtype)) return ADASUM_ERR_INVALID_ARG;
  if (adasum_status_t st = check_iteration(steps, coefficients, eps)) return st;
  if (!fits(rows, cols)) return ADASUM_ERR_UNSUPPORTED;
  if (batch == 0 || rows == 0 || cols == 0) return ADASUM_OK;
  const int64_t e = dtype_bytes(dtype);
  if (x == nullptr || out == nullptr || !valid_ld(rows, cols, ld) || (batch > 1 && batch_stride < (rows - 1) * ld + cols))
    return ADASUM_ERR_INVALID_ARG;
  if (batch > INT64_MAX / 64 / (rows * cols) || (batch > 1 && batch_stride > INT64_MAX / 64 / batch)) return ADASUM_ERR_UNSUPPORTED;
  const int64_t need = adasum_orthogonalize_scratch_bytes(batch, rows, cols, dtype);
  if (scratch == nullptr || scratch_bytes < need || !is_aligned(scratch, 256)) return ADASUM_ERR_INVALID_ARG;
  BufferSet set;
  set.read(x, ((batch - 1) * batch_stride + (rows - 1) * ld + cols) * e, e);
  set.write(out, batch * rows * cols * e, e);
  set.write(scratch, need, 256);
  if (adasum_status_t st = set.check()) return st;
  if (encode_tiled() == nullptr) return ADASUM_ERR_CUDA;
  const int64_t m = std::min(rows, cols), n = std::max(rows, cols);
  const bool fine = fine_for(dtype, m, n), transposed = rows > cols;
  const int64_t chunk = chunk_of(m, n, batch, fine);
  for (int64_t b0 = 0; b0 < batch; b0 += chunk) {
    const int count = static_cast<int>(std::min(chunk, batch - b0));
    Places from = {}, to = {};
    for (int i = 0; i < count; ++i) {
      from.at[i] = 2 * i * batch_stride + transposed;
      to.at[i] = 2 * i * rows * cols + transposed;
    }
    SourceArgs src = {};
    src.x = static_cast<const char*>(x) + b0 * batch_stride * e;
    src.dtype = dtype;
    src.rows = rows;
    src.cols = cols;
    src.ld = ld;
    const Result res = {1, static_cast<char*>(out) + b0 * rows * cols * e, static_cast<int>(dtype), 0.f};
    const Piece piece = {m, n, count, {0.f, 0.f}};
    if (adasum_status_t st = iterate(src, from, to, &piece, 1, fine, {steps, coefficients, eps}, res, static_cast<char*>(scratch), stream))
      return st;
  }
  return ADASUM_OK;
}

int64_t adasum_muon_step_scratch_bytes(const int64_t* rows, const int64_t* cols, int L) {
  if (rows == nullptr || cols == nullptr || L < 1) return 0;
  for (int s = 0; s < L; ++s)
    if (!fits(rows[s], cols[s])) return 0;
  try {
    const StepPlan plan = plan_step(rows, cols, L);
    int64_t most = 0, bytes = 0;
    for (size_t i = 0; i < plan.pieces.size();) {
      i += take_pieces(plan.pieces.data() + i, plan.pieces.data() + plan.pieces.size(), true, bytes);
      most = std::max(most, bytes);
    }
    return most;
  } catch (...) {  // (out of host memory)
    return -1;
  }
}

adasum_status_t adasum_muon_step(const void* grad, adasum_dtype_t dtype, const int64_t* seg_offsets, const int64_t* rows,
                                 const int64_t* cols, int L, float* master_w, float* momentum, float lr, float mu, int nesterov,
                                 float weight_decay, adasum_muon_scale_t scale, int steps, const float* coefficients, float eps,
                                 void* scratch, int64_t scratch_bytes, adasum_stream_t stream_) {
  EntryScope scope("adasum_muon_step");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (L < 0 || seg_offsets == nullptr || !valid_dtype(dtype) || scale < ADASUM_MUON_SCALE_NONE || scale > ADASUM_MUON_SCALE_RMS)
    return ADASUM_ERR_INVALID_ARG;
  if (adasum_status_t st = check_iteration(steps, coefficients, eps)) return st;
  if (seg_offsets[0] != 0 || (L > 0 && (rows == nullptr || cols == nullptr))) return ADASUM_ERR_INVALID_ARG;
  for (int s = 0; s < L; ++s) {
    if (seg_offsets[s + 1] < seg_offsets[s] || rows[s] < 0 || cols[s] < 0) return ADASUM_ERR_INVALID_ARG;
    if (rows[s] == 0 || cols[s] == 0) continue;
    if (!fits(rows[s], cols[s])) return ADASUM_ERR_UNSUPPORTED;
    if (rows[s] * cols[s] != seg_offsets[s + 1] - seg_offsets[s]) return ADASUM_ERR_INVALID_ARG;
  }
  const int64_t N = seg_offsets[L];
  if (N > INT64_MAX / 64) return ADASUM_ERR_UNSUPPORTED;
  const int64_t need = adasum_muon_step_scratch_bytes(rows, cols, L);
  if (need < 0) return ADASUM_ERR_NO_MEMORY;
  if (need == 0) return ADASUM_OK;  // no matrices
  if (grad == nullptr || master_w == nullptr || momentum == nullptr || scratch == nullptr || scratch_bytes < need ||
      !is_aligned(scratch, 256))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype);
  BufferSet set;
  set.read(grad, N * e, e);
  set.write(master_w, N * 4, 4);
  set.write(momentum, N * 4, 4);
  set.write(scratch, need, 256);
  if (adasum_status_t st = set.check()) return st;
  if (encode_tiled() == nullptr) return ADASUM_ERR_CUDA;
  try {
    StepPlan plan = plan_step(rows, cols, L);
    for (Piece& p : plan.pieces) {  // the step of a wide matrix (rows <= cols), and of a tall one
      const double wide = scale == ADASUM_MUON_SCALE_RMS ? 0.2 * std::sqrt(static_cast<double>(p.n)) : 1.0;
      const double tall = scale == ADASUM_MUON_SCALE_SPECTRAL ? std::sqrt(static_cast<double>(p.n) / static_cast<double>(p.m)) : wide;
      p.step[0] = static_cast<float>(lr * wide);
      p.step[1] = static_cast<float>(lr * tall);
    }
    SourceArgs src = {};
    src.x = grad;
    src.momentum = momentum;
    src.dtype = dtype;
    src.mu = mu;
    src.nesterov = nesterov != 0;
    const Result res = {2, master_w, kF32, static_cast<float>(1.0 - static_cast<double>(lr) * weight_decay)};
    const int* segment = plan.order.data();
    for (size_t i = 0; i < plan.pieces.size();) {
      int64_t bytes;
      const int count = take_pieces(plan.pieces.data() + i, plan.pieces.data() + plan.pieces.size(), true, bytes);
      Places places = {};
      int at = 0;
      for (int k = 0; k < count; ++k)
        for (int j = 0; j < plan.pieces[i + k].batch; ++j, ++segment)
          places.at[at++] = 2 * seg_offsets[*segment] + (rows[*segment] > cols[*segment]);
      if (adasum_status_t st = iterate(src, places, places, plan.pieces.data() + i, count, true, {steps, coefficients, eps}, res,
                                       static_cast<char*>(scratch), stream))
        return st;
      i += count;
    }
  } catch (...) {
    return ADASUM_ERR_NO_MEMORY;
  }
  return ADASUM_OK;
}

}  // extern "C"
