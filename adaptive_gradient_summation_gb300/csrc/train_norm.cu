// train_norm.cu -- layer norm, its gradient with the per-worker reduction of the
// parameters' gradients, and both with the normalised activation kept in 8 bits.
//
// Times in the comments are those of one launch between two events (the library's profiler; 4
// to 6 us of it are the launch), unless they are said to be of a call in a graph of many or of a
// pass, a call among others through the Python binding.
#include "adasum_host.h"
#include "adasum_launch.h"
#include "adasum_train.cuh"

namespace adasum {
namespace {

constexpr int kSlice = 256;        // columns of a warp's eight per lane
constexpr int kNormCtasPerSm = 2;  // of the persistent grids
constexpr int kGradCluster = 8;    // CTAs of a worker when the gradient runs as one launch

struct NormArgs {
  const void* x;
  int64_t rows, cols, ld;
  const void* weight;  // null: 1
  const void* bias;    // null: 0
  int weight_dtype;
  float eps;
  void* y;
  float* mean;         // may be null
  float* rstd;         // may be null
  int8_t* codes;       // null: no checkpoint
  float* scales;
};

// Rows of worker k are [off[k], off[k+1]) and belong to CTAs [cta_off[k], cta_off[k+1]),
// `rows_per_cta` each.
struct WorkerRows {
  int K, rows_per_cta;
  int64_t off[kMaxK + 1];
  int cta_off[kMaxK + 1];
};

struct NormGradArgs {
  const void* dy;
  int64_t ld_dy;
  const void* x;       // null: from the checkpoint
  int64_t ld_x;
  const float* mean;
  const int8_t* codes;
  const float* scales;
  const float* rstd;
  int64_t rows, cols;
  const void* weight;
  const void* bias;
  int weight_dtype;
  void* dx;
  void* y;             // null: not wanted
  float* partials;     // [CTA][weight, bias][cols]; null: parameters' gradients not wanted, or
  int cluster;         // joined by a cluster of this many CTAs per worker (0: no)
};

struct ParamGradArgs {
  const float* partials;
  int64_t cols;
  int dtype, accumulate;
  void* dw[kMaxK];     // null: not wanted
  void* db[kMaxK];
  int cta_off[kMaxK + 1];
};

// A row is shared by a team of W warps, each holding NV slices of 256 columns in registers
// (slice j * W + w for warp w), so that a row is read once.  A CTA holds TEAMS teams.
// A warp that has a whole row of one or two slices to itself takes kRows rows at a time, so
// that their sums over the lanes, chains of shuffles, run side by side: a pass over 393216 rows
// x 128 bf16 in 104 us against 186 one at a time, 196608 x 256 in 40 against 58, 98304 x 512 in
// 35 against 41.  The gradient, which has its parameters' sums in registers too, takes one row
// at every width: two lost at 512 columns and beside the checkpoint.  (At 128 columns without
// it they gained, 120 -> 97 us a pass; that form does not exist.)
template <int W, int NV>
constexpr int kRows = W == 1 && NV <= 2 ? 4 / NV : 1;

template <int W, int NV>
struct Team {
  static constexpr int kWarps = W < 8 ? 8 : W;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTeams = kWarps / W;
  static constexpr int kCols = W * NV * kSlice;
  // one team's barrier (a CTA of one team uses the CTA's)
  static __device__ __forceinline__ void sync(int team) {
    if constexpr (kTeams == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
  }
};

// Writes (or adds) one sum of a worker's weight (bias: its bias) gradient.
__device__ __forceinline__ void put_param(const ParamGradArgs& p, int k, bool bias, int64_t c, float s) {
  void* out = bias ? p.db[k] : p.dw[k];
  if (out == nullptr || c >= p.cols) return;
  if (p.accumulate) s += load_any(out, p.dtype, c);
  store_any(out, p.dtype, c, s);
}

// The weight and bias of a CTA's columns as floats in shared memory, 1 and 0 where absent.
template <int LAYOUT, int COLS, int THREADS>
__device__ __forceinline__ void stage_params(float* w, float* b, const void* weight, const void* bias, int dtype,
                                             int64_t cols) {
  for (int i = threadIdx.x; i < COLS; i += THREADS) {
    const int c = smem_col<LAYOUT>(i);
    if (w) w[i] = c < cols && weight ? load_any(weight, dtype, c) : 1.f;
    if (b) b[i] = c < cols && bias ? load_any(bias, dtype, c) : 0.f;
  }
}

// Sums over the lanes of several values side by side.
template <int R>
__device__ __forceinline__ void warp_sums(float (&v)[R]) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xFFFFFFFFu, v[r], d);
}

__device__ __forceinline__ float sum_parts(F2 x) {
  const float2 p = parts(x);
  return p.x + p.y;
}

// Zeroes the columns past the row's end in the slice where it lies.
template <int LAYOUT>
__device__ __forceinline__ void clear_past(F2 (&v)[4], int left, int lane) {
  if (left >= kSlice) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 p = parts(v[i]);
    if (lane_col<LAYOUT>(lane, 2 * i) >= left) p.x = 0.f;
    if (lane_col<LAYOUT>(lane, 2 * i + 1) >= left) p.y = 0.f;
    v[i] = f2(p.x, p.y);
  }
}

// Layer norm.  Mean and variance of a row from registers, the variance about the mean; with
// several warps a row, each has the mean and the sum of squares about it of its own columns
// and one exchange joins them: with n_w columns, mean m_w and sum of squares S_w,
//     mean = sum n_w m_w / n,   S = sum S_w + n_w (m_w - mean)^2.
// Bound by the bytes of x and y, which the next row's loads, held in registers while a row is
// worked on, keep coming: 65536 x 2048 bf16 in 90 us, 5.9 TB/s (through shared memory by
// asynchronous copies, one to three rows ahead, 101 to 105).  Rows that fill their team's
// columns (FULL) need no test per column: with the checkpoint kept 113 us against 121.
template <typename T, int LAYOUT, int W, int NV, bool KEEP, bool FULL>
__global__ void __launch_bounds__(Team<W, NV>::kThreads, W < 16 ? kNormCtasPerSm : 1) norm_kernel(const NormArgs a) {
  using TM = Team<W, NV>;
  pdl_enter();
  extern __shared__ __align__(16) float sm[];
  float *ws = sm, *bs = sm + TM::kCols;
  __shared__ float2 ex[2][TM::kTeams][W];
  stage_params<LAYOUT, TM::kCols, TM::kThreads>(ws, bs, a.weight, a.bias, a.weight_dtype, a.cols);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / W, w = warp % W;
  const float inv_n = 1.f / static_cast<float>(a.cols);
  const int64_t step = static_cast<int64_t>(gridDim.x) * TM::kTeams;
  const int64_t pitch = ckpt_pitch(a.cols), nscales = ckpt_scales(a.cols);
  int left[NV], count = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) count += left[j] = FULL ? kSlice : slice_left(a.cols, (j * W + w) * kSlice);
  const float inv_count = count > 0 ? 1.f / static_cast<float>(count) : 0.f;
  constexpr int R = kRows<W, NV>;
  Raw8<T, LAYOUT> next[R][NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r, row += step)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        next[r][j] = load8<T, LAYOUT>(static_cast<const T*>(a.x) + row * a.ld + (j * W + w) * kSlice,
                                      row < a.rows ? left[j] : 0, lane);
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * TM::kTeams + team;
  fetch(row);
  for (int it = 0; row < a.rows; row += R * step, it ^= 1) {
    F2 v[R][NV][4];
    float mean[R], sq[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < NV; ++j) unpack8<T, LAYOUT>(next[r][j], v[r][j]);
    fetch(row + R * step);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F2 acc = f2(0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = add2(acc, v[r][j][i]);
      mean[r] = sum_parts(acc);
    }
    warp_sums(mean);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] *= W == 1 ? inv_n : inv_count;
      F2 acc = f2(0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[r][j][i] = add2(v[r][j][i], f2(-mean[r]));
        clear_past<LAYOUT>(v[r][j], left[j], lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = fma2(v[r][j][i], v[r][j][i], acc);
      }
      sq[r] = sum_parts(acc);
    }
    warp_sums(sq);
    if constexpr (W > 1) {
      if (lane == 0) ex[it][team][w] = make_float2(mean[0], sq[0]);
      TM::sync(team);
      auto columns = [&](int i) {  // of warp i
        int n = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) n += FULL ? kSlice : slice_left(a.cols, (j * W + i) * kSlice);
        return static_cast<float>(n);
      };
      const float mine = mean[0];
      float total = 0.f;
      float2 p[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        p[i] = ex[it][team][i];
        total = __fmaf_rn(columns(i), p[i].x, total);
      }
      mean[0] = total * inv_n;
      sq[0] = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float d = p[i].x - mean[0];
        sq[0] += __fmaf_rn(columns(i) * d, d, p[i].y);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[0][j][i] = add2(v[0][j][i], f2(mine - mean[0]));
        if (KEEP) clear_past<LAYOUT>(v[0][j], left[j], lane);
      }
    }
    float top[KEEP ? R * NV : 1][2];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rstd[r] = 1.f / sqrtf(__fmaf_rn(sq[r], inv_n, a.eps));
      if (w == 0 && lane == 0 && row + r * step < a.rows) {
        if (a.mean) a.mean[row + r * step] = mean[r];
        if (a.rstd) a.rstd[row + r * step] = rstd[r];
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[r][j][i] = mul2(v[r][j][i], f2(rstd[r]));
        if constexpr (KEEP) block_tops<LAYOUT>(v[r][j], top[r * NV + j]);
      }
    }
    CkptScale sc[KEEP ? R * NV : 1][2];
    if constexpr (KEEP) block_scales<LAYOUT, R * NV>(top, lane, sc);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * W + w) * kSlice;
      if (left[j] <= 0) break;
      if constexpr (KEEP) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int64_t at = row + r * step;
          if (R > 1 && at >= a.rows) break;
          store_codes8<LAYOUT>(a.codes + at * pitch + c0, left[j], lane, ckpt_codes<LAYOUT>(v[r][j], sc[r * NV + j]));
          store_scales<LAYOUT>(a.scales + at * nscales + c0 / kCkptBlock, left[j], lane, sc[r * NV + j]);
        }
      }
      F2 wv[4], bv[4];
      lds8(ws + c0, lane, wv);
      lds8(bs + c0, lane, bv);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t at = row + r * step;
        if (R > 1 && at >= a.rows) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[r][j][i] = fma2(v[r][j][i], wv[i], bv[i]);
        store8<T, LAYOUT>(static_cast<T*>(a.y) + at * a.cols + c0, left[j], lane, v[r][j]);
      }
    }
  }
}

// Rows of dy and x (or of h's codes) on their way to the gradient kernel, one warp's part.
// A lane copies the bytes that it will use itself, kStages rows ahead, so that the copies take
// no registers and need no barrier (N = 1: no row ahead).
template <typename T, int N, int NV, bool KEPT>
struct RowCopy {
  LaneSlot<T, N> dy[NV], x[NV];
};
template <typename T, int N, int NV>
struct RowCopy<T, N, NV, true> {
  LaneSlot<T, N> dy[NV];
  alignas(8) uint32_t q[NV][8 / N][32][N == kVec8 ? 2 : 1];  // codes
};
template <typename T, int W, int NV>
struct GradShape {
  // (three stages: 73.4 us where two take 72.1; one where two rows of 64 KiB do not fit)
  static constexpr int kStages = W * NV > 32 && sizeof(T) == 4 ? 1 : 2;
  // g and h of the row are computed twice instead of kept in registers, which the parameters'
  // sums of four slices leave no room for
  static constexpr bool kTwice = NV > 2;
  static constexpr int kCtas = W < 16 ? kNormCtasPerSm : 1;
};

// The gradient.  With g = dy w and h the normalised row,
//     dx = rstd (g - mean(g) - h mean(g h)),   dw += dy h,   db += dy:
// one read of dy and x (or of h's codes), two sums per row, and the parameters' sums of a
// CTA's rows in registers, joined over its teams at the end and written as the CTA's partial.
// A CTA's rows all belong to one worker.  Bound by the bytes of dy, x and dx: 65536 x 1024 bf16
// of 16 workers in 72 us, 5.6 TB/s; from codes, 65536 x 2048 with the output once more, 159 us,
// 5.9 TB/s.
template <typename T, int LAYOUT, int W, int NV, bool KEPT, bool FULL>
__global__ void __launch_bounds__(Team<W, NV>::kThreads, GradShape<T, W, NV>::kCtas)
    norm_grad_kernel(const NormGradArgs a, const __grid_constant__ WorkerRows rows,
                     const __grid_constant__ ParamGradArgs params) {
  using TM = Team<W, NV>;
  using Copy = RowCopy<T, LAYOUT, NV, KEPT>;
  constexpr int S = GradShape<T, W, NV>::kStages;
  constexpr bool kTwice = GradShape<T, W, NV>::kTwice;
  pdl_enter();
  extern __shared__ __align__(16) float sm[];  // weight, bias (KEPT), copies; at the end the teams' sums
  float *ws = sm, *bs = sm + TM::kCols;
  Copy* copies = reinterpret_cast<Copy*>(sm + (KEPT ? 2 : 1) * TM::kCols);
  __shared__ float2 ex[2][TM::kTeams][W];
  stage_params<LAYOUT, TM::kCols, TM::kThreads>(ws, KEPT ? bs : nullptr, a.weight, a.bias, a.weight_dtype, a.cols);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / W, w = warp % W;
  const float inv_n = 1.f / static_cast<float>(a.cols);
  const int64_t pitch = ckpt_pitch(a.cols), nscales = ckpt_scales(a.cols);
  int k = 0;
  int64_t r0, r1;
  if (a.cluster) {
    k = blockIdx.x / a.cluster;
    const int64_t per = (rows.off[k + 1] - rows.off[k] + a.cluster - 1) / a.cluster;
    r0 = rows.off[k] + static_cast<int64_t>(blockIdx.x - k * a.cluster) * per;
    r1 = min(r0 + per, rows.off[k + 1]);
  } else {
    for (int hi = rows.K; hi - k > 1;) {
      const int m = (k + hi) >> 1;
      if (rows.cta_off[m] <= static_cast<int>(blockIdx.x)) k = m;
      else hi = m;
    }
    r0 = rows.off[k] + static_cast<int64_t>(blockIdx.x - rows.cta_off[k]) * rows.rows_per_cta;
    r1 = min(r0 + rows.rows_per_cta, rows.off[k + 1]);
  }
  int left[NV];
  F2 dw[NV][4], db[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    left[j] = FULL ? kSlice : slice_left(a.cols, (j * W + w) * kSlice);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = db[j][i] = f2(0.f);
  }
  auto issue = [&](int64_t row, int stage) {
    if constexpr (LAYOUT != kStrided) {
      if (row < r1) {
        Copy& c = copies[stage * TM::kWarps + warp];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c0 = (j * W + w) * kSlice;
          c.dy[j].copy(static_cast<const T*>(a.dy) + row * a.ld_dy + c0, left[j], lane);
          if constexpr (!KEPT) {
            c.x[j].copy(static_cast<const T*>(a.x) + row * a.ld_x + c0, left[j], lane);
          } else {  // (rows of codes are padded, so a begun piece is always there)
#pragma unroll
            for (int i = 0; i < 8 / LAYOUT; ++i) {
              const int at = lane_col<LAYOUT>(lane, i * LAYOUT);
              const bool in = at < left[j];
              cp_async_small<LAYOUT>(smem_addr(c.q[j][i][lane]), a.codes + row * pitch + c0 + (in ? at : 0), in ? LAYOUT : 0);
            }
          }
        }
      }
      cp_async_commit();
    }
  };
  // dy and h of slice j of the row; N = 1: from `raw`, loaded by `load_raw`
  struct Raw {
    Raw8<T, LAYOUT> dy[LAYOUT != kStrided ? 1 : NV], x[LAYOUT != kStrided || KEPT ? 1 : NV];
    uint2 q[LAYOUT == kStrided && KEPT ? NV : 1];
  } raw;
  auto load_raw = [&](int64_t row, int j) {
    const int c0 = (j * W + w) * kSlice;
    raw.dy[j] = load8<T, LAYOUT>(static_cast<const T*>(a.dy) + row * a.ld_dy + c0, left[j], lane);
    if constexpr (KEPT) raw.q[j] = load_codes8<LAYOUT>(a.codes + row * pitch + c0, left[j], lane);
    else raw.x[j] = load8<T, LAYOUT>(static_cast<const T*>(a.x) + row * a.ld_x + c0, left[j], lane);
  };
  auto take = [&](int stage, int j, float mean, float rstd, float s0, float s1, F2 (&dy)[4], F2 (&h)[4]) {
    if constexpr (LAYOUT != kStrided) {
      const Copy& c = copies[stage * TM::kWarps + warp];
      unpack8<T, LAYOUT>(c.dy[j].take(lane), dy);
      if constexpr (!KEPT) unpack8<T, LAYOUT>(c.x[j].take(lane), h);
      else if constexpr (LAYOUT == kVec8) ckpt_values8(*reinterpret_cast<const uint2*>(c.q[j][0][lane]), s0, s1, h);
      else ckpt_values8(make_uint2(c.q[j][0][lane][0], c.q[j][1][lane][0]), s0, s1, h);
    } else {
      unpack8<T, LAYOUT>(raw.dy[j], dy);
      if constexpr (KEPT) ckpt_values8(raw.q[j], s0, s1, h);
      else unpack8<T, LAYOUT>(raw.x[j], h);
    }
    if constexpr (!KEPT) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = mul2(add2(h[i], f2(-mean)), f2(rstd));
      clear_past<LAYOUT>(h, left[j], lane);
    }
  };
  int64_t row = r0 + team;
#pragma unroll
  for (int s = 0; s < S; ++s) issue(row + s * TM::kTeams, s);
  struct Stats {
    float mean, rstd, scale[KEPT ? NV : 1][2];
  } next;
  auto stats = [&](int64_t row) {
    const bool in = row < r1;
    next.mean = !KEPT && in ? a.mean[row] : 0.f;
    next.rstd = in ? a.rstd[row] : 0.f;
    if constexpr (KEPT) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int n = in ? left[j] : 0;
        const float* s = a.scales + row * nscales + (j * W + w) * (kSlice / kCkptBlock);
        if constexpr (LAYOUT == kVec8) {
          next.scale[j][0] = next.scale[j][1] = lane * 8 < n ? s[lane >> 4] : 0.f;
        } else {
          next.scale[j][0] = n > 0 ? s[0] : 0.f;
          next.scale[j][1] = n > kCkptBlock ? s[1] : 0.f;
        }
      }
    }
  };
  stats(row);
  int stage = 0;
  for (int it = 0; row < r1; row += TM::kTeams, it ^= 1, stage = stage + 1 == S ? 0 : stage + 1) {
    const Stats cur = next;
    stats(row + TM::kTeams);
    if constexpr (LAYOUT != kStrided) {
      cp_async_wait<S - 1>();
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) load_raw(row, j);
    }
    F2 g[kTwice ? 1 : NV][4], h[kTwice ? 1 : NV][4], sg2 = f2(0.f), sgh2 = f2(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = kTwice ? 0 : j;
      take(stage, j, cur.mean, cur.rstd, cur.scale[KEPT ? j : 0][0], cur.scale[KEPT ? j : 0][1], g[at], h[at]);
      F2 wv[4];
      lds8(ws + (j * W + w) * kSlice, lane, wv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dw[j][i] = fma2(g[at][i], h[at][i], dw[j][i]);
        db[j][i] = add2(g[at][i], db[j][i]);
        g[at][i] = mul2(g[at][i], wv[i]);
        sg2 = add2(sg2, g[at][i]);
        sgh2 = fma2(g[at][i], h[at][i], sgh2);
      }
    }
    if constexpr (!kTwice) issue(row + S * TM::kTeams, stage);
    float sg = warp_sum(sum_parts(sg2)), sgh = warp_sum(sum_parts(sgh2));
    if constexpr (W > 1) {
      if (lane == 0) ex[it][team][w] = make_float2(sg, sgh);
      TM::sync(team);
      sg = sgh = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        sg += ex[it][team][i].x;
        sgh += ex[it][team][i].y;
      }
    }
    const F2 mg = f2(-sg * inv_n * cur.rstd), mgh = f2(-sgh * inv_n * cur.rstd), r = f2(cur.rstd);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * W + w) * kSlice, at = kTwice ? 0 : j;
      if (left[j] <= 0) break;
      F2 wv[4];
      if (kTwice || (KEPT && a.y != nullptr)) lds8(ws + c0, lane, wv);
      if constexpr (kTwice) {
        take(stage, j, cur.mean, cur.rstd, cur.scale[KEPT ? j : 0][0], cur.scale[KEPT ? j : 0][1], g[0], h[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[0][i] = mul2(g[0][i], wv[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) g[at][i] = fma2(h[at][i], mgh, fma2(g[at][i], r, mg));
      store8<T, LAYOUT>(static_cast<T*>(a.dx) + row * a.cols + c0, left[j], lane, g[at]);
      if (KEPT && a.y != nullptr) {
        F2 bv[4];
        lds8(bs + c0, lane, bv);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[at][i] = fma2(h[at][i], wv[i], bv[i]);
        store8<T, LAYOUT>(static_cast<T*>(a.y) + row * a.cols + c0, left[j], lane, h[at]);
      }
    }
    if constexpr (kTwice) issue(row + S * TM::kTeams, stage);
  }
  if (a.partials == nullptr && a.cluster == 0) return;
  // the teams' sums in shared memory, the first team's place taking their total
  if constexpr (LAYOUT != kStrided) cp_async_wait<0>();
  __syncthreads();
  float* mine = sm + team * 2 * TM::kCols;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    sts8(mine + (j * W + w) * kSlice, lane, dw[j]);
    sts8(mine + TM::kCols + (j * W + w) * kSlice, lane, db[j]);
  }
  __syncthreads();
  float* out = a.cluster ? nullptr : a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  for (int i = threadIdx.x; i < 2 * TM::kCols; i += TM::kThreads) {
    const int c = smem_col<LAYOUT>(i % TM::kCols);
    float s = sm[i];
#pragma unroll
    for (int t = 1; t < TM::kTeams; ++t) s += sm[t * 2 * TM::kCols + i];
    if (a.cluster) sm[i] = s;
    else if (c < a.cols) out[(i / TM::kCols) * a.cols + c] = s;
  }
  if (a.cluster == 0) return;
  // few rows: the worker's CTAs are one cluster, and each adds its share of the columns over
  // them, in their order
  cluster_sync_all();
  const int share = 2 * TM::kCols / kGradCluster, rank = static_cast<int>(cluster_ctarank());
  for (int i = rank * share + threadIdx.x; i < (rank + 1) * share; i += TM::kThreads) {
    const int c = smem_col<LAYOUT>(i % TM::kCols);
    float v[kGradCluster], s = 0.f;
#pragma unroll
    for (int r = 0; r < kGradCluster; ++r) v[r] = *map_rank(sm + i, r);
#pragma unroll
    for (int r = 0; r < kGradCluster; ++r) s += v[r];
    put_param(params, k, i >= TM::kCols, c, s);
  }
  cluster_sync_all();  // the others may still read this CTA's sums
}

// Joins the CTAs' partials of one worker: 32 columns per CTA, eight partials at a time.  Bound
// by latency: 2.5 MB of 16 workers x 1024 columns in 7 us.
__global__ void __launch_bounds__(256) norm_params_kernel(const __grid_constant__ ParamGradArgs p) {
  pdl_enter();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = blockIdx.y;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // weight columns, then bias columns
  float s = 0.f;
  if (i < 2 * p.cols) {
#pragma unroll 4
    for (int c = p.cta_off[k] + warp; c < p.cta_off[k + 1]; c += 8) s += p.partials[c * 2 * p.cols + i];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp > 0 || i >= 2 * p.cols) return;
#pragma unroll
  for (int j = 1; j < 8; ++j) s += red[j][lane];
  put_param(p, k, i >= p.cols, i < p.cols ? i : i - p.cols, s);
}

template <typename T, int LAYOUT, int W, int NV>
int launch_norm_as(const NormArgs& a, cudaStream_t stream) {
  using TM = Team<W, NV>;
  const size_t smem = 2 * TM::kCols * sizeof(float);
  static SmemAllowed allowed[2][2];
  const bool full = LAYOUT != kStrided && a.cols == TM::kCols, keep = a.codes != nullptr;
  constexpr bool kCan = LAYOUT != kStrided;
  auto kernel = full ? (keep ? norm_kernel<T, LAYOUT, W, NV, true, kCan> : norm_kernel<T, LAYOUT, W, NV, false, kCan>)
                     : (keep ? norm_kernel<T, LAYOUT, W, NV, true, false> : norm_kernel<T, LAYOUT, W, NV, false, false>);
  if (int rc = allow_smem(kernel, smem, allowed[full][keep])) return rc;
  const int64_t need = (a.rows + TM::kTeams - 1) / TM::kTeams;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(need, static_cast<int64_t>(kNormCtasPerSm) * sm_count()));
  return launch_pdl(kernel, dim3(grid), dim3(TM::kThreads), smem, stream, a);
}
// The smallest team that holds a row: up to four slices a warp, then more warps.  (Two slices a
// warp: 65536 x 2048 bf16 109 us against 90, with the checkpoint 132 against 113, as a row's
// sums over the lanes and its exchange between warps are then spread over fewer bytes.)
// Above 8192 columns a CTA of 16 warps has an SM to itself and one row on its way: passes over
// 16384 columns run at 4.3 TB/s, the gradient's, whose sums do not all stay in registers, at 3.4.
template <typename T, int LAYOUT>
int launch_norm(const NormArgs& a, cudaStream_t stream) {
  const int64_t slices = (a.cols + kSlice - 1) / kSlice;
  if (slices <= 1) return launch_norm_as<T, LAYOUT, 1, 1>(a, stream);
  if (slices <= 2) return launch_norm_as<T, LAYOUT, 1, 2>(a, stream);
  if (slices <= 4) return launch_norm_as<T, LAYOUT, 1, 4>(a, stream);
  if (slices <= 8) return launch_norm_as<T, LAYOUT, 2, 4>(a, stream);
  if (slices <= 16) return launch_norm_as<T, LAYOUT, 4, 4>(a, stream);
  if (slices <= 32) return launch_norm_as<T, LAYOUT, 8, 4>(a, stream);
  return launch_norm_as<T, LAYOUT, 16, 4>(a, stream);
}

template <typename T, int LAYOUT, int W, int NV, bool KEPT>
int launch_norm_grad_as(const NormGradArgs& a, const WorkerRows& rows, const ParamGradArgs& params, cudaStream_t stream) {
  using TM = Team<W, NV>;
  const size_t work = (KEPT ? 2 : 1) * TM::kCols * sizeof(float) +
                      (LAYOUT != kStrided ? GradShape<T, W, NV>::kStages * TM::kWarps * sizeof(RowCopy<T, LAYOUT, NV, KEPT>) : 0);
  const size_t sums = TM::kTeams * 2 * TM::kCols * sizeof(float);
  const size_t smem = std::max(work, sums);
  static SmemAllowed allowed[2];
  constexpr bool kCan = LAYOUT != kStrided;
  const bool full = kCan && a.cols == TM::kCols;
  auto kernel = full ? norm_grad_kernel<T, LAYOUT, W, NV, KEPT, kCan> : norm_grad_kernel<T, LAYOUT, W, NV, KEPT, false>;
  if (int rc = allow_smem(kernel, smem, allowed[full])) return rc;
  if (a.cluster)
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(rows.K * a.cluster)), dim3(TM::kThreads), a.cluster, smem,
                              stream, a, rows, params);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(rows.cta_off[rows.K])), dim3(TM::kThreads), smem, stream, a, rows, params);
}
// Teams of the gradient kernel: two slices a warp, since each costs 16 registers of sums
// (65536 x 1024 bf16 72 us, with four slices 148; 128 rows from codes 14 and 18).
int grad_teams(int64_t cols) {
  const int64_t slices = (cols + kSlice - 1) / kSlice;
  return slices <= 2 ? 8 : slices <= 4 ? 4 : slices <= 8 ? 2 : 1;
}
template <typename T, int LAYOUT, bool KEPT>
int launch_norm_grad_kept(const NormGradArgs& a, const WorkerRows& rows, const ParamGradArgs& p, cudaStream_t stream) {
  const int64_t slices = (a.cols + kSlice - 1) / kSlice;
  if (slices <= 1) return launch_norm_grad_as<T, LAYOUT, 1, 1, KEPT>(a, rows, p, stream);
  if (slices <= 2) return launch_norm_grad_as<T, LAYOUT, 1, 2, KEPT>(a, rows, p, stream);
  if (slices <= 4) return launch_norm_grad_as<T, LAYOUT, 2, 2, KEPT>(a, rows, p, stream);
  if (slices <= 8) return launch_norm_grad_as<T, LAYOUT, 4, 2, KEPT>(a, rows, p, stream);
  if (slices <= 16) return launch_norm_grad_as<T, LAYOUT, 8, 2, KEPT>(a, rows, p, stream);
  if (slices <= 32) return launch_norm_grad_as<T, LAYOUT, 16, 2, KEPT>(a, rows, p, stream);
  return launch_norm_grad_as<T, LAYOUT, 16, 4, KEPT>(a, rows, p, stream);
}
template <typename T, int LAYOUT>
int launch_norm_grad(const NormGradArgs& a, const WorkerRows& rows, const ParamGradArgs& p, cudaStream_t stream) {
  return a.codes ? launch_norm_grad_kept<T, LAYOUT, true>(a, rows, p, stream)
                 : launch_norm_grad_kept<T, LAYOUT, false>(a, rows, p, stream);
}

// Whether the gradient's sums are joined by clusters in the same launch.  That saves the host
// a launch, the scratch memory and its size: 10 us of a pass of 50.  The
// device takes longer, since a worker's rows have eight CTAs only: 1 us of 5 at 4 rows a team
// (128 x 1024 bf16, replayed from a graph), 2 of 6 at 8, 5 of 6 at 16 and 10 of 9 at 32.  So
// up to 16 rows a team for the worker with the most.
bool one_launch(const int64_t* offs, int K, int64_t cols) {
  if (K > 32) return false;
  const int64_t most = static_cast<int64_t>(16) * kGradCluster * grad_teams(cols);
  for (int k = 0; k < K; ++k)
    if (offs[k + 1] - offs[k] > most) return false;
  return true;
}

// Deals the workers' rows to at most about `target` CTAs, none of them to two workers.
void deal_rows(WorkerRows& r, const int64_t* offs, int K, int teams, int target) {
  r.K = K;
  for (int k = 0; k <= K; ++k) r.off[k] = offs[k];
  const int64_t rows = offs[K];
  int64_t per = std::max<int64_t>(teams, (rows + target - 1) / target);
  for (;;) {
    per = (per + teams - 1) / teams * teams;
    int64_t ctas = 0;
    for (int k = 0; k < K; ++k) {
      ctas += (offs[k + 1] - offs[k] + per - 1) / per;
      r.cta_off[k + 1] = static_cast<int>(ctas);
    }
    if (ctas <= target || per >= rows) break;
    per += std::max<int64_t>(1, per / 16);
  }
  r.rows_per_cta = static_cast<int>(std::min<int64_t>(per, INT32_MAX));
}

// Size and type checks shared by the norm entry points.
adasum_status_t check_norm(int64_t rows, int64_t cols, int dtype, int weight_dtype) {
  if (rows < 0 || cols < 1 || !valid_dtype(dtype) || !valid_dtype(weight_dtype)) return ADASUM_ERR_INVALID_ARG;
  if (cols > ADASUM_NORM_MAX_COLS || rows > INT32_MAX) return ADASUM_ERR_UNSUPPORTED;
  return ADASUM_OK;
}

adasum_status_t norm_backward(NormGradArgs a, int dtype, const int64_t* offs, int K, void* const* dw,
                              void* const* db, int grad_dtype, int accumulate, void* scratch,
                              int64_t scratch_bytes, cudaStream_t stream) {
  if (adasum_status_t st = check_worker_offsets(offs, K)) return st;
  a.rows = offs[K];
  if (adasum_status_t st = check_norm(a.rows, a.cols, dtype, a.weight_dtype)) return st;
  if (!valid_dtype(grad_dtype)) return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype), we = dtype_bytes(a.weight_dtype), ge = dtype_bytes(grad_dtype);
  const bool kept = a.codes != nullptr;
  const bool want = dw != nullptr || db != nullptr;
  if (a.rows > 0) {
    if (a.dy == nullptr || a.rstd == nullptr || a.dx == nullptr) return ADASUM_ERR_INVALID_ARG;
    if (kept ? a.scales == nullptr : (a.x == nullptr || a.mean == nullptr)) return ADASUM_ERR_INVALID_ARG;
    if (!valid_ld(a.rows, a.cols, a.ld_dy) || (!kept && !valid_ld(a.rows, a.cols, a.ld_x)) || (kept && !is_aligned(a.codes, 16)))
      return ADASUM_ERR_INVALID_ARG;
  }
  const int64_t need = adasum_layer_norm_backward_scratch_bytes(offs, K, a.cols);
  if (want && need > 0 && (scratch == nullptr || scratch_bytes < need || !is_aligned(scratch, 256)))
    return ADASUM_ERR_INVALID_ARG;
  WorkerRows rows = {};
  ParamGradArgs p = {};
  BufferSet set;
  set.read(a.dy, span_bytes(a.rows, a.cols, a.ld_dy, e), e);
  if (kept) {
    set.read(a.codes, a.rows * ckpt_pitch(a.cols), 16);
    set.read(a.scales, a.rows * ckpt_scales(a.cols) * 4, 4);
  } else {
    set.read(a.x, span_bytes(a.rows, a.cols, a.ld_x, e), e);
    set.read(a.mean, a.rows * 4, 4);
  }
  set.read(a.rstd, a.rows * 4, 4);
  set.read(a.weight, a.cols * we, we);
  set.read(a.bias, a.cols * we, we);
  set.write(a.dx, a.rows * a.cols * e, e);
  set.write(a.y, a.rows * a.cols * e, e);
  if (want) set.write(scratch, need, 256);
  for (int k = 0; k < K; ++k) {
    if (dw != nullptr) {
      if (dw[k] == nullptr) return ADASUM_ERR_INVALID_ARG;
      set.write(p.dw[k] = dw[k], a.cols * ge, ge);
    }
    if (db != nullptr) {
      if (db[k] == nullptr) return ADASUM_ERR_INVALID_ARG;
      set.write(p.db[k] = db[k], a.cols * ge, ge);
    }
  }
  if (adasum_status_t st = set.check()) return st;
  const double n = static_cast<double>(a.rows) * a.cols;
  deal_rows(rows, offs, K, grad_teams(a.cols), kNormCtasPerSm * sm_count());
  p.cols = a.cols;
  p.dtype = grad_dtype;
  p.accumulate = accumulate != 0;
  const bool joined = want && a.rows > 0 && one_launch(offs, K, a.cols);
  a.cluster = joined ? kGradCluster : 0;
  const bool vec = is_aligned(a.dy, 16) && is_aligned(a.dx, 16) && is_aligned(a.y, 16) && a.ld_dy * e % 16 == 0 &&
                   a.cols * e % 16 == 0 && (kept || (is_aligned(a.x, 16) && a.ld_x * e % 16 == 0));
  a.partials = want && !joined ? static_cast<float*>(scratch) : nullptr;
  if (a.rows > 0)
    if (adasum_status_t st = counted_launch(stream, kept ? "norm_grad_checkpoint" : "norm_grad",
                                            n * (kept ? 2 * e + 1 + (a.y ? e : 0) : 3 * e), [&] {
          if (dtype == kBF16)
            return vec ? launch_norm_grad<bf16, kVec8>(a, rows, p, stream) : launch_norm_grad<bf16, kStrided>(a, rows, p, stream);
          return vec ? launch_norm_grad<float, kVec4>(a, rows, p, stream) : launch_norm_grad<float, kStrided>(a, rows, p, stream);
        }))
      return st;
  if (!want || joined) return ADASUM_OK;
  p.partials = a.partials;
  std::copy(rows.cta_off, rows.cta_off + K + 1, p.cta_off);
  return counted_launch(stream, "norm_params", 0.0, [&] {
    return launch_pdl(norm_params_kernel, dim3(static_cast<unsigned>((2 * a.cols + 31) / 32), K), dim3(256), 0, stream, p);
  });
}

}  // namespace
}  // namespace adasum

using namespace adasum;

extern "C" {

adasum_status_t adasum_layer_norm(const void* x, int64_t rows, int64_t cols, int64_t ld, adasum_dtype_t dtype,
                                  const void* weight, const void* bias, adasum_dtype_t weight_dtype, float eps,
                                  void* y, float* mean, float* rstd, int8_t* codes, float* scales,
                                  adasum_stream_t stream_) {
  EntryScope scope("adasum_layer_norm");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (adasum_status_t st = check_norm(rows, cols, dtype, weight_dtype)) return st;
  if ((codes == nullptr) != (scales == nullptr) || !(eps >= 0.f)) return ADASUM_ERR_INVALID_ARG;
  if (rows == 0) return ADASUM_OK;
  if (x == nullptr || y == nullptr || !valid_ld(rows, cols, ld) || !is_aligned(codes, 16)) return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
  BufferSet set;
  set.read(x, span_bytes(rows, cols, ld, e), e);
  set.read(weight, cols * we, we);
  set.read(bias, cols * we, we);
  set.write(y, rows * cols * e, e);
  set.write(mean, rows * 4, 4);
  set.write(rstd, rows * 4, 4);
  set.write(codes, rows * ckpt_pitch(cols), 16);
  set.write(scales, rows * ckpt_scales(cols) * 4, 4);
  if (adasum_status_t st = set.check()) return st;
  const NormArgs a = {x, rows, cols, ld, weight, bias, static_cast<int>(weight_dtype), eps, y, mean, rstd, codes, scales};
  const bool vec = is_aligned(x, 16) && is_aligned(y, 16) && ld * e % 16 == 0 && cols * e % 16 == 0;
  const double n = static_cast<double>(rows) * cols;
  return counted_launch(stream, codes ? "norm_checkpoint" : "norm", n * (2 * e + (codes ? 1 : 0)), [&] {
    if (dtype == ADASUM_BF16) return vec ? launch_norm<bf16, kVec8>(a, stream) : launch_norm<bf16, kStrided>(a, stream);
    return vec ? launch_norm<float, kVec4>(a, stream) : launch_norm<float, kStrided>(a, stream);
  });
}

int64_t adasum_layer_norm_backward_scratch_bytes(const int64_t* worker_offsets, int K, int64_t cols) {
  if (check_worker_offsets(worker_offsets, K) || cols <= 0 || cols > ADASUM_NORM_MAX_COLS) return 0;
  const int64_t rows = worker_offsets[K];
  if (rows == 0 || one_launch(worker_offsets, K, cols)) return 0;
  // one partial per CTA: the persistent grid, or one CTA for every worker
  const int64_t ctas = std::min<int64_t>(rows, kNormCtasPerSm * sm_count() + static_cast<int64_t>(K));
  return (ctas * 2 * cols * 4 + 255) / 256 * 256;
}

adasum_status_t adasum_layer_norm_backward(const void* grad_out, int64_t ld_grad, const void* x, int64_t ld_x,
                                           const float* mean, const float* rstd, int64_t cols, adasum_dtype_t dtype,
                                           const void* weight, adasum_dtype_t weight_dtype,
                                           const int64_t* worker_offsets, int K, void* grad_x,
                                           void* const* grad_weights, void* const* grad_biases,
                                           adasum_dtype_t grad_dtype, int accumulate, void* scratch,
                                           int64_t scratch_bytes, adasum_stream_t stream) {
  EntryScope scope("adasum_layer_norm_backward");
  NormGradArgs a = {};
  a.dy = grad_out;
  a.ld_dy = ld_grad;
  a.x = x;
  a.ld_x = ld_x;
  a.mean = mean;
  a.rstd = rstd;
  a.cols = cols;
  a.weight = weight;
  a.weight_dtype = static_cast<int>(weight_dtype);
  a.dx = grad_x;
  return norm_backward(a, dtype, worker_offsets, K, grad_weights, grad_biases, grad_dtype, accumulate, scratch,
                       scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

adasum_status_t adasum_layer_norm_backward_checkpointed(
    const void* grad_out, int64_t ld_grad, const int8_t* codes, const float* scales, const float* rstd, int64_t cols,
    adasum_dtype_t dtype, const void* weight, const void* bias, adasum_dtype_t weight_dtype,
    const int64_t* worker_offsets, int K, void* grad_x, void* y, void* const* grad_weights, void* const* grad_biases,
    adasum_dtype_t grad_dtype, int accumulate, void* scratch, int64_t scratch_bytes, adasum_stream_t stream) {
  EntryScope scope("adasum_layer_norm_backward_checkpointed");
  if (codes == nullptr && (worker_offsets == nullptr || K < 1 || K > kMaxK || worker_offsets[K] > 0))
    return ADASUM_ERR_INVALID_ARG;
  NormGradArgs a = {};
  a.dy = grad_out;
  a.ld_dy = ld_grad;
  a.codes = codes;
  a.scales = scales;
  a.rstd = rstd;
  a.cols = cols;
  a.weight = weight;
  a.bias = bias;
  a.weight_dtype = static_cast<int>(weight_dtype);
  a.dx = grad_x;
  a.y = y;
  return norm_backward(a, dtype, worker_offsets, K, grad_weights, grad_biases, grad_dtype, accumulate, scratch,
                       scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
