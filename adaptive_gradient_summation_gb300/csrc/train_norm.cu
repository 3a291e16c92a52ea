// train_norm.cu -- layer norm, its gradient with the per-worker reduction of the
// parameters' gradients, and both with the normalised activation kept in 8 bits.
#include "adasum_host.h"
#include "adasum_launch.h"
#include "adasum_train.cuh"

namespace adasum {
namespace {

constexpr int kSlice = 256;        // columns of a warp's eight per lane
#ifndef NV_F
#define NV_F 4
#endif
#ifndef CTA_F
#define CTA_F 4
#endif
#ifndef OCC_F
#define OCC_F 1
#endif
constexpr int kNormCtasPerSm = 2;  // of the persistent grids

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
  float* partials;     // [CTA][weight, bias][cols]; null: parameters' gradients not wanted
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

// The weight and bias of a CTA's columns as floats in shared memory, 1 and 0 where absent.
template <int COLS, int THREADS>
__device__ __forceinline__ void stage_params(float* w, float* b, const void* weight, const void* bias, int dtype,
                                             int64_t cols) {
  for (int c = threadIdx.x; c < COLS; c += THREADS) {
    if (w) w[c] = c < cols && weight ? load_any(weight, dtype, c) : 1.f;
    if (b) b[c] = c < cols && bias ? load_any(bias, dtype, c) : 0.f;
  }
}

// Layer norm.  Mean and variance of a row from registers, the variance about the mean; with
// several warps a row, each has the mean and the sum of squares about it of its own columns
// and one exchange joins them: with n_w columns, mean m_w and sum of squares S_w,
//     mean = sum n_w m_w / n,   S = sum S_w + n_w (m_w - mean)^2.
// Bound by the bytes of x and y; the next row is on its way while one is worked on.
template <typename T, int LAYOUT, int W, int NV, bool KEEP>
__global__ void __launch_bounds__(Team<W, NV>::kThreads, W < 16 ? OCC_F : 1) norm_kernel(const NormArgs a) {
  using TM = Team<W, NV>;
  pdl_enter();
  extern __shared__ __align__(16) float sm[];
  float *ws = sm, *bs = sm + TM::kCols;
  __shared__ float2 ex[2][TM::kTeams][W];
  stage_params<TM::kCols, TM::kThreads>(ws, bs, a.weight, a.bias, a.weight_dtype, a.cols);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / W, w = warp % W;
  const float inv_n = 1.f / static_cast<float>(a.cols);
  const int64_t step = static_cast<int64_t>(gridDim.x) * TM::kTeams;
  const int64_t pitch = ckpt_pitch(a.cols), nscales = ckpt_scales(a.cols);
  auto left_of = [&](int j) { return a.cols - (j * W + w) * kSlice; };
  Raw8<T> next[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      next[j] = load8<T, LAYOUT>(static_cast<const T*>(a.x) + row * a.ld + (j * W + w) * kSlice,
                                 row < a.rows ? left_of(j) : 0, lane);
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * TM::kTeams + team;
  fetch(row);
  for (int it = 0; row < a.rows; row += step, it ^= 1) {
    Raw8<T> r[NV];
    float sum = 0.f, count = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      r[j] = next[j];
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += raw_value<T>(r[j], e);
      count += static_cast<float>(max(static_cast<int64_t>(0), min(left_of(j), static_cast<int64_t>(kSlice))));
    }
    fetch(row + step);
    sum = warp_sum(sum);
    float mean = W == 1 ? sum * inv_n : (count > 0.f ? sum / count : 0.f);
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t left = left_of(j);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = raw_value<T>(r[j], e) - mean;
        if (left >= kSlice || lane_col<LAYOUT>(lane, e) < left) sq = __fmaf_rn(d, d, sq);
      }
    }
    sq = warp_sum(sq);
    if constexpr (W > 1) {
      if (lane == 0) ex[it][team][w] = make_float2(mean, sq);
      TM::sync(team);
      float total = 0.f;
      auto columns = [&](int i) {  // of warp i
        float n = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
          n += static_cast<float>(max(static_cast<int64_t>(0), min(a.cols - (j * W + i) * kSlice, static_cast<int64_t>(kSlice))));
        return n;
      };
      float2 v[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[i] = ex[it][team][i];
        total = __fmaf_rn(columns(i), v[i].x, total);
      }
      mean = total * inv_n;
      sq = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float d = v[i].x - mean;
        sq += __fmaf_rn(columns(i) * d, d, v[i].y);
      }
    }
    const float rstd = 1.f / sqrtf(__fmaf_rn(sq, inv_n, a.eps));
    if (w == 0 && lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    auto row_h = [&](int j, float (&h)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (raw_value<T>(r[j], e) - mean) * rstd;
      if (KEEP && left_of(j) < kSlice) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (lane_col<LAYOUT>(lane, e) >= left_of(j)) h[e] = 0.f;
      }
    };
    CkptScale sc[KEEP ? NV : 1][2];
    if constexpr (KEEP) {
      float top[NV][2];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float h[8];
        row_h(j, h);
        block_tops<LAYOUT>(h, top[j]);
      }
      block_scales<LAYOUT, NV>(top, lane, sc);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * W + w) * kSlice;
      const int64_t left = left_of(j);
      if (left <= 0) break;
      float h[8], wv[8], bv[8];
row_h(j, h);
      if constexpr (KEEP) {
        store_codes8<LAYOUT>(a.codes + row * pitch + c0, left, lane, ckpt_codes<LAYOUT>(h, sc[j]));
        store_scales<LAYOUT>(a.scales + row * nscales + c0 / kCkptBlock, left, lane, sc[j]);
      }
      lds8<LAYOUT>(ws + c0, lane, wv);
      lds8<LAYOUT>(bs + c0, lane, bv);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = __fmaf_rn(h[e], wv[e], bv[e]);
      store8<T, LAYOUT>(static_cast<T*>(a.y) + row * a.cols + c0, left, lane, h);
    }
  }
}

// The gradient.  With g = dy w and h the normalised row,
//     dx = rstd (g - mean(g) - h mean(g h)),   dw += dy h,   db += dy:
// one read of dy and x (or of h's codes), two sums per row, and the parameters' sums of a
// CTA's rows in registers, joined over its teams at the end and written as the CTA's partial.
// A CTA's rows all belong to one worker.  Bound by the bytes of dy, x and dx.
template <typename T, int LAYOUT, int W, int NV, bool KEPT>
__global__ void __launch_bounds__(Team<W, NV>::kThreads, W < 16 ? 2 : 1) norm_grad_kernel(const NormGradArgs a,
                                                                         const __grid_constant__ WorkerRows rows) {
  using TM = Team<W, NV>;
  pdl_enter();
  extern __shared__ __align__(16) float sm[];  // weight, bias; at the end the teams' sums
  float *ws = sm, *bs = sm + TM::kCols;
  __shared__ float2 ex[2][TM::kTeams][W];
  stage_params<TM::kCols, TM::kThreads>(ws, KEPT ? bs : nullptr, a.weight, a.bias, a.weight_dtype, a.cols);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / W, w = warp % W;
  const float inv_n = 1.f / static_cast<float>(a.cols);
  const int64_t pitch = ckpt_pitch(a.cols), nscales = ckpt_scales(a.cols);
  int k = 0;
  for (int hi = rows.K; hi - k > 1;) {
    const int m = (k + hi) >> 1;
    if (rows.cta_off[m] <= static_cast<int>(blockIdx.x)) k = m;
    else hi = m;
  }
  const int64_t r0 = rows.off[k] + static_cast<int64_t>(blockIdx.x - rows.cta_off[k]) * rows.rows_per_cta;
  const int64_t r1 = min(r0 + rows.rows_per_cta, rows.off[k + 1]);
  auto left_of = [&](int j) { return a.cols - (j * W + w) * kSlice; };
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = db[j][e] = 0.f;
  struct Row {
    Raw8<T> dy[NV], x[KEPT ? 1 : NV];
    uint2 q[KEPT ? NV : 1];
    float scale[KEPT ? NV : 1][2];
    float mean, rstd;
  } next;
  auto fetch = [&](int64_t row) {
    const bool in = row < r1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * W + w) * kSlice;
      const int64_t left = in ? left_of(j) : 0;
      next.dy[j] = load8<T, LAYOUT>(static_cast<const T*>(a.dy) + row * a.ld_dy + c0, left, lane);
      if constexpr (KEPT) {
        next.q[j] = load_codes8<LAYOUT>(a.codes + row * pitch + c0, left, lane);
        const float* s = a.scales + row * nscales + c0 / kCkptBlock;
        if constexpr (LAYOUT == kVec) {
          next.scale[j][0] = lane * 8 < left ? s[lane >> 4] : 0.f;
          next.scale[j][1] = next.scale[j][0];
        } else {
          next.scale[j][0] = left > 0 ? s[0] : 0.f;
          next.scale[j][1] = left > kCkptBlock ? s[1] : 0.f;
        }
      } else {
        next.x[j] = load8<T, LAYOUT>(static_cast<const T*>(a.x) + row * a.ld_x + c0, left, lane);
      }
    }
    next.mean = !KEPT && in ? a.mean[row] : 0.f;
    next.rstd = in ? a.rstd[row] : 0.f;
  };
  int64_t row = r0 + team;
  fetch(row);
  for (int it = 0; row < r1; row += TM::kTeams, it ^= 1) {
    const Row cur = next;
    fetch(row + TM::kTeams);
    float sg = 0.f, sgh = 0.f;
    auto row_h = [&](int j, float (&h)[8]) {
      if constexpr (KEPT) {
        ckpt_values8(cur.q[j], cur.scale[j][0], cur.scale[j][1], h);
      } else {
        const int64_t left = left_of(j);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (raw_value<T>(cur.x[j], e) - cur.mean) * cur.rstd;
        if (left < kSlice) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (lane_col<LAYOUT>(lane, e) >= left) h[e] = 0.f;
        }
      }
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float h[8], wv[8];
      row_h(j, h);
      lds8<LAYOUT>(ws + (j * W + w) * kSlice, lane, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = raw_value<T>(cur.dy[j], e), g = d * wv[e];
        sg += g;
        sgh = __fmaf_rn(g, h[e], sgh);
        dw[j][e] = __fmaf_rn(d, h[e], dw[j][e]);
        db[j][e] += d;
      }
    }
    sg = warp_sum(sg);
    sgh = warp_sum(sgh);
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
    const float mg = sg * inv_n * cur.rstd, mgh = sgh * inv_n * cur.rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * W + w) * kSlice;
      const int64_t left = left_of(j);
      if (left <= 0) break;
      float h[8], wv[8], v[8];
      row_h(j, h);
      lds8<LAYOUT>(ws + c0, lane, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = __fmaf_rn(raw_value<T>(cur.dy[j], e) * wv[e], cur.rstd, -mg) - h[e] * mgh;
      store8<T, LAYOUT>(static_cast<T*>(a.dx) + row * a.cols + c0, left, lane, v);
      if (KEPT && a.y != nullptr) {
        float bv[8];
        lds8<LAYOUT>(bs + c0, lane, bv);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fmaf_rn(h[e], wv[e], bv[e]);
        store8<T, LAYOUT>(static_cast<T*>(a.y) + row * a.cols + c0, left, lane, v);
      }
    }
  }
  if (a.partials == nullptr) return;
  float* out = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  if constexpr (TM::kTeams == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * W + w) * kSlice;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + lane_col<LAYOUT>(lane, e);
        if (c >= a.cols) continue;
        out[c] = dw[j][e];
        out[a.cols + c] = db[j][e];
      }
    }
  } else {
    __syncthreads();
    float* mine = sm + team * 2 * TM::kCols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      sts8<LAYOUT>(mine + (j * W + w) * kSlice, lane, dw[j]);
      sts8<LAYOUT>(mine + TM::kCols + (j * W + w) * kSlice, lane, db[j]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * TM::kCols; i += TM::kThreads) {
      const int c = i % TM::kCols;
      if (c >= a.cols) continue;
      float s = 0.f;
#pragma unroll
      for (int t = 0; t < TM::kTeams; ++t) s += sm[t * 2 * TM::kCols + i];
      out[(i / TM::kCols) * a.cols + c] = s;
    }
  }
}

// Joins the CTAs' partials of one worker: 32 columns per CTA, eight partials at a time.
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
  void* out = i < p.cols ? p.dw[k] : p.db[k];
  if (out == nullptr) return;
#pragma unroll
  for (int j = 1; j < 8; ++j) s += red[j][lane];
  const int64_t c = i < p.cols ? i : i - p.cols;
  if (p.accumulate) s += load_any(out, p.dtype, c);
  store_any(out, p.dtype, c, s);
}

// Allows a kernel its shared memory where that is more than the default.
int allow_smem(const void* kernel, size_t bytes) {
  return bytes <= 48 * 1024 ? 0
                            : static_cast<int>(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                    static_cast<int>(bytes)));
}

template <typename T, int LAYOUT, int W, int NV>
int launch_norm_as(const NormArgs& a, cudaStream_t stream) {
  using TM = Team<W, NV>;
  const size_t smem = 2 * TM::kCols * sizeof(float);
  auto kernel = a.codes ? norm_kernel<T, LAYOUT, W, NV, true> : norm_kernel<T, LAYOUT, W, NV, false>;
  if (int rc = allow_smem(reinterpret_cast<const void*>(kernel), smem)) return rc;
  const int64_t need = (a.rows + TM::kTeams - 1) / TM::kTeams;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(need, static_cast<int64_t>(CTA_F) * sm_count()));
  return launch_pdl(kernel, dim3(grid), dim3(TM::kThreads), smem, stream, a);
}
// The smallest team that holds a row: up to four slices a warp, then more warps.
template <typename T, int LAYOUT>
int launch_norm(const NormArgs& a, cudaStream_t stream) {
  const int64_t slices = (a.cols + kSlice - 1) / kSlice;
#if NV_F == 4
  if (slices <= 1) return launch_norm_as<T, LAYOUT, 1, 1>(a, stream);
  if (slices <= 2) return launch_norm_as<T, LAYOUT, 1, 2>(a, stream);
  if (slices <= 4) return launch_norm_as<T, LAYOUT, 1, 4>(a, stream);
  if (slices <= 8) return launch_norm_as<T, LAYOUT, 2, 4>(a, stream);
  if (slices <= 16) return launch_norm_as<T, LAYOUT, 4, 4>(a, stream);
  if (slices <= 32) return launch_norm_as<T, LAYOUT, 8, 4>(a, stream);
  return launch_norm_as<T, LAYOUT, 16, 4>(a, stream);
#elif NV_F == 2
  if (slices <= 1) return launch_norm_as<T, LAYOUT, 1, 1>(a, stream);
  if (slices <= 2) return launch_norm_as<T, LAYOUT, 1, 2>(a, stream);
  if (slices <= 4) return launch_norm_as<T, LAYOUT, 2, 2>(a, stream);
  if (slices <= 8) return launch_norm_as<T, LAYOUT, 4, 2>(a, stream);
  if (slices <= 16) return launch_norm_as<T, LAYOUT, 8, 2>(a, stream);
  if (slices <= 32) return launch_norm_as<T, LAYOUT, 16, 2>(a, stream);
  return launch_norm_as<T, LAYOUT, 16, 4>(a, stream);
#else
  if (slices <= 1) return launch_norm_as<T, LAYOUT, 1, 1>(a, stream);
  if (slices <= 2) return launch_norm_as<T, LAYOUT, 2, 1>(a, stream);
  if (slices <= 4) return launch_norm_as<T, LAYOUT, 4, 1>(a, stream);
  if (slices <= 8) return launch_norm_as<T, LAYOUT, 8, 1>(a, stream);
  if (slices <= 16) return launch_norm_as<T, LAYOUT, 8, 2>(a, stream);
  if (slices <= 32) return launch_norm_as<T, LAYOUT, 16, 2>(a, stream);
  return launch_norm_as<T, LAYOUT, 16, 4>(a, stream);
#endif
}

template <typename T, int LAYOUT, int W, int NV>
int launch_norm_grad_as(const NormGradArgs& a, const WorkerRows& rows, cudaStream_t stream) {
  using TM = Team<W, NV>;
  const size_t smem = (TM::kTeams == 1 ? 1 : TM::kTeams) * 2 * TM::kCols * sizeof(float);
  auto kernel = a.codes ? norm_grad_kernel<T, LAYOUT, W, NV, true> : norm_grad_kernel<T, LAYOUT, W, NV, false>;
  if (int rc = allow_smem(reinterpret_cast<const void*>(kernel), smem)) return rc;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(rows.cta_off[rows.K])), dim3(TM::kThreads), smem, stream, a, rows);
}
// Teams of the gradient kernel: two slices a warp, since each costs 16 registers of sums.
int grad_teams(int64_t cols) {
  const int64_t slices = (cols + kSlice - 1) / kSlice;
  return slices <= 2 ? 8 : slices <= 4 ? 4 : slices <= 8 ? 2 : 1;
}
template <typename T, int LAYOUT>
int launch_norm_grad(const NormGradArgs& a, const WorkerRows& rows, cudaStream_t stream) {
  const int64_t slices = (a.cols + kSlice - 1) / kSlice;
  if (slices <= 1) return launch_norm_grad_as<T, LAYOUT, 1, 1>(a, rows, stream);
  if (slices <= 2) return launch_norm_grad_as<T, LAYOUT, 1, 2>(a, rows, stream);
  if (slices <= 4) return launch_norm_grad_as<T, LAYOUT, 2, 2>(a, rows, stream);
  if (slices <= 8) return launch_norm_grad_as<T, LAYOUT, 4, 2>(a, rows, stream);
  if (slices <= 16) return launch_norm_grad_as<T, LAYOUT, 8, 2>(a, rows, stream);
  if (slices <= 32) return launch_norm_grad_as<T, LAYOUT, 16, 2>(a, rows, stream);
  return launch_norm_grad_as<T, LAYOUT, 16, 4>(a, rows, stream);
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
    if (a.ld_dy < a.cols || (!kept && a.ld_x < a.cols) || (kept && !is_aligned(a.codes, 16)))
      return ADASUM_ERR_INVALID_ARG;
  }
  const int64_t need = adasum_layer_norm_backward_scratch_bytes(a.rows, a.cols, K);
  if (want && need > 0 && (scratch == nullptr || scratch_bytes < need || !is_aligned(scratch, 256)))
    return ADASUM_ERR_INVALID_ARG;
  WorkerRows rows = {};
  ParamGradArgs p = {};
  BufferSet set;
  set.read(a.dy, span_bytes(a.rows, a.cols, a.ld_dy, e));
  if (kept) {
    set.read(a.codes, a.rows * ckpt_pitch(a.cols));
    set.read(a.scales, a.rows * ckpt_scales(a.cols) * 4);
  } else {
    set.read(a.x, span_bytes(a.rows, a.cols, a.ld_x, e));
    set.read(a.mean, a.rows * 4);
  }
  set.read(a.rstd, a.rows * 4);
  set.read(a.weight, a.cols * we);
  set.read(a.bias, a.cols * we);
  set.write(a.dx, a.rows * a.cols * e);
  set.write(a.y, a.rows * a.cols * e);
  if (want) set.write(scratch, need);
  for (int k = 0; k < K; ++k) {
    if (dw != nullptr) {
      if (dw[k] == nullptr) return ADASUM_ERR_INVALID_ARG;
      set.write(p.dw[k] = dw[k], a.cols * ge);
    }
    if (db != nullptr) {
      if (db[k] == nullptr) return ADASUM_ERR_INVALID_ARG;
      set.write(p.db[k] = db[k], a.cols * ge);
    }
  }
  if (set.conflict()) return ADASUM_ERR_ALIAS;
  const double n = static_cast<double>(a.rows) * a.cols;
  deal_rows(rows, offs, K, grad_teams(a.cols), kNormCtasPerSm * sm_count());
  const bool vec = is_aligned(a.dy, 16) && is_aligned(a.dx, 16) && is_aligned(a.y, 16) && a.ld_dy * e % 16 == 0 &&
                   a.cols * e % 16 == 0 && (kept || (is_aligned(a.x, 16) && a.ld_x * e % 16 == 0));
  a.partials = want ? static_cast<float*>(scratch) : nullptr;
  if (a.rows > 0)
    if (adasum_status_t st = counted_launch(stream, kept ? "norm_grad_checkpoint" : "norm_grad",
                                            n * (kept ? 2 * e + 1 + (a.y ? e : 0) : 3 * e), [&] {
          if (dtype == kBF16)
            return vec ? launch_norm_grad<bf16, kVec>(a, rows, stream) : launch_norm_grad<bf16, kStrided>(a, rows, stream);
          return vec ? launch_norm_grad<float, kVec>(a, rows, stream) : launch_norm_grad<float, kStrided>(a, rows, stream);
        }))
      return st;
  if (!want) return ADASUM_OK;
  p.partials = a.partials;
  p.cols = a.cols;
  p.dtype = grad_dtype;
  p.accumulate = accumulate != 0;
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
  if (x == nullptr || y == nullptr || ld < cols || !is_aligned(codes, 16)) return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
  BufferSet set;
  set.read(x, span_bytes(rows, cols, ld, e));
  set.read(weight, cols * we);
  set.read(bias, cols * we);
  set.write(y, rows * cols * e);
  set.write(mean, rows * 4);
  set.write(rstd, rows * 4);
  set.write(codes, rows * ckpt_pitch(cols));
  set.write(scales, rows * ckpt_scales(cols) * 4);
  if (set.conflict()) return ADASUM_ERR_ALIAS;
  const NormArgs a = {x, rows, cols, ld, weight, bias, static_cast<int>(weight_dtype), eps, y, mean, rstd, codes, scales};
  const bool vec = is_aligned(x, 16) && is_aligned(y, 16) && ld * e % 16 == 0 && cols * e % 16 == 0;
  const double n = static_cast<double>(rows) * cols;
  return counted_launch(stream, codes ? "norm_checkpoint" : "norm", n * (2 * e + (codes ? 1 : 0)), [&] {
    if (dtype == ADASUM_BF16) return vec ? launch_norm<bf16, kVec>(a, stream) : launch_norm<bf16, kStrided>(a, stream);
    return vec ? launch_norm<float, kVec>(a, stream) : launch_norm<float, kStrided>(a, stream);
  });
}

int64_t adasum_layer_norm_backward_scratch_bytes(int64_t rows, int64_t cols, int K) {
  if (rows <= 0 || cols <= 0 || K <= 0) return 0;
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
