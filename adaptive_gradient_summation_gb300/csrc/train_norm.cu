// train_norm.cu -- layer norm, its gradient with the per-worker reduction of the
// parameters' gradients, and both with the normalised activation kept in 8 bits.
#include "adasum_host.h"
#include "adasum_launch.h"
#include "adasum_train.cuh"

namespace adasum {
namespace {

constexpr int kNormThreads = 256;

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
};

struct ParamGradArgs {
  void* dw[kMaxK];
  void* db[kMaxK];
  int64_t off[kMaxK + 1];
  int K;
  int dtype, accumulate, want_w, want_b;
};

__device__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < kNormThreads / 32; ++i) s += red[i];
  return s;
}

// One CTA per row; the row is read three times (the second and third from cache).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ float red[kNormThreads / 32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  T* y = static_cast<T*>(a.y) + row * a.cols;
  float s = 0.f;
  for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) s += widen(x[c]);
  const float mean = block_sum(s, red) / static_cast<float>(a.cols);
  float v = 0.f;
  for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
    const float d = widen(x[c]) - mean;
    v = __fmaf_rn(d, d, v);
  }
  const float rstd = 1.f / sqrtf(block_sum(v, red) / static_cast<float>(a.cols) + a.eps);
  for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
    const float h = (widen(x[c]) - mean) * rstd;
    const float w = a.weight ? load_any(a.weight, a.weight_dtype, c) : 1.f;
    const float b = a.bias ? load_any(a.bias, a.weight_dtype, c) : 0.f;
    y[c] = narrow<T>(__fmaf_rn(h, w, b));
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  if (a.codes == nullptr) return;
  const int lane = threadIdx.x & 31;
  for (int64_t blk = threadIdx.x >> 5; blk < ckpt_scales(a.cols); blk += kNormThreads / 32) {
    float h[4], top = 0.f;
    bool bad = false;
    for (int e = 0; e < 4; ++e) {
      const int64_t c = blk * kCkptBlock + e * 32 + lane;
      h[e] = c < a.cols ? (widen(x[c]) - mean) * rstd : 0.f;
      bad |= !isfinite(h[e]);
      top = fmaxf(top, fabsf(h[e]));
    }
    const CkptScale sc = ckpt_scale(warp_max(top), __any_sync(0xFFFFFFFFu, bad));
    for (int e = 0; e < 4; ++e) {
      const int64_t c = blk * kCkptBlock + e * 32 + lane;
      if (c < a.cols) a.codes[row * ckpt_pitch(a.cols) + c] = static_cast<int8_t>(ckpt_code(h[e], sc.inv));
    }
    if (lane == 0) a.scales[row * ckpt_scales(a.cols) + blk] = sc.scale;
  }
}

// h of one element, from x or from the checkpoint.
template <typename T>
__device__ float norm_h(const NormGradArgs& a, int64_t row, int64_t c) {
  if (a.codes != nullptr)
    return ckpt_value(a.codes[row * ckpt_pitch(a.cols) + c], a.scales[row * ckpt_scales(a.cols) + c / kCkptBlock]);
  return (widen(static_cast<const T*>(a.x)[row * a.ld_x + c]) - a.mean[row]) * a.rstd[row];
}

// grad_x: one CTA per row.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_grad_kernel(const NormGradArgs a) {
  pdl_enter();
  __shared__ float red[kNormThreads / 32];
  const int64_t row = blockIdx.x;
  const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
  float sg = 0.f, sgh = 0.f;
  for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
    const float g = widen(dy[c]) * (a.weight ? load_any(a.weight, a.weight_dtype, c) : 1.f);
    sg += g;
    sgh = __fmaf_rn(g, norm_h<T>(a, row, c), sgh);
  }
  const float mg = block_sum(sg, red) / static_cast<float>(a.cols);
  const float mgh = block_sum(sgh, red) / static_cast<float>(a.cols);
  const float rstd = a.rstd[row];
  for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
    const float w = a.weight ? load_any(a.weight, a.weight_dtype, c) : 1.f;
    const float h = norm_h<T>(a, row, c);
    static_cast<T*>(a.dx)[row * a.cols + c] = narrow<T>(rstd * (widen(dy[c]) * w - mg - h * mgh));
    if (a.y != nullptr) {
      const float b = a.bias ? load_any(a.bias, a.weight_dtype, c) : 0.f;
      static_cast<T*>(a.y)[row * a.cols + c] = narrow<T>(__fmaf_rn(h, w, b));
    }
  }
}

// Parameter gradients: 32 columns of one worker per CTA, eight rows at a time.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_params_kernel(const NormGradArgs a,
                                                                  const __grid_constant__ ParamGradArgs p) {
  pdl_enter();
  __shared__ float red[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = blockIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sw = 0.f, sb = 0.f;
  if (c < a.cols)
    for (int64_t row = p.off[k] + warp; row < p.off[k + 1]; row += 8) {
      const float d = widen(static_cast<const T*>(a.dy)[row * a.ld_dy + c]);
      sw = __fmaf_rn(d, norm_h<T>(a, row, c), sw);
      sb += d;
    }
  red[0][warp][lane] = sw;
  red[1][warp][lane] = sb;
  __syncthreads();
  if (warp >= 2 || c >= a.cols || !(warp ? p.want_b : p.want_w)) return;
  float s = 0.f;
  for (int i = 0; i < 8; ++i) s += red[warp][i][lane];
  void* out = warp ? p.db[k] : p.dw[k];
  if (p.accumulate) s += load_any(out, p.dtype, c);
  store_any(out, p.dtype, c, s);
}

template <typename T>
int launch_norm(const NormArgs& a, cudaStream_t stream) {
  return launch_pdl(norm_kernel<T>, dim3(static_cast<unsigned>(a.rows)), dim3(kNormThreads), 0, stream, a);
}
template <typename T>
int launch_norm_grad(const NormGradArgs& a, cudaStream_t stream) {
  return launch_pdl(norm_grad_kernel<T>, dim3(static_cast<unsigned>(a.rows)), dim3(kNormThreads), 0, stream, a);
}
template <typename T>
int launch_norm_params(const NormGradArgs& a, const ParamGradArgs& p, cudaStream_t stream) {
  return launch_pdl(norm_params_kernel<T>, dim3(static_cast<unsigned>((a.cols + 31) / 32), p.K), dim3(kNormThreads), 0,
                    stream, a, p);
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
    p.off[k + 1] = offs[k + 1];
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
  p.K = K;
  p.dtype = grad_dtype;
  p.accumulate = accumulate != 0;
  p.want_w = dw != nullptr;
  p.want_b = db != nullptr;
  const double n = static_cast<double>(a.rows) * a.cols;
  if (a.rows > 0)
    if (adasum_status_t st = counted_launch(stream, kept ? "norm_grad_checkpoint" : "norm_grad",
                                            n * (kept ? 2 * e + 1 : 3 * e), [&] {
          return dtype == kBF16 ? launch_norm_grad<bf16>(a, stream) : launch_norm_grad<float>(a, stream);
        }))
      return st;
  if (!want) return ADASUM_OK;
  return counted_launch(stream, "norm_params", 0.0, [&] {
    return dtype == kBF16 ? launch_norm_params<bf16>(a, p, stream) : launch_norm_params<float>(a, p, stream);
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
  const double n = static_cast<double>(rows) * cols;
  return counted_launch(stream, codes ? "norm_checkpoint" : "norm", n * (2 * e + (codes ? 1 : 0)), [&] {
    return dtype == ADASUM_BF16 ? launch_norm<bf16>(a, stream) : launch_norm<float>(a, stream);
  });
}

int64_t adasum_layer_norm_backward_scratch_bytes(int64_t rows, int64_t cols, int K) {
  (void)rows;
  (void)cols;
  (void)K;
  return 0;
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
