// train_rms.cu -- entry points of the root-mean-square norm, and its forward kernels
// (adasum_norm.cuh).
#include "adasum_norm.cuh"

using namespace adasum;

extern "C" {

adasum_status_t adasum_rms_norm(const void* x, int64_t rows, int64_t cols, int64_t ld, adasum_dtype_t dtype,
                                const void* residual, int64_t ld_residual, void* total, const void* weight,
                                adasum_dtype_t weight_dtype, float eps, void* y, float* rstd, int8_t* codes, float* scales,
                                adasum_stream_t stream_) {
  EntryScope scope("adasum_rms_norm");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (adasum_status_t st = check_norm(rows, cols, dtype, weight_dtype)) return st;
  if ((codes == nullptr) != (scales == nullptr) || !(eps >= 0.f)) return ADASUM_ERR_INVALID_ARG;
  if (rows == 0) return ADASUM_OK;
  if ((residual == nullptr) != (total == nullptr)) return ADASUM_ERR_INVALID_ARG;
  if (x == nullptr || y == nullptr || !valid_ld(rows, cols, ld) || !is_aligned(codes, 16) ||
      (residual != nullptr && !valid_ld(rows, cols, ld_residual)))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
  BufferSet set;
  set.read(x, span_bytes(rows, cols, ld, e), e);
  if (residual != nullptr) set.read(residual, span_bytes(rows, cols, ld_residual, e), e);
  set.read(weight, cols * we, we);
  set.write(total, rows * cols * e, e);
  set.write(y, rows * cols * e, e);
  set.write(rstd, rows * 4, 4);
  set.write(codes, rows * ckpt_pitch(cols), 16);
  set.write(scales, rows * ckpt_scales(cols) * 4, 4);
  if (adasum_status_t st = set.check()) return st;
  const NormArgs a = {x, rows, cols, ld, residual, ld_residual, total, weight, nullptr, static_cast<int>(weight_dtype), eps, y,
                      nullptr, rstd, codes, scales};
  const bool vec = is_aligned(x, 16) && is_aligned(y, 16) && ld * e % 16 == 0 && cols * e % 16 == 0 &&
                   (residual == nullptr || (is_aligned(residual, 16) && ld_residual * e % 16 == 0 && is_aligned(total, 16)));
  const double n = static_cast<double>(rows) * cols;
  return counted_launch(stream, codes ? "rms_checkpoint" : "rms", n * ((residual ? 4 : 2) * e + (codes ? 1 : 0)), [&] {
    return residual ? launch_norm_of<kRmsSum>(a, dtype, vec, stream) : launch_norm_of<kRms>(a, dtype, vec, stream);
  });
}

int64_t adasum_rms_norm_backward_scratch_bytes(const int64_t* worker_offsets, int K, int64_t cols) {
  return norm_scratch_bytes(worker_offsets, K, cols, 1);
}

adasum_status_t adasum_rms_norm_backward(const void* grad_out, int64_t ld_grad, const void* x, int64_t ld_x, const float* rstd,
                                         int64_t cols, adasum_dtype_t dtype, const void* weight, adasum_dtype_t weight_dtype,
                                         const void* grad_residual, int64_t ld_residual, const int64_t* worker_offsets, int K,
                                         void* grad_x, void* const* grad_weights, adasum_dtype_t grad_dtype, int accumulate,
                                         void* scratch, int64_t scratch_bytes, adasum_stream_t stream) {
  EntryScope scope("adasum_rms_norm_backward");
  NormGradArgs a = {};
  a.dy = grad_out;
  a.ld_dy = ld_grad;
  a.past = grad_residual;
  a.ld_past = ld_residual;
  a.x = x;
  a.ld_x = ld_x;
  a.rstd = rstd;
  a.cols = cols;
  a.weight = weight;
  a.weight_dtype = static_cast<int>(weight_dtype);
  a.dx = grad_x;
  return norm_backward<true>(a, dtype, worker_offsets, K, grad_weights, nullptr, grad_dtype, accumulate, scratch, scratch_bytes,
                             reinterpret_cast<cudaStream_t>(stream));
}

adasum_status_t adasum_rms_norm_backward_checkpointed(const void* grad_out, int64_t ld_grad, const int8_t* codes,
                                                      const float* scales, const float* rstd, int64_t cols, adasum_dtype_t dtype,
                                                      const void* weight, adasum_dtype_t weight_dtype, const void* grad_residual,
                                                      int64_t ld_residual, const int64_t* worker_offsets, int K, void* grad_x,
                                                      void* y, void* const* grad_weights, adasum_dtype_t grad_dtype,
                                                      int accumulate, void* scratch, int64_t scratch_bytes,
                                                      adasum_stream_t stream) {
  EntryScope scope("adasum_rms_norm_backward_checkpointed");
  if (codes == nullptr && (worker_offsets == nullptr || K < 1 || K > kMaxK || worker_offsets[K] > 0))
    return ADASUM_ERR_INVALID_ARG;
  NormGradArgs a = {};
  a.dy = grad_out;
  a.ld_dy = ld_grad;
  a.past = grad_residual;
  a.ld_past = ld_residual;
  a.codes = codes;
  a.scales = scales;
  a.rstd = rstd;
  a.cols = cols;
  a.weight = weight;
  a.weight_dtype = static_cast<int>(weight_dtype);
  a.dx = grad_x;
  a.y = y;
  return norm_backward<true>(a, dtype, worker_offsets, K, grad_weights, nullptr, grad_dtype, accumulate, scratch, scratch_bytes,
                             reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
