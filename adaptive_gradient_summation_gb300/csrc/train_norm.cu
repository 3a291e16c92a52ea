// train_norm.cu -- entry points of layer norm (kernels: adasum_norm.cuh).
#include "adasum_norm.cuh"

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
  const NormArgs a = {x, rows, cols, ld, nullptr, 0, nullptr, weight, bias, static_cast<int>(weight_dtype), eps, y, mean, rstd, codes, scales};
  const bool vec = is_aligned(x, 16) && is_aligned(y, 16) && ld * e % 16 == 0 && cols * e % 16 == 0;
  const double n = static_cast<double>(rows) * cols;
  return counted_launch(stream, codes ? "norm_checkpoint" : "norm", n * (2 * e + (codes ? 1 : 0)), [&] {
    return launch_norm_of<kLayer>(a, dtype, vec, stream);
  });
}

int64_t adasum_layer_norm_backward_scratch_bytes(const int64_t* worker_offsets, int K, int64_t cols) {
  return norm_scratch_bytes(worker_offsets, K, cols, 2);
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
  return norm_backward<false>(a, dtype, worker_offsets, K, grad_weights, grad_biases, grad_dtype, accumulate, scratch,
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
  return norm_backward<false>(a, dtype, worker_offsets, K, grad_weights, grad_biases, grad_dtype, accumulate, scratch,
                       scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
