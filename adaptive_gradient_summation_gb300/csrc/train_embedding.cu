// train_embedding.cu -- token embeddings and the table's gradient, per worker.
#include "adasum_host.h"
#include "adasum_launch.h"
#include "adasum_train.cuh"

namespace adasum {
namespace {

constexpr int kEmbThreads = 256;

struct LookupArgs {
  const void* table;
  int64_t num_rows, cols;
  const void* tokens;
  int token_bytes;
  int64_t n;
  float scale;
  void* out;
};

struct TableGradArgs {
  const void* dy;
  int64_t cols, ld;
  const void* tokens;
  int token_bytes;
  int64_t num_rows;
  float scale;
  int64_t padding_idx;
  int grad_dtype, accumulate;
  int K;
  void* grads[kMaxK];
  int64_t off[kMaxK + 1];
};

__device__ __forceinline__ int64_t load_token(const void* tokens, int bytes, int64_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

// One CTA per token.
template <typename T>
__global__ void __launch_bounds__(kEmbThreads) lookup_kernel(const LookupArgs a) {
  pdl_enter();
  const int64_t i = blockIdx.x, t = load_token(a.tokens, a.token_bytes, i);
  const bool there = t >= 0 && t < a.num_rows;
  const T* src = static_cast<const T*>(a.table) + t * a.cols;
  T* dst = static_cast<T*>(a.out) + i * a.cols;
  for (int64_t c = threadIdx.x; c < a.cols; c += kEmbThreads)
    dst[c] = narrow<T>(there ? a.scale * widen(src[c]) : 0.f);
}

// One warp per (worker, table row): it looks through the worker's tokens for the row's.
template <typename T>
__global__ void __launch_bounds__(kEmbThreads) table_grad_kernel(const __grid_constant__ TableGradArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31, k = blockIdx.y;
  const int64_t v = static_cast<int64_t>(blockIdx.x) * (kEmbThreads / 32) + (threadIdx.x >> 5);
  if (v >= a.num_rows) return;
  const int64_t lo = a.off[k], hi = a.off[k + 1];
  for (int64_t c0 = 0; c0 < a.cols; c0 += 32 * 32) {
    float s[32];
    for (int j = 0; j < 32; ++j) s[j] = 0.f;
    bool any = false;
    if (v != a.padding_idx)
      for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        unsigned m = __ballot_sync(0xFFFFFFFFu, i0 + lane < hi && load_token(a.tokens, a.token_bytes, i0 + lane) == v);
        any |= m != 0;
        for (; m != 0; m &= m - 1) {
          const T* dy = static_cast<const T*>(a.dy) + (i0 + __ffs(m) - 1) * a.ld;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int64_t c = c0 + j * 32 + lane;
            if (c < a.cols) s[j] += widen(dy[c]);
          }
        }
      }
    if (!any && a.accumulate) continue;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int64_t c = c0 + j * 32 + lane;
      if (c >= a.cols) continue;
      float g = a.scale * s[j];
      if (a.accumulate) g += load_any(a.grads[k], a.grad_dtype, v * a.cols + c);
      store_any(a.grads[k], a.grad_dtype, v * a.cols + c, g);
    }
  }
}

}  // namespace
}  // namespace adasum

using namespace adasum;

extern "C" {

adasum_status_t adasum_embedding(const void* table, int64_t num_rows, int64_t cols, adasum_dtype_t dtype,
                                 const void* tokens, int token_bytes, int64_t n, float scale, void* out,
                                 adasum_stream_t stream_) {
  EntryScope scope("adasum_embedding");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!valid_dtype(dtype) || num_rows < 0 || cols < 1 || n < 0 || (token_bytes != 4 && token_bytes != 8))
    return ADASUM_ERR_INVALID_ARG;
  if (cols > INT32_MAX || n > INT32_MAX || num_rows > INT32_MAX) return ADASUM_ERR_UNSUPPORTED;
  if (n == 0) return ADASUM_OK;
  if ((table == nullptr && num_rows > 0) || tokens == nullptr || out == nullptr) return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype);
  BufferSet set;
  set.read(table, num_rows * cols * e);
  set.read(tokens, n * token_bytes);
  set.write(out, n * cols * e);
  if (set.conflict()) return ADASUM_ERR_ALIAS;
  const LookupArgs a = {table, num_rows, cols, tokens, token_bytes, n, scale, out};
  return counted_launch(stream, "embedding", static_cast<double>(n) * (2 * cols * e + token_bytes), [&] {
    return launch_pdl(dtype == ADASUM_BF16 ? lookup_kernel<bf16> : lookup_kernel<float>, dim3(static_cast<unsigned>(n)),
                      dim3(kEmbThreads), 0, stream, a);
  });
}

int64_t adasum_embedding_backward_scratch_bytes(int64_t n, int64_t cols, int K) {
  (void)n;
  (void)cols;
  (void)K;
  return 0;
}

adasum_status_t adasum_embedding_backward(const void* grad_out, int64_t cols, int64_t ld, adasum_dtype_t dtype,
                                          const void* tokens, int token_bytes, const int64_t* worker_offsets, int K,
                                          int64_t num_rows, float scale, int64_t padding_idx, void* const* grads,
                                          adasum_dtype_t grad_dtype, int accumulate, void* scratch,
                                          int64_t scratch_bytes, adasum_stream_t stream_) {
  EntryScope scope("adasum_embedding_backward");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!valid_dtype(dtype) || !valid_dtype(grad_dtype) || num_rows < 0 || cols < 1 ||
      (token_bytes != 4 && token_bytes != 8))
    return ADASUM_ERR_INVALID_ARG;
  if (adasum_status_t st = check_worker_offsets(worker_offsets, K)) return st;
  const int64_t n = worker_offsets[K];
  if (cols > INT32_MAX || n > INT32_MAX || num_rows > INT32_MAX) return ADASUM_ERR_UNSUPPORTED;
  if (num_rows == 0) return ADASUM_OK;
  if (grads == nullptr || (n > 0 && (grad_out == nullptr || tokens == nullptr || ld < cols)))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t need = adasum_embedding_backward_scratch_bytes(n, cols, K);
  if (need > 0 && (scratch == nullptr || scratch_bytes < need || !is_aligned(scratch, 256)))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype), ge = dtype_bytes(grad_dtype);
  TableGradArgs a = {};
  BufferSet set;
  set.read(grad_out, span_bytes(n, cols, ld, e));
  set.read(tokens, n * token_bytes);
  set.write(scratch, need);
  for (int k = 0; k < K; ++k) {
    if (grads[k] == nullptr) return ADASUM_ERR_INVALID_ARG;
    a.grads[k] = grads[k];
    a.off[k + 1] = worker_offsets[k + 1];
    set.write(grads[k], num_rows * cols * ge);
  }
  if (set.conflict()) return ADASUM_ERR_ALIAS;
  a.dy = grad_out;
  a.cols = cols;
  a.ld = ld;
  a.tokens = tokens;
  a.token_bytes = token_bytes;
  a.num_rows = num_rows;
  a.scale = scale;
  a.padding_idx = padding_idx;
  a.grad_dtype = static_cast<int>(grad_dtype);
  a.accumulate = accumulate != 0;
  a.K = K;
  const double bytes = static_cast<double>(n) * (cols * e + token_bytes) +
                       (accumulate ? 0.0 : static_cast<double>(K) * num_rows * cols * ge);
  return counted_launch(stream, "embedding_grad", bytes, [&] {
    const dim3 grid(static_cast<unsigned>((num_rows + kEmbThreads / 32 - 1) / (kEmbThreads / 32)), K);
    return launch_pdl(dtype == ADASUM_BF16 ? table_grad_kernel<bf16> : table_grad_kernel<float>, grid,
                      dim3(kEmbThreads), 0, stream, a);
  });
}

}  // extern "C"
