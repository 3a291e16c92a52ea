// train_checkpoint.cu -- activations kept in 8 bits: pack, unpack, and the GELU whose
// forward pass packs its input and whose backward pass starts from the codes.
#include "adasum_host.h"
#include "adasum_launch.h"
#include "adasum_train.cuh"

namespace adasum {
namespace {

constexpr int kCkptThreads = 256;

enum Act : int { kActNone = 0, kActErf = 1, kActTanh = 2 };

// gelu(x) and its slope.
template <int ACT>
__device__ float gelu_value(float x) {
  if constexpr (ACT == kActTanh) {
    const float u = 0.7978845608f * (x + 0.044715f * x * x * x);
    return 0.5f * x * (1.f + tanhf(u));
  }
  return 0.5f * x * (1.f + erff(x * 0.70710678f));
}
template <int ACT>
__device__ float gelu_slope(float x) {
  if constexpr (ACT == kActTanh) {
    const float t = tanhf(0.7978845608f * (x + 0.044715f * x * x * x));
    return 0.5f * (1.f + t) + 0.5f * x * (1.f - t * t) * 0.7978845608f * (1.f + 0.134145f * x * x);
  }
  return 0.5f * (1.f + erff(x * 0.70710678f)) + x * 0.3989422804f * expf(-0.5f * x * x);
}

struct PackArgs {
  const void* x;
  int64_t rows, cols, ld;
  int8_t* codes;
  float* scales;
  void* y;  // the activation's output (kActNone: null)
};
struct UnpackArgs {
  const int8_t* codes;
  const float* scales;
  int64_t rows, cols;
  const void* dy;  // kActNone: null
  int64_t ld_dy;
  void* out;       // the values (kActNone) or grad_x
  void* y;         // the activation again; null: not wanted
};

// One warp per block of 128 columns.
template <typename T, int ACT>
__global__ void __launch_bounds__(kCkptThreads) pack_kernel(const PackArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t nb = ckpt_scales(a.cols);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kCkptThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kCkptThreads / 32) + (threadIdx.x >> 5); i < a.rows * nb; i += step) {
    const int64_t row = i / nb, c0 = (i - row * nb) * kCkptBlock;
    const T* x = static_cast<const T*>(a.x) + row * a.ld;
    float v[4], top = 0.f;
    bool bad = false;
    for (int e = 0; e < 4; ++e) {
      const int64_t c = c0 + e * 32 + lane;
      v[e] = c < a.cols ? widen(x[c]) : 0.f;
      bad |= !isfinite(v[e]);
      top = fmaxf(top, fabsf(v[e]));
    }
    const CkptScale sc = ckpt_scale(warp_max(top), __any_sync(0xFFFFFFFFu, bad));
    for (int e = 0; e < 4; ++e) {
      const int64_t c = c0 + e * 32 + lane;
      if (c >= a.cols) continue;
      a.codes[row * ckpt_pitch(a.cols) + c] = static_cast<int8_t>(ckpt_code(v[e], sc.inv));
      if constexpr (ACT != kActNone) static_cast<T*>(a.y)[row * a.cols + c] = narrow<T>(gelu_value<ACT>(v[e]));
    }
    if (lane == 0) a.scales[i] = sc.scale;
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kCkptThreads) unpack_kernel(const UnpackArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t nb = ckpt_scales(a.cols);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kCkptThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kCkptThreads / 32) + (threadIdx.x >> 5); i < a.rows * nb; i += step) {
    const int64_t row = i / nb, c0 = (i - row * nb) * kCkptBlock;
    const float scale = a.scales[i];
    for (int e = 0; e < 4; ++e) {
      const int64_t c = c0 + e * 32 + lane;
      if (c >= a.cols) continue;
      const float v = ckpt_value(a.codes[row * ckpt_pitch(a.cols) + c], scale);
      T* out = static_cast<T*>(a.out) + row * a.cols + c;
      if constexpr (ACT == kActNone) {
        *out = narrow<T>(v);
      } else {
        *out = narrow<T>(widen(static_cast<const T*>(a.dy)[row * a.ld_dy + c]) * gelu_slope<ACT>(v));
        if (a.y != nullptr) static_cast<T*>(a.y)[row * a.cols + c] = narrow<T>(gelu_value<ACT>(v));
      }
    }
  }
}

unsigned ckpt_grid(int64_t rows, int64_t cols) {
  const int64_t need = (rows * ckpt_scales(cols) + kCkptThreads / 32 - 1) / (kCkptThreads / 32);
  return static_cast<unsigned>(std::min<int64_t>(need, 8 * static_cast<int64_t>(sm_count())));
}

template <typename T>
int launch_pack(const PackArgs& a, int act, cudaStream_t stream) {
  auto k = act == kActNone ? pack_kernel<T, kActNone> : act == kActErf ? pack_kernel<T, kActErf> : pack_kernel<T, kActTanh>;
  return launch_pdl(k, dim3(ckpt_grid(a.rows, a.cols)), dim3(kCkptThreads), 0, stream, a);
}
template <typename T>
int launch_unpack(const UnpackArgs& a, int act, cudaStream_t stream) {
  auto k = act == kActNone ? unpack_kernel<T, kActNone> : act == kActErf ? unpack_kernel<T, kActErf> : unpack_kernel<T, kActTanh>;
  return launch_pdl(k, dim3(ckpt_grid(a.rows, a.cols)), dim3(kCkptThreads), 0, stream, a);
}

adasum_status_t check_shape(int64_t rows, int64_t cols, int dtype) {
  if (rows < 0 || cols < 1 || !valid_dtype(dtype)) return ADASUM_ERR_INVALID_ARG;
  if (cols > INT32_MAX || rows > INT64_MAX / (8 * cols)) return ADASUM_ERR_UNSUPPORTED;
  return ADASUM_OK;
}

adasum_status_t pack(const PackArgs& a, int dtype, int act, cudaStream_t stream) {
  if (adasum_status_t st = check_shape(a.rows, a.cols, dtype)) return st;
  if (a.rows == 0) return ADASUM_OK;
  if (a.x == nullptr || a.codes == nullptr || a.scales == nullptr || (act != kActNone && a.y == nullptr) ||
      a.ld < a.cols || !is_aligned(a.codes, 16))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype);
  BufferSet set;
  set.read(a.x, span_bytes(a.rows, a.cols, a.ld, e));
  set.write(a.codes, a.rows * ckpt_pitch(a.cols));
  set.write(a.scales, a.rows * ckpt_scales(a.cols) * 4);
  set.write(a.y, a.rows * a.cols * e);
  if (set.conflict()) return ADASUM_ERR_ALIAS;
  const double n = static_cast<double>(a.rows) * a.cols;
  return counted_launch(stream, act ? "gelu_checkpoint" : "checkpoint_pack", n * (e + 1 + (act ? e : 0)), [&] {
    return dtype == kBF16 ? launch_pack<bf16>(a, act, stream) : launch_pack<float>(a, act, stream);
  });
}

adasum_status_t unpack(const UnpackArgs& a, int dtype, int act, cudaStream_t stream) {
  if (adasum_status_t st = check_shape(a.rows, a.cols, dtype)) return st;
  if (a.rows == 0) return ADASUM_OK;
  if (a.codes == nullptr || a.scales == nullptr || a.out == nullptr || !is_aligned(a.codes, 16) ||
      (act != kActNone && (a.dy == nullptr || a.ld_dy < a.cols)))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype);
  BufferSet set;
  set.read(a.codes, a.rows * ckpt_pitch(a.cols));
  set.read(a.scales, a.rows * ckpt_scales(a.cols) * 4);
  if (act != kActNone) set.read(a.dy, span_bytes(a.rows, a.cols, a.ld_dy, e));
  set.write(a.out, a.rows * a.cols * e);
  set.write(a.y, a.rows * a.cols * e);
  if (set.conflict()) return ADASUM_ERR_ALIAS;
  const double n = static_cast<double>(a.rows) * a.cols;
  return counted_launch(stream, act ? "gelu_grad_checkpoint" : "checkpoint_unpack",
                        n * (1 + e + (act ? e : 0) + (a.y ? e : 0)), [&] {
    return dtype == kBF16 ? launch_unpack<bf16>(a, act, stream) : launch_unpack<float>(a, act, stream);
  });
}

}  // namespace
}  // namespace adasum

using namespace adasum;

extern "C" {

adasum_status_t adasum_checkpoint_pack(const void* x, int64_t rows, int64_t cols, int64_t ld, adasum_dtype_t dtype,
                                       int8_t* codes, float* scales, adasum_stream_t stream) {
  EntryScope scope("adasum_checkpoint_pack");
  return pack(PackArgs{x, rows, cols, ld, codes, scales, nullptr}, dtype, kActNone,
              reinterpret_cast<cudaStream_t>(stream));
}

adasum_status_t adasum_checkpoint_unpack(const int8_t* codes, const float* scales, int64_t rows, int64_t cols,
                                         adasum_dtype_t dtype, void* out, adasum_stream_t stream) {
  EntryScope scope("adasum_checkpoint_unpack");
  return unpack(UnpackArgs{codes, scales, rows, cols, nullptr, 0, out, nullptr}, dtype, kActNone,
                reinterpret_cast<cudaStream_t>(stream));
}

adasum_status_t adasum_gelu_checkpointed(const void* x, int64_t rows, int64_t cols, int64_t ld, adasum_dtype_t dtype,
                                         int tanh_form, void* y, int8_t* codes, float* scales,
                                         adasum_stream_t stream) {
  EntryScope scope("adasum_gelu_checkpointed");
  return pack(PackArgs{x, rows, cols, ld, codes, scales, y}, dtype, tanh_form ? kActTanh : kActErf,
              reinterpret_cast<cudaStream_t>(stream));
}

adasum_status_t adasum_gelu_checkpointed_backward(const void* grad_out, int64_t ld_grad, const int8_t* codes,
                                                  const float* scales, int64_t rows, int64_t cols,
                                                  adasum_dtype_t dtype, int tanh_form, void* grad_x, void* y,
                                                  adasum_stream_t stream) {
  EntryScope scope("adasum_gelu_checkpointed_backward");
  return unpack(UnpackArgs{codes, scales, rows, cols, grad_out, ld_grad, grad_x, y}, dtype,
                tanh_form ? kActTanh : kActErf, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
