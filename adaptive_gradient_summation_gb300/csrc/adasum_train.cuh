// adasum_train.cuh -- device helpers shared by the training operators (train_*.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "adasum_internal.h"
#include "adasum_ptx.cuh"

namespace adasum {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 narrow<bf16>(float x) { return __float2bfloat16_rn(x); }

// Element i of a parameter or gradient whose type is known at run time.
__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  return dtype == kBF16 ? widen(static_cast<const bf16*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float v) {
  if (dtype == kBF16) static_cast<bf16*>(p)[i] = narrow<bf16>(v);
  else static_cast<float*>(p)[i] = v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}

// ------------------------------------------------------------------- 8-bit checkpoints

constexpr int kCkptBlock = 128;
// Blocks below this magnitude are kept as zeros: 127 / m would leave fp32's range.
constexpr float kCkptTiny = 0x1p-119f;

__host__ __device__ constexpr int64_t ckpt_pitch(int64_t cols) { return (cols + 15) / 16 * 16; }
__host__ __device__ constexpr int64_t ckpt_scales(int64_t cols) { return (cols + kCkptBlock - 1) / kCkptBlock; }

// Scale of a block, and what its values are multiplied with before they are rounded.
// `bad`: the block holds a NaN or an infinity.  Both quotients are correctly rounded, so
// the codes of a given block do not depend on who computes them.
struct CkptScale {
  float scale, inv;
};
__device__ __forceinline__ CkptScale ckpt_scale(float top, bool bad) {
  if (bad) return {__int_as_float(0x7FC00000), 0.f};
  if (top < kCkptTiny) return {0.f, 0.f};
  return {__fdiv_rn(top, 127.f), __fdiv_rn(127.f, top)};
}
// round(x * inv), ties to even; |x * inv| <= 127 up to rounding, so adding 1.5 * 2^23
// leaves the integer in the low bits of the sum.  (A NaN or infinity, in a block whose
// scale is NaN, gives an arbitrary code.)
__device__ __forceinline__ uint32_t ckpt_code(float x, float inv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.f)) & 0xFFu;
}
__device__ __forceinline__ float ckpt_value(int8_t q, float scale) { return __fmul_rn(static_cast<float>(q), scale); }

}  // namespace adasum
