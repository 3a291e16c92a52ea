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

// ------------------------------------------------------------- eight columns of a lane

// A warp covers 256 columns of a row at a time, eight per lane.  kVec: lane l holds the
// neighbouring columns 8 l .. 8 l + 7, moved as 16-byte vectors; it needs rows that start
// on 16-byte boundaries.  kStrided: lane l holds columns l, l + 32, ..., l + 224, moved one
// by one but coalesced over the lanes; for every other address.
enum Layout : int { kStrided = 0, kVec = 1 };

template <int LAYOUT>
__device__ __forceinline__ int lane_col(int lane, int e) {
  return LAYOUT == kVec ? lane * 8 + e : e * 32 + lane;
}

// Raw bits of a lane's eight values.
template <typename T>
struct Raw8 {
  uint32_t w[sizeof(T) * 2];
};

template <typename T>
__device__ __forceinline__ float raw_value(const Raw8<T>& r, int e) {
  if constexpr (sizeof(T) == 2) return __uint_as_float(e & 1 ? r.w[e >> 1] & 0xFFFF0000u : r.w[e >> 1] << 16);
  else return __uint_as_float(r.w[e]);
}

// Loads the values of 256 columns starting at p, of which `left` exist (others are 0).
// KEEP: the data will be read again (default: streaming).
template <typename T, int LAYOUT, bool KEEP = false>
__device__ __forceinline__ Raw8<T> load8(const T* p, int64_t left, int lane) {
  Raw8<T> r;
  if (LAYOUT == kVec && lane * 8 + 8 <= left) {
    const uint4* q = reinterpret_cast<const uint4*>(p + lane * 8);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
      const uint4 v = KEEP ? __ldg(q + i) : __ldcs(q + i);
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) * 2; ++i) r.w[i] = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = lane_col<LAYOUT>(lane, e);
    if (c >= left) continue;
    if constexpr (sizeof(T) == 2) r.w[e >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[c]) << (16 * (e & 1));
    else r.w[e] = reinterpret_cast<const uint32_t*>(p)[c];
  }
  return r;
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Stores eight values of 256 columns starting at p, of which `left` exist.
template <typename T, int LAYOUT>
__device__ __forceinline__ void store8(T* p, int64_t left, int lane, const float (&v)[8]) {
  if (LAYOUT == kVec && lane * 8 + 8 <= left) {
    uint4* q = reinterpret_cast<uint4*>(p + lane * 8);
    if constexpr (sizeof(T) == 2) {
      __stcs(q, make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7])));
    } else {
      __stcs(reinterpret_cast<float4*>(q), make_float4(v[0], v[1], v[2], v[3]));
      __stcs(reinterpret_cast<float4*>(q) + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = lane_col<LAYOUT>(lane, e);
    if (c < left) p[c] = narrow<T>(v[e]);
  }
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
