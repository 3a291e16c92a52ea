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

// ------------------------------------------------------------- pairs of fp32 operations

// Two fp32 operations per instruction (each rounded as the scalar one would be).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 parts(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// max of magnitudes that keeps a NaN.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ------------------------------------------------------------- eight columns of a lane

// A warp covers 256 columns of a row at a time, eight per lane, as 8 / N pieces of N
// neighbouring columns: piece i of lane l holds columns (32 i + l) N .. (32 i + l) N + N - 1,
// so that a warp's access to a piece is contiguous.  N = 8 for bf16 and 4 for fp32 make
// pieces of 16 bytes (fp32 as eight neighbours a lane, two accesses with gaps, measured 35
// against 30 us for a lookup of 32768 x 1024); N = 4 also serves bf16 beside fp32 in one
// kernel.  They need rows that start on a piece's boundary; N = 1 takes every address.
enum Layout : int { kStrided = 1, kVec4 = 4, kVec8 = 8 };
template <typename T>
constexpr int kWide = sizeof(T) == 2 ? kVec8 : kVec4;

template <int N>
__device__ __forceinline__ int lane_col(int lane, int e) {
  return (e / N * 32 + lane) * N + e % N;
}

// Raw bits of a lane's eight values; with N = 1 a word each, so that bf16 loads need not have
// arrived to be held (packing them on arrival made a prefetch of the next row wait for them).
template <typename T, int N>
struct Raw8 {
  uint32_t w[N == kStrided ? 8 : sizeof(T) * 2];
};

template <typename T, int N>
__device__ __forceinline__ float raw_value(const Raw8<T, N>& r, int e) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[e]);
  else if constexpr (N == kStrided) return __uint_as_float(r.w[e] << 16);
  else return __uint_as_float(e & 1 ? r.w[e >> 1] & 0xFFFF0000u : r.w[e >> 1] << 16);
}

// The eight values as pairs.
template <typename T, int N>
__device__ __forceinline__ void unpack8(const Raw8<T, N>& r, F2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2(raw_value<T, N>(r, 2 * i), raw_value<T, N>(r, 2 * i + 1));
}

// Columns of a slice that starts at c0, at most 256, none past the row's end.
__device__ __forceinline__ int slice_left(int64_t cols, int64_t c0) {
  return static_cast<int>(max(static_cast<int64_t>(0), min(cols - c0, static_cast<int64_t>(256))));
}

// Loads the values of 256 columns starting at p, of which `left` exist (others are 0).
// KEEP: the data will be read again (default: streaming).
template <typename T, int N, bool KEEP = false>
__device__ __forceinline__ Raw8<T, N> load8(const T* p, int left, int lane) {
  constexpr int kWords = N * static_cast<int>(sizeof(T)) / 4;  // of a piece
  Raw8<T, N> r;
  auto element = [&](int c) -> uint32_t {
    if constexpr (sizeof(T) == 2) return reinterpret_cast<const uint16_t*>(p)[c];
    else return reinterpret_cast<const uint32_t*>(p)[c];
  };
  if constexpr (N == kStrided) {
    if (left >= 256) {  // (uniform over the warp: no check per element)
#pragma unroll
      for (int e = 0; e < 8; ++e) r.w[e] = element(lane_col<N>(lane, e));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.w[e] = lane_col<N>(lane, e) < left ? element(lane_col<N>(lane, e)) : 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
      const int c = lane_col<N>(lane, i * N);
      uint32_t* w = r.w + i * kWords;
      if (c + N <= left) {
        if constexpr (kWords == 4) {
          const uint4* q = reinterpret_cast<const uint4*>(p + c);
          const uint4 v = KEEP ? __ldg(q) : __ldcs(q);
          w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
          static_assert(kWords == 2 || kWords == 4, "pieces of 8 or 16 bytes");
          const uint2* q = reinterpret_cast<const uint2*>(p + c);
          const uint2 v = KEEP ? __ldg(q) : __ldcs(q);
          w[0] = v.x, w[1] = v.y;
        }
      } else if (c < left) {
        uint32_t v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = c + e < left ? element(c + e) : 0u;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if constexpr (sizeof(T) == 4) w[e] = v[e];
          else if (e & 1) w[e >> 1] = __byte_perm(v[e - 1], v[e], 0x5410);
        }
      } else {  // (most lanes of a narrow row)
#pragma unroll
        for (int e = 0; e < kWords; ++e) w[e] = 0u;
      }
    }
  }
  return r;
}

// 256 columns on their way through shared memory.  A lane copies the pieces that it will use
// itself, so that nothing has to be exchanged: `copy` starts it (past the row's end come
// zeros), `take` reads them once cp_async_wait has returned.
template <typename T, int N>
struct alignas(16) LaneSlot {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T)), kWords = kBytes / 4;  // of a piece
  uint32_t w[8 / N][32][kWords];
  __device__ __forceinline__ void copy(const T* p, int left, int lane) {
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
      const int c = lane_col<N>(lane, i * N);
      const int bytes = max(0, min(kBytes, (left - c) * static_cast<int>(sizeof(T))));
      const T* from = p + (bytes > 0 ? c : 0);
      if constexpr (kBytes == 16) cp_async16(smem_addr(w[i][lane]), from, bytes);
      else cp_async_small<kBytes>(smem_addr(w[i][lane]), from, bytes);
    }
  }
  __device__ __forceinline__ Raw8<T, N> take(int lane) const {
    Raw8<T, N> r;
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
      if constexpr (kWords == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(w[i][lane]);
        r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(w[i][lane]);
        r.w[2 * i] = v.x, r.w[2 * i + 1] = v.y;
      }
    }
    return r;
  }
};

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Stores eight values of 256 columns starting at p, of which `left` exist.
template <typename T, int N>
__device__ __forceinline__ void store8(T* p, int left, int lane, const float (&v)[8]) {
  if constexpr (N == kStrided) {
    if (left >= 256) {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[lane_col<N>(lane, e)] = narrow<T>(v[e]);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8 / N; ++i) {
    const int c = lane_col<N>(lane, i * N);
    const float* x = v + i * N;
    if constexpr (N > 1) {
      if (c + N <= left) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int e = 0; e < N; e += 4) __stcs(reinterpret_cast<float4*>(p + c + e), make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]));
        } else if constexpr (N == 8) {
          __stcs(reinterpret_cast<uint4*>(p + c), make_uint4(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]),
                                                             pack2_bf16(x[4], x[5]), pack2_bf16(x[6], x[7])));
        } else {
          __stcs(reinterpret_cast<uint2*>(p + c), make_uint2(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3])));
        }
        continue;
      }
      if (c >= left) continue;
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < left) p[c + e] = narrow<T>(x[e]);
  }
}

template <typename T, int LAYOUT>
__device__ __forceinline__ void store8(T* p, int left, int lane, const F2 (&v)[4]) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = parts(v[i]);
    s[2 * i] = x.x;
    s[2 * i + 1] = x.y;
  }
  store8<T, LAYOUT>(p, left, lane, s);
}

// Floats of 256 columns in shared memory: first values 0..3 of every lane, then 4..7, so
// that a warp's 16-byte accesses meet no bank twice.  `smem_col` is the column of place i.
template <int LAYOUT>
__device__ __forceinline__ int smem_col(int i) {
  const int r = i & 255;
  return (i & ~255) + lane_col<LAYOUT>((r >> 2) & 31, (r >> 7) * 4 + (r & 3));
}
__device__ __forceinline__ void lds8(const float* p, int lane, F2 (&v)[4]) {
  const float4 a = reinterpret_cast<const float4*>(p)[lane], b = reinterpret_cast<const float4*>(p)[32 + lane];
  v[0] = f2(a.x, a.y);
  v[1] = f2(a.z, a.w);
  v[2] = f2(b.x, b.y);
  v[3] = f2(b.z, b.w);
}
__device__ __forceinline__ void sts8(float* p, int lane, const F2 (&v)[4]) {
  const float2 a = parts(v[0]), b = parts(v[1]), c = parts(v[2]), d = parts(v[3]);
  reinterpret_cast<float4*>(p)[lane] = make_float4(a.x, a.y, b.x, b.y);
  reinterpret_cast<float4*>(p)[32 + lane] = make_float4(c.x, c.y, d.x, d.y);
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
// Codes are round(x * inv), ties to even; |x * inv| <= 127 up to rounding, so adding
// 1.5 * 2^23 leaves the integer in the low bits of the sum.  (A NaN or infinity, in a block
// whose scale is NaN, gives an arbitrary code.)
// The codes of eight values (two words, in the order of the values): the sum's low byte of
// each.  (The products are scalar: a packed product and sum were measured to be contracted
// to a fused one, which rounds differently next to ties.)
__device__ __forceinline__ uint2 ckpt_codes8(const F2 (&v)[4], float inv_lo, float inv_hi) {
  uint32_t b[8];
  const F2 magic = f2(12582912.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float k = i < 2 ? inv_lo : inv_hi;
    const float2 x = parts(v[i]), s = parts(add2(f2(__fmul_rn(x.x, k), __fmul_rn(x.y, k)), magic));
    b[2 * i] = __float_as_uint(s.x);
    b[2 * i + 1] = __float_as_uint(s.y);
  }
  return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}
// The values of eight codes: a code plus 128 becomes the low byte of 2^23 as a float, and
// the rest is exact up to the product with the scale.
__device__ __forceinline__ void ckpt_values8(uint2 q, float lo_scale, float hi_scale, F2 (&v)[4]) {
  const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};
  const F2 bias = f2(-8388736.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = w[i >> 1];
    const float lo = __uint_as_float(__byte_perm(x, 0x4B000000u, i & 1 ? 0x7442 : 0x7440));
    const float hi = __uint_as_float(__byte_perm(x, 0x4B000000u, i & 1 ? 0x7443 : 0x7441));
    v[i] = mul2(add2(f2(lo, hi), bias), f2(i < 2 ? lo_scale : hi_scale));
  }
}

// Codes of 256 columns, the same columns per lane as the values'; rows of codes start on
// 16-byte boundaries, and are padded to them, so that a begun piece is always there.
template <int N>
__device__ __forceinline__ uint2 load_codes8(const int8_t* p, int left, int lane) {
  if constexpr (N == kVec8) {
    return lane * 8 < left ? __ldcs(reinterpret_cast<const uint2*>(p) + lane) : make_uint2(0u, 0u);
  } else if constexpr (N == kVec4) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p) + lane;
    return make_uint2(lane * 4 < left ? __ldcs(q) : 0u, 128 + lane * 4 < left ? __ldcs(q + 32) : 0u);
  } else {
    uint32_t v[8];
    if (left >= 256) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = static_cast<uint8_t>(p[lane_col<N>(lane, e)]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = lane_col<N>(lane, e);
        v[e] = c < left ? static_cast<uint8_t>(p[c]) : 0u;
      }
    }
    return make_uint2(__byte_perm(__byte_perm(v[0], v[1], 0x0040), __byte_perm(v[2], v[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(v[4], v[5], 0x0040), __byte_perm(v[6], v[7], 0x0040), 0x5410));
  }
}
template <int N>
__device__ __forceinline__ void store_codes8(int8_t* p, int left, int lane, uint2 q) {
  if constexpr (N == kVec8) {
    if (lane * 8 < left) __stcs(reinterpret_cast<uint2*>(p) + lane, q);
  } else if constexpr (N == kVec4) {
    uint32_t* to = reinterpret_cast<uint32_t*>(p) + lane;
    if (lane * 4 < left) __stcs(to, q.x);
    if (128 + lane * 4 < left) __stcs(to + 32, q.y);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = lane_col<N>(lane, e);
      if (c < left) p[c] = static_cast<int8_t>(((e < 4 ? q.x : q.y) >> (8 * (e & 3))) & 0xFFu);
    }
  }
}

// Largest magnitudes of the (one or two) blocks that a lane's eight of 256 columns lie in,
// from all the lanes' values (NaN if there is one); columns past the row's end hold 0.
// N = 8: a block is half a warp; otherwise it is four values of every lane.
template <int LAYOUT>
__device__ __forceinline__ void block_tops(const F2 (&v)[4], float (&top)[2]) {
  const float2 a = parts(v[0]), b = parts(v[1]), c = parts(v[2]), d = parts(v[3]);
  top[0] = max_abs_nan(max_abs_nan(a.x, a.y, b.x), b.y, b.y);
  top[1] = max_abs_nan(max_abs_nan(c.x, c.y, d.x), d.y, d.y);
  if constexpr (LAYOUT == kVec8) {
    top[0] = max_nan(top[0], top[1]);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) top[0] = max_nan(top[0], __shfl_xor_sync(0xFFFFFFFFu, top[0], d));
    top[1] = top[0];
  } else {
    // (magnitudes as integers are ordered like the values, with NaN above infinity)
#pragma unroll
    for (int b = 0; b < 2; ++b)
      top[b] = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top[b])));
  }
}

// Scales of the blocks of N slices of 256 columns, from block_tops.  The two quotients cost
// more than the codes of a lane's eight values, so each lane computes those of one slice
// (and one block) and the others take them from it.
template <int LAYOUT, int N>
__device__ __forceinline__ void block_scales(const float (&top)[N][2], int lane, CkptScale (&s)[N][2]) {
  constexpr int kJobs = LAYOUT == kVec8 ? N : 2 * N;
  static_assert(kJobs <= 16, "one lane of a half warp per scale");
  float mine = top[0][0];
#pragma unroll
  for (int j = 1; j < kJobs; ++j)
    if ((lane & 15) == j) mine = LAYOUT == kVec8 ? top[j][0] : top[j >> 1][j & 1];
  const CkptScale r = ckpt_scale(mine, !(mine < __int_as_float(0x7F800000)));
#pragma unroll
  for (int j = 0; j < kJobs; ++j) {
    const int from = (lane & 16) | j;
    CkptScale& to = LAYOUT == kVec8 ? s[j][0] : s[j >> 1][j & 1];
    to.scale = __shfl_sync(0xFFFFFFFFu, r.scale, from);
    to.inv = __shfl_sync(0xFFFFFFFFu, r.inv, from);
    if (LAYOUT == kVec8) s[j][1] = to;
  }
}
// Stores the scales of 256 columns, of which `left` exist, at p.
template <int LAYOUT>
__device__ __forceinline__ void store_scales(float* p, int left, int lane, const CkptScale (&s)[2]) {
  if constexpr (LAYOUT == kVec8) {
    if ((lane & 15) == 0 && lane * 8 < left) p[lane >> 4] = s[0].scale;
  } else {
    if (lane == 0) {
      p[0] = s[0].scale;
      if (left > kCkptBlock) p[1] = s[1].scale;
    }
  }
}
template <int LAYOUT>
__device__ __forceinline__ uint2 ckpt_codes(const F2 (&v)[4], const CkptScale (&s)[2]) {
  return ckpt_codes8(v, s[0].inv, LAYOUT == kVec8 ? s[0].inv : s[1].inv);
}
// Values of 256 columns' codes, of which `left` columns exist; p: their scales.
template <int LAYOUT>
__device__ __forceinline__ void ckpt_values(uint2 q, const float* p, int left, int lane, F2 (&v)[4]) {
  if constexpr (LAYOUT == kVec8) {
    const float s = lane * 8 < left ? p[lane >> 4] : 0.f;
    ckpt_values8(q, s, s, v);
  } else {
    ckpt_values8(q, p[0], left > kCkptBlock ? p[1] : 0.f, v);
  }
}

}  // namespace adasum
