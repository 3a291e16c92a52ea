// train_checkpoint.cu -- activations kept in 8 bits: pack, unpack, and the GELU whose
// forward pass packs its input and whose backward pass starts from the codes.
//
// Times in the comments are those of one launch between two events (the library's profiler; 4
// to 6 us of it are the launch), unless they are said to be of a call in a graph of many or of a
// pass, a call among others through the Python binding.
#include "adasum_host.h"
#include "adasum_launch.h"
#include "adasum_train.cuh"

namespace adasum {
namespace {

constexpr int kCkptThreads = 256;
constexpr int kCkptWarps = kCkptThreads / 32;
constexpr int kSlice = 256;  // columns a warp moves at a time
constexpr int kItems = 4;    // of them in flight

enum Act : int { kActNone = 0, kActErf = 1, kActTanh = 2 };

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ F2 rcp2(F2 x) {
  const float2 p = parts(x);
  return f2(rcp_approx(p.x), rcp_approx(p.y));
}
__device__ __forceinline__ F2 exp2_2(F2 x) {
  const float2 p = parts(x);
  return f2(ex2_approx(p.x), ex2_approx(p.y));
}

// gelu of two values, and its slope.
//
// Erf form: gelu = max(x, 0) - b q with b = |x| and q = 1/2 erfc(b / sqrt 2), the upper tail
// of the normal distribution; slope = Phi + x phi, where the density phi takes q's
// exponential.
// FINE (fp32 activations): q = H(z) exp(-b^2 / 2), z = 0.35 b / (1 + 0.35 b), where H is
// 1/2 exp(b^2 / 2) erfc(b / sqrt 2) as a polynomial of degree 9 in z, fitted here for the
// least relative error over 0 <= b <= 14.5 (3e-8; reweighted least squares at Chebyshev
// nodes).  z is small where q is large, so the roundings of the quotient do not reach q
// there: q is right to (22 + 2 b^2) 2^-24 of itself (ex2's and rcp's stated errors, 2^-22 and
// 2^-23, and one 2^-24 per rounding).
// Normal activations: value and slope off by 2.9e-8 and 4.1e-8 of their norm (the form below:
// 8.3e-8 and 1.0e-7), for 32768 x 4096, a call in a graph, forward 183 us against 181, backward
// 226 against 215, with the output 302 against 286.
// Else (bf16): the five terms of Abramowitz and Stegun, Handbook of Mathematical Functions,
// 7.1.26,
//     q = 1/2 (a1 t + ... + a5 t^5) exp(-b^2 / 2), t = 1 / (1 + p b / sqrt 2),
// whose error of erf, below 1.5e-7, is nothing beside bf16's rounding but twice fp32's.
// Two special-function operations per value and 10 to 16 others, in pairs, where the
// library's erf and exp would be bound by instruction issue.
// Tanh form: 1/2 (1 + tanh u) is the logistic function of 2 u, s = 1 / (1 + exp(-2 u));
// gelu = x s, slope = s + x s (1 - s) (2 u)', with 1 - s = s exp(-2 u) so that nothing cancels.
// x is held within the range where s differs from 0 and 1 in fp32's normal range, so that no
// product of zero and infinity arises; NaN passes.
template <int ACT, bool FINE, bool VALUE, bool SLOPE>
__device__ __forceinline__ void gelu2(F2 x, F2& value, F2& slope) {
  const float2 xs = parts(x);
  if constexpr (ACT == kActErf && FINE) {
    // a = -|x|; beyond 16 q is 0, and the bound keeps 0 * infinity out
    const F2 a = f2(max_nan(-fabsf(xs.x), -16.f), max_nan(-fabsf(xs.y), -16.f));
    const F2 z = mul2(mul2(a, f2(-0.35f)), rcp2(fma2(a, f2(-0.35f), f2(1.f))));
    const F2 e = exp2_2(mul2(mul2(a, a), f2(-0.72134752044f)));
    F2 p = fma2(z, f2(0.028265389f), f2(-0.11498016f));
    p = fma2(p, z, f2(0.14782675f));
    p = fma2(p, z, f2(-0.043232292f));
    p = fma2(p, z, f2(0.045680154f));
    p = fma2(p, z, f2(-0.16608815f));
    p = fma2(p, z, f2(-0.15852852f));
    p = fma2(p, z, f2(0.9008877f));
    p = fma2(p, z, f2(-1.1398324f));
    p = fma2(p, z, f2(0.5f));
    const F2 q = mul2(p, e);
    if constexpr (VALUE) value = fma2(a, q, f2(max_nan(xs.x, 0.f), max_nan(xs.y, 0.f)));
    if constexpr (SLOPE) {  // Phi is q up to 0 and 1 - q above
      const float2 qs = parts(q);
      const F2 phi = f2(xs.x > 0.f ? 1.f - qs.x : qs.x, xs.y > 0.f ? 1.f - qs.y : qs.y);
      slope = fma2(mul2(x, f2(0.39894228040f)), e, phi);
    }
  } else if constexpr (ACT == kActErf) {
    // a = -|x|; beyond 16 q is 0, and the bound keeps 0 * infinity out
    const F2 a = f2(max_nan(-fabsf(xs.x), -16.f), max_nan(-fabsf(xs.y), -16.f));
    const F2 t = rcp2(fma2(a, f2(-0.3275911f * 0.70710678118f), f2(1.f)));
    const F2 e = exp2_2(mul2(mul2(a, a), f2(-0.72134752044f)));
    F2 p = fma2(t, f2(0.5f * 1.061405429f), f2(0.5f * -1.453152027f));
    p = fma2(p, t, f2(0.5f * 1.421413741f));
    p = fma2(p, t, f2(0.5f * -0.284496736f));
    p = fma2(p, t, f2(0.5f * 0.254829592f));
    const F2 q = mul2(mul2(p, t), e);
    if constexpr (VALUE) value = fma2(a, q, f2(max_nan(xs.x, 0.f), max_nan(xs.y, 0.f)));
    if constexpr (SLOPE) {
      const float2 qs = parts(q);
      const F2 phi = add2(f2(copysignf(0.5f - qs.x, xs.x), copysignf(0.5f - qs.y, xs.y)), f2(0.5f));
      slope = fma2(mul2(x, f2(0.39894228040f)), e, phi);
    }
  } else {
    constexpr float kTwoC = 1.5957691216f, kLog2e = 1.4426950409f, kCube = 0.044715f;
    const F2 c = f2(max_nan(xs.x, -8.f), max_nan(xs.y, -8.f));
    F2 b = c;
    if constexpr (SLOPE) {
      const float2 cs = parts(c);
      b = f2(min_nan(cs.x, 8.f), min_nan(cs.y, 8.f));
    }
    const F2 sq = mul2(b, b);
    const F2 e = exp2_2(mul2(b, fma2(sq, f2(-kTwoC * kLog2e * kCube), f2(-kTwoC * kLog2e))));
    const F2 s = rcp2(add2(e, f2(1.f)));
    if constexpr (VALUE) value = mul2(c, s);
    if constexpr (SLOPE) {
      const F2 du = mul2(b, fma2(sq, f2(3.f * kTwoC * kCube), f2(kTwoC)));
      slope = fma2(mul2(du, s), mul2(s, e), s);
    }
  }
}

struct PackArgs {
  const void* x;
  int64_t rows, cols, ld;
  int8_t* codes;
  float* scales;
  void* y;  // the activation's output (kActNone: null)
  int64_t pitch, nscales;  // of a row's codes and scales
  uint32_t groups;         // warps that share a row
};
struct UnpackArgs {
  const int8_t* codes;
  const float* scales;
  int64_t rows, cols;
  const void* dy;  // kActNone: null
  int64_t ld_dy;
  void* out;       // the values (kActNone) or grad_x
  void* y;         // the activation again; null: not wanted
  int64_t pitch, nscales;
  uint32_t groups;
};

// A warp takes kItems slices of 256 columns and loads them all before it works on the first:
// ROW neighbouring ones of each of kItems / ROW rows, so that a slice's place is the warp's
// plus a few constants.  Bound by bytes, each value is read and written once: 32768 x 4096
// bf16 with GELU forward 114 us, 5.9 TB/s, backward with the output once more 139 us, 6.7
// TB/s.  (Eight slices in flight: 178 and 185 us.)  513 x 1000 fp32
// takes 7 us each way, its launch and one round of latency.
template <int ROW>
struct Place {
  int64_t row, c0;
  int rows, cols;  // that exist from here on, as far as the warp goes
  template <typename A>
  __device__ __forceinline__ Place(const A& a) {
    const uint32_t warp = blockIdx.x * kCkptWarps + (threadIdx.x >> 5), block = warp / a.groups;
    row = static_cast<int64_t>(block) * (kItems / ROW);
    c0 = static_cast<int64_t>(warp - block * a.groups) * (ROW * kSlice);
    rows = static_cast<int>(max(static_cast<int64_t>(0), min(a.rows - row, static_cast<int64_t>(kItems))));
    cols = static_cast<int>(min(a.cols - c0, static_cast<int64_t>(ROW * kSlice)));
  }
  // of slice i: its columns that exist, and its offset from the warp's place in a matrix
  // whose rows are ld apart
  __device__ __forceinline__ int left(int i) const {
    return i / ROW < rows ? max(0, min(cols - i % ROW * kSlice, kSlice)) : 0;
  }
  __device__ __forceinline__ static int64_t step(int i, int64_t ld) { return i / ROW * ld + i % ROW * kSlice; }
  __device__ __forceinline__ static int64_t scale_step(int i, int64_t n) {
    return i / ROW * n + i % ROW * (kSlice / kCkptBlock);
  }
};

template <typename T, int ACT, int LAYOUT, int ROW>
__global__ void __launch_bounds__(kCkptThreads, sizeof(T) == 2 ? 4 : 3) pack_kernel(const PackArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const Place<ROW> at(a);
  if (at.rows == 0) return;
  F2 v[kItems][4];
  {
    const T* x = static_cast<const T*>(a.x) + at.row * a.ld + at.c0;
    Raw8<T, LAYOUT> r[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) r[i] = load8<T, LAYOUT>(x + at.step(i, a.ld), at.left(i), lane);
#pragma unroll
    for (int i = 0; i < kItems; ++i) unpack8<T, LAYOUT>(r[i], v[i]);
  }
  float top[kItems][2];
#pragma unroll
  for (int i = 0; i < kItems; ++i) block_tops<LAYOUT>(v[i], top[i]);
  CkptScale sc[kItems][2];
  block_scales<LAYOUT, kItems>(top, lane, sc);
  int8_t* codes = a.codes + at.row * a.pitch + at.c0;
  float* scales = a.scales + at.row * a.nscales + at.c0 / kCkptBlock;
  T* y = static_cast<T*>(a.y) + at.row * a.cols + at.c0;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int left = at.left(i);
    if (left <= 0) continue;
    store_codes8<LAYOUT>(codes + at.step(i, a.pitch), left, lane, ckpt_codes<LAYOUT>(v[i], sc[i]));
    store_scales<LAYOUT>(scales + at.scale_step(i, a.nscales), left, lane, sc[i]);
    if constexpr (ACT != kActNone) {
      F2 unused;
#pragma unroll
      for (int e = 0; e < 4; ++e) gelu2<ACT, sizeof(T) == 4, true, false>(v[i][e], v[i][e], unused);
      store8<T, LAYOUT>(y + at.step(i, a.cols), left, lane, v[i]);
    }
  }
}

template <typename T, int ACT, bool AGAIN, int LAYOUT, int ROW>
__global__ void __launch_bounds__(kCkptThreads, 4) unpack_kernel(const UnpackArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const Place<ROW> at(a);
  if (at.rows == 0) return;
  const int8_t* codes = a.codes + at.row * a.pitch + at.c0;
  const float* scales = a.scales + at.row * a.nscales + at.c0 / kCkptBlock;
  const T* dy = static_cast<const T*>(a.dy) + at.row * a.ld_dy + at.c0;
  uint2 q[kItems];
  Raw8<T, LAYOUT> r[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    q[i] = load_codes8<LAYOUT>(codes + at.step(i, a.pitch), at.left(i), lane);
    if constexpr (ACT != kActNone) r[i] = load8<T, LAYOUT>(dy + at.step(i, a.ld_dy), at.left(i), lane);
  }
  T* out = static_cast<T*>(a.out) + at.row * a.cols + at.c0;
  T* again = static_cast<T*>(a.y) + at.row * a.cols + at.c0;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int left = at.left(i);
    if (left <= 0) continue;
    F2 v[4];
    ckpt_values<LAYOUT>(q[i], scales + at.scale_step(i, a.nscales), left, lane, v);
    if constexpr (ACT != kActNone) {
      F2 d[4], y[4];
      unpack8<T, LAYOUT>(r[i], d);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        F2 slope;
        gelu2<ACT, sizeof(T) == 4, AGAIN, true>(v[e], y[e], slope);
        v[e] = mul2(slope, d[e]);
      }
      if constexpr (AGAIN) store8<T, LAYOUT>(again + at.step(i, a.cols), left, lane, y);
    }
    store8<T, LAYOUT>(out + at.step(i, a.cols), left, lane, v);
  }
}

// Slices of a warp that lie in one row.
template <typename A>
int slices_per_row(const A& a) {
  return a.cols <= kSlice ? 1 : a.cols <= 2 * kSlice ? 2 : 4;
}

template <typename T, int LAYOUT, int ROW>
int launch_pack_as(const PackArgs& a, int act, unsigned grid, cudaStream_t stream) {
  auto k = act == kActNone  ? pack_kernel<T, kActNone, LAYOUT, ROW>
           : act == kActErf ? pack_kernel<T, kActErf, LAYOUT, ROW>
                            : pack_kernel<T, kActTanh, LAYOUT, ROW>;
  return launch_pdl(k, dim3(grid), dim3(kCkptThreads), 0, stream, a);
}
template <typename T, int LAYOUT>
int launch_pack(const PackArgs& a, int act, unsigned grid, cudaStream_t stream) {
  const int row = slices_per_row(a);
  if (row == 1) return launch_pack_as<T, LAYOUT, 1>(a, act, grid, stream);
  if (row == 2) return launch_pack_as<T, LAYOUT, 2>(a, act, grid, stream);
  return launch_pack_as<T, LAYOUT, 4>(a, act, grid, stream);
}
template <typename T, int LAYOUT, int ROW>
int launch_unpack_as(const UnpackArgs& a, int act, unsigned grid, cudaStream_t stream) {
  const bool y = a.y != nullptr;
  auto k = act == kActNone  ? unpack_kernel<T, kActNone, false, LAYOUT, ROW>
           : act == kActErf ? (y ? unpack_kernel<T, kActErf, true, LAYOUT, ROW> : unpack_kernel<T, kActErf, false, LAYOUT, ROW>)
                            : (y ? unpack_kernel<T, kActTanh, true, LAYOUT, ROW> : unpack_kernel<T, kActTanh, false, LAYOUT, ROW>);
  return launch_pdl(k, dim3(grid), dim3(kCkptThreads), 0, stream, a);
}
template <typename T, int LAYOUT>
int launch_unpack(const UnpackArgs& a, int act, unsigned grid, cudaStream_t stream) {
  const int row = slices_per_row(a);
  if (row == 1) return launch_unpack_as<T, LAYOUT, 1>(a, act, grid, stream);
  if (row == 2) return launch_unpack_as<T, LAYOUT, 2>(a, act, grid, stream);
  return launch_unpack_as<T, LAYOUT, 4>(a, act, grid, stream);
}

// Deals a call's slices to warps; the grid, or 0 when there are too many.  Dense rows of whole
// blocks follow each other without a gap in every buffer, so they are taken as one long row.
template <typename A>
unsigned deal(A& a, int64_t ld) {
  if (a.cols % kCkptBlock == 0 && (ld == a.cols || a.rows == 1)) {
    a.cols *= a.rows;
    a.rows = 1;
  }
  a.pitch = ckpt_pitch(a.cols);
  a.nscales = ckpt_scales(a.cols);
  const int row = slices_per_row(a);
  const int64_t groups = (a.cols + row * kSlice - 1) / (row * kSlice);
  const int64_t blocks = (a.rows + kItems / row - 1) / (kItems / row);
  if (groups > INT32_MAX / blocks) return 0;
  a.groups = static_cast<uint32_t>(groups);
  return static_cast<unsigned>((groups * blocks + kCkptWarps - 1) / kCkptWarps);
}

adasum_status_t check_shape(int64_t rows, int64_t cols, int dtype) {
  if (rows < 0 || cols < 1 || !valid_dtype(dtype)) return ADASUM_ERR_INVALID_ARG;
  if (cols > INT32_MAX || rows > INT64_MAX / (8 * cols)) return ADASUM_ERR_UNSUPPORTED;
  return ADASUM_OK;
}

adasum_status_t pack(PackArgs a, int dtype, int act, cudaStream_t stream) {
  if (adasum_status_t st = check_shape(a.rows, a.cols, dtype)) return st;
  if (a.rows == 0) return ADASUM_OK;
  if (a.x == nullptr || a.codes == nullptr || a.scales == nullptr || (act != kActNone && a.y == nullptr) ||
      !valid_ld(a.rows, a.cols, a.ld) || !is_aligned(a.codes, 16))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype);
  BufferSet set;
  set.read(a.x, span_bytes(a.rows, a.cols, a.ld, e), e);
  set.write(a.codes, a.rows * ckpt_pitch(a.cols), 16);
  set.write(a.scales, a.rows * ckpt_scales(a.cols) * 4, 4);
  set.write(a.y, a.rows * a.cols * e, e);
  if (adasum_status_t st = set.check()) return st;
  const double n = static_cast<double>(a.rows) * a.cols;
  const bool vec = is_aligned(a.x, 16) && is_aligned(a.y, 16) && a.ld * e % 16 == 0 && (act == kActNone || a.cols * e % 16 == 0);
  const unsigned grid = deal(a, a.ld);
  if (grid == 0) return ADASUM_ERR_UNSUPPORTED;
  return counted_launch(stream, act ? "gelu_checkpoint" : "checkpoint_pack", n * (e + 1 + (act ? e : 0)), [&] {
    if (dtype == kBF16)
      return vec ? launch_pack<bf16, kVec8>(a, act, grid, stream) : launch_pack<bf16, kStrided>(a, act, grid, stream);
    return vec ? launch_pack<float, kVec4>(a, act, grid, stream) : launch_pack<float, kStrided>(a, act, grid, stream);
  });
}

adasum_status_t unpack(UnpackArgs a, int dtype, int act, cudaStream_t stream) {
  if (adasum_status_t st = check_shape(a.rows, a.cols, dtype)) return st;
  if (a.rows == 0) return ADASUM_OK;
  if (a.codes == nullptr || a.scales == nullptr || a.out == nullptr || !is_aligned(a.codes, 16) ||
      (act != kActNone && (a.dy == nullptr || !valid_ld(a.rows, a.cols, a.ld_dy))))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype);
  BufferSet set;
  set.read(a.codes, a.rows * ckpt_pitch(a.cols), 16);
  set.read(a.scales, a.rows * ckpt_scales(a.cols) * 4, 4);
  if (act != kActNone) set.read(a.dy, span_bytes(a.rows, a.cols, a.ld_dy, e), e);
  set.write(a.out, a.rows * a.cols * e, e);
  set.write(a.y, a.rows * a.cols * e, e);
  if (adasum_status_t st = set.check()) return st;
  const double n = static_cast<double>(a.rows) * a.cols;
  const bool vec = is_aligned(a.out, 16) && is_aligned(a.y, 16) && a.cols * e % 16 == 0 &&
                   (act == kActNone || (is_aligned(a.dy, 16) && a.ld_dy * e % 16 == 0));
  const unsigned grid = deal(a, act == kActNone ? a.cols : a.ld_dy);
  if (grid == 0) return ADASUM_ERR_UNSUPPORTED;
  return counted_launch(stream, act ? "gelu_grad_checkpoint" : "checkpoint_unpack",
                        n * (1 + e + (act ? e : 0) + (a.y ? e : 0)), [&] {
    if (dtype == kBF16)
      return vec ? launch_unpack<bf16, kVec8>(a, act, grid, stream) : launch_unpack<bf16, kStrided>(a, act, grid, stream);
    return vec ? launch_unpack<float, kVec4>(a, act, grid, stream) : launch_unpack<float, kStrided>(a, act, grid, stream);
  });
}

}  // namespace
}  // namespace adasum

using namespace adasum;

extern "C" {

adasum_status_t adasum_checkpoint_pack(const void* x, int64_t rows, int64_t cols, int64_t ld, adasum_dtype_t dtype,
                                       int8_t* codes, float* scales, adasum_stream_t stream) {
  EntryScope scope("adasum_checkpoint_pack");
  return pack(PackArgs{x, rows, cols, ld, codes, scales, nullptr, 0, 0, 0}, dtype, kActNone,
              reinterpret_cast<cudaStream_t>(stream));
}

adasum_status_t adasum_checkpoint_unpack(const int8_t* codes, const float* scales, int64_t rows, int64_t cols,
                                         adasum_dtype_t dtype, void* out, adasum_stream_t stream) {
  EntryScope scope("adasum_checkpoint_unpack");
  return unpack(UnpackArgs{codes, scales, rows, cols, nullptr, 0, out, nullptr, 0, 0, 0}, dtype, kActNone,
                reinterpret_cast<cudaStream_t>(stream));
}

adasum_status_t adasum_gelu_checkpointed(const void* x, int64_t rows, int64_t cols, int64_t ld, adasum_dtype_t dtype,
                                         int tanh_form, void* y, int8_t* codes, float* scales,
                                         adasum_stream_t stream) {
  EntryScope scope("adasum_gelu_checkpointed");
  return pack(PackArgs{x, rows, cols, ld, codes, scales, y, 0, 0, 0}, dtype, tanh_form ? kActTanh : kActErf,
              reinterpret_cast<cudaStream_t>(stream));
}

adasum_status_t adasum_gelu_checkpointed_backward(const void* grad_out, int64_t ld_grad, const int8_t* codes,
                                                  const float* scales, int64_t rows, int64_t cols,
                                                  adasum_dtype_t dtype, int tanh_form, void* grad_x, void* y,
                                                  adasum_stream_t stream) {
  EntryScope scope("adasum_gelu_checkpointed_backward");
  return unpack(UnpackArgs{codes, scales, rows, cols, grad_out, ld_grad, grad_x, y, 0, 0, 0}, dtype,
                tanh_form ? kActTanh : kActErf, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
