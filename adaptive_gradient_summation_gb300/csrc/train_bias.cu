// train_bias.cu -- the learned relative position bias of attention scores by buckets, and the
// gradient of its table per worker.
//
// Times in the comments are those of one launch between two events (the library's profiler; 4
// to 6 us of it are the launch), unless they are said to be of a pass, a call among others
// through the Python binding.
#include <cmath>
#include <numeric>
#include <type_traits>
#include <vector>

#include "adasum_host.h"
#include "adasum_launch.h"
#include "adasum_train.cuh"

namespace adasum {
namespace {

constexpr int kMaxBuckets = ADASUM_BIAS_MAX_BUCKETS;
constexpr int kBiasThreads = 256, kBiasWarps = 8;

#ifdef ADASUM_BOUNDS_CHECK
__device__ int g_status;  // what an index check leaves (adasum_get_last_error)
#endif

// Buckets of one direction: distance d belongs to the last j with border[j] <= d.
struct Buckets {
  int n;               // of one direction
  int both;            // keys ahead have n of their own, after the others; else all are in bucket 0
  int64_t border[kMaxBuckets];
};

// `rel`: key's position less the query's.
__device__ __forceinline__ int bucket_of(const Buckets& b, int64_t rel) {
  int64_t d = rel < 0 ? -rel : b.both ? rel : 0;
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (b.border[m] <= d) lo = m;
    else hi = m;
  }
  return b.both && rel > 0 ? b.n + lo : lo;
}

// ------------------------------------------------------------------------------ forward

struct BiasArgs {
  const void* table;
  int table_dtype;
  int64_t heads, batch, queries, keys, offset;
  const void* scores;  // null: the bias alone
  int64_t stride_b, stride_h, stride_q;
  void* out;
  int row_groups;      // of a CTA's warps, four rows each; the others take other sequences
  int64_t per_cta;     // sequences
  Buckets buckets;
};

// Value e of a piece of 16 bytes, and a piece of values rounded and stored.
template <typename T>
__device__ __forceinline__ float value_of(const uint4& x, int e) {
  const uint32_t* w = &x.x;
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
  else return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
}
template <typename T, int E>
__device__ __forceinline__ void put_piece(T* to, const float (&v)[E]) {
  uint4 y;
  if constexpr (sizeof(T) == 4)
    y = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    y = make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[E - 4], v[E - 3]), pack2_bf16(v[E - 2], v[E - 1]));
  __stcs(reinterpret_cast<uint4*>(to), y);
}

// A piece of 16 bytes, all of them values of [first, last).
template <typename T>
__device__ __forceinline__ uint4 load_piece(const uint4* p, const T* first, const T* last) {
  const bool inside = ADASUM_CHECK(&g_status, reinterpret_cast<const T*>(p) >= first && reinterpret_cast<const T*>(p + 1) <= last);
  return inside ? __ldcs(p) : make_uint4(0u, 0u, 0u, 0u);
}
// A piece of which only some values may be of [first, last): the others are not read, and come as
// zeros.
template <typename T>
__device__ __forceinline__ uint4 load_edge(const uint4* p, const T* first, const T* last) {
  constexpr int E = 16 / sizeof(T);
  using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
  const T* at = reinterpret_cast<const T*>(p);
  uint32_t v[E];
#pragma unroll
  for (int e = 0; e < E; ++e)  // (all on their way before one is used)
    v[e] = at + e >= first && at + e < last ? reinterpret_cast<const Bits*>(at)[e] : 0u;
  if constexpr (sizeof(T) == 4) return make_uint4(v[0], v[1], v[2], v[3]);
  else return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[E - 4] | v[E - 3] << 16, v[E - 2] | v[E - 1] << 16);
}

// E keys a lane: neighbours (16 bytes, VEC) or 32 apart.  A CTA has up to 32 rows of one head
// and a warp's 32 E keys; the biases that occur there, one for each diagonal, go through shared
// memory (a word of padding every 32, so that lanes 4 or 8 apart meet no bank twice) into the
// registers of a warp's four rows, which serve all its sequences.  Bound by the bytes of the
// scores: 64 x 16 x 512 x 512 bf16 in 180 us, 6.0 TB/s, fp32 337, 6.4 TB/s; 511 x 511 of them bf16 behind
// a stride of 512, one value a load and store, 298; the bias alone of 16 x 2048 x 2048 fp32 51, 5.3 TB/s.
template <typename T, int E, bool VEC, bool SCORES>
__global__ void __launch_bounds__(kBiasThreads) bias_kernel(const __grid_constant__ BiasArgs a) {
  pdl_enter();
  __shared__ float lut[(32 * E + 32) * 33 / 32 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tiles = (a.keys + 32 * E - 1) / (32 * E);
  const int64_t k0 = blockIdx.x % tiles * (32 * E), h = blockIdx.y;
  const int rows = 4 * a.row_groups;
  const int64_t q0 = blockIdx.x / tiles * rows;
  // lut[i]: of key k0 + i - (rows - 1) against query q0
  const int64_t rel0 = k0 - (rows - 1) - q0 - a.offset;
  for (int i = threadIdx.x; i < 32 * E + rows - 1; i += kBiasThreads)
    lut[i + (i >> 5)] = load_any(a.table, a.table_dtype, bucket_of(a.buckets, rel0 + i) * a.heads + h);
  __syncthreads();
  const int group = warp % a.row_groups, first = warp / a.row_groups, step = kBiasWarps / a.row_groups;
  float bias[4][E];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = (VEC ? lane * E + e : lane + 32 * e) + rows - 1 - (group * 4 + r);
      bias[r][e] = lut[i + (i >> 5)];
    }
  const int64_t q = q0 + group * 4, k = k0 + (VEC ? lane * E : lane);
  const int64_t b0 = blockIdx.z * a.per_cta, b1 = min(b0 + a.per_cta, a.batch);
  const int left = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(4), a.queries - q)));
#pragma unroll 2
  for (int64_t b = b0 + first; b < b1; b += step) {
    const T* from = static_cast<const T*>(a.scores) + b * a.stride_b + h * a.stride_h + q * a.stride_q + k;
    T* to = static_cast<T*>(a.out) + ((b * a.heads + h) * a.queries + q) * a.keys + k;
    if constexpr (VEC) {
      uint4 x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (SCORES && r < left && k < a.keys) x[r] = __ldcs(reinterpret_cast<const uint4*>(from + r * a.stride_q));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r >= left || k >= a.keys) continue;
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = SCORES ? value_of<T>(x[r], e) + bias[r][e] : bias[r][e];
        put_piece(to + r * a.keys, v);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r >= left) break;
        T x[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (SCORES && k + 32 * e < a.keys) x[e] = from[r * a.stride_q + 32 * e];
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (k + 32 * e < a.keys) to[r * a.keys + 32 * e] = narrow<T>(SCORES ? widen(x[e]) + bias[r][e] : bias[r][e]);
      }
    }
  }
}

// Dense scores whose rows are no multiple of 16 bytes, or do not begin on one: the rows of a head
// and sequence as one run of values, in the pieces of 16 bytes that hold them, E values each, four
// a thread.  A piece may hold the end of a row and the next row's beginning, and the run's first
// and last are shared with other heads.  The biases of all diagonals that a CTA's kFlatPieces
// pieces meet are in shared memory, padded as above.  64 x 16 x 511 x 505 bf16 in 172 us, 6.2 TB/s,
// 511 x 513 fp32 333, 6.5 TB/s (one value a load and store 293 and 549; rows one by one in pieces
// shifted by each row's offset 236 and 412).
constexpr int kFlatPieces = 4 * kBiasThreads, kFlatMaxKeys = 8192;
constexpr int kFlatCtas = 5;  // of an SM, at the least
// Rows after the first that the pieces of a CTA may reach into, and the diagonals then.
__host__ __device__ __forceinline__ int flat_rows(int keys, int E) { return (keys - 1 + (kFlatPieces + 1) * E) / keys; }
__host__ __device__ __forceinline__ int flat_diagonals(int keys, int E) { return keys + flat_rows(keys, E) + E; }
template <typename T, int E, bool SCORES>
__global__ void __launch_bounds__(kBiasThreads, kFlatCtas) bias_flat_kernel(const __grid_constant__ BiasArgs a) {
  pdl_enter();
  extern __shared__ float lut[];
  const int keys = static_cast<int>(a.keys), rows = flat_rows(keys, E);
  const int64_t size = a.queries * a.keys, h = blockIdx.y, first = static_cast<int64_t>(blockIdx.x) * (kFlatPieces * E);
  const int64_t q0 = first / keys;
  const int k0 = static_cast<int>(first - q0 * keys);
  // lut[i]: of key i - rows against query q0
  for (int i = threadIdx.x; i < flat_diagonals(keys, E); i += kBiasThreads)
    lut[i + (i >> 5)] = load_any(a.table, a.table_dtype, bucket_of(a.buckets, i - rows - q0 - a.offset) * a.heads + h);
  __syncthreads();
  int key[4], row[4];  // of a piece's first value, were the run to begin on a piece
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = k0 + (threadIdx.x + j * kBiasThreads) * E;
    row[j] = at / keys;
    key[j] = at - row[j] * keys;
  }
  const int64_t b0 = blockIdx.z * a.per_cta, b1 = min(b0 + a.per_cta, a.batch);
  auto sweep = [&](auto edge) {  // (inside the run all pieces are whole)
    constexpr bool EDGE = decltype(edge)::value;
    for (int64_t b = b0; b < b1; ++b) {
      T* const to = static_cast<T*>(a.out) + (b * a.heads + h) * size;
      const T* const from = static_cast<const T*>(a.scores) + (b * a.heads + h) * size;
      const int before = static_cast<int>(reinterpret_cast<uintptr_t>(to) / sizeof(T) % E);  // others' values in the first piece
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = first + (threadIdx.x + j * kBiasThreads) * E - before;
        uint32_t whole = !EDGE || (at >= 0 && at + E <= size);
        if (EDGE) asm("" : "+r"(whole));  // (seen to be the store's condition, each load would wait for the one before: 13% more)
        if (SCORES && whole) x[j] = load_piece(reinterpret_cast<const uint4*>(from + at), from, from + size);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = first + (threadIdx.x + j * kBiasThreads) * E - before;
        if (EDGE && at >= size) break;
        int k = key[j] - before, i = k - row[j] + rows;
        while (k < 0) k += keys, i += keys + 1;  // (the key, in the row before)
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float add = lut[i + (i >> 5)];
          v[e] = SCORES ? value_of<T>(x[j], e) + add : add;
          const bool ends = ++k == keys;
          i += ends ? -keys : 1;
          if (ends) k = 0;
        }
        if (!EDGE || (at >= 0 && at + E <= size)) put_piece(to + at, v);
      }
    }
  };
  if (blockIdx.x > 0 && first + (kFlatPieces + 1) * E <= size) return sweep(std::false_type{});
  sweep(std::true_type{});
  // The run's first and last piece of every sequence, where others' values are in them, value by
  // value: those are not the caller's to have read, or another CTA's to write.
  for (int64_t item = threadIdx.x; item < (b1 - b0) * 2 * E; item += kBiasThreads) {
    const int64_t at_b = ((b0 + item / (2 * E)) * a.heads + h) * size;
    T* const to = static_cast<T*>(a.out) + at_b;
    const int before = static_cast<int>(reinterpret_cast<uintptr_t>(to) / sizeof(T) % E), e = static_cast<int>(item % E);
    const int64_t last = (size - 1 + before) / E, piece = item / E % 2 ? last : 0;
    const int64_t start = piece * E - before, at = start + e;
    const bool whole = start >= 0 && start + E <= size;
    if (whole || piece / kFlatPieces != blockIdx.x || (item / E % 2 && last == 0) || at < 0 || at >= size) continue;
    const int from_k0 = k0 + static_cast<int>(at - first);  // (negative: in the row before)
    const int r = from_k0 < 0 ? -((keys - 1 - from_k0) / keys) : from_k0 / keys;
    const int i = from_k0 - r * keys - r + rows;
    const float add = lut[i + (i >> 5)];
    to[at] = narrow<T>(SCORES ? widen(static_cast<const T*>(a.scores)[at_b + at]) + add : add);
  }
}

// ----------------------------------------------------------------------------- gradient

constexpr int kBiasRows = 256;  // at most, of a warp
constexpr int kBiasKeys = 256;  // of a warp at most, eight a lane
constexpr int kBiasGradCtas = 2;  // of an SM (3 with half as many rows on their way: 140 us against 99)

struct BiasGradArgs {
  const void *d, *end;  // its first value, and past its last
  int64_t stride_b, stride_h, stride_q;
  int64_t heads, queries, keys, offset;
  int rows, width;     // queries and keys of a unit
  int row_units, key_units, batch_units, per_unit;  // units of one worker and head; sequences of a unit
  int groups;          // CTAs of one worker and head, eight units each
  float* partials;     // [worker, head][group][bucket]; null: one group, the gradient is written
  int total;           // buckets of both directions
  Buckets buckets;
  int64_t off[kMaxK + 1];
};
struct BiasOut {
  void* grads[kMaxK];
  int dtype, accumulate;
  int64_t heads;
  int total, groups;
  const float* partials;
};

__device__ __forceinline__ void put_bucket(const BiasOut& o, int k, int64_t h, int bucket, float s) {
  const int64_t at = bucket * o.heads + h;
  if (o.accumulate) s += load_any(o.grads[k], o.dtype, at);
  store_any(o.grads[k], o.dtype, at, s);
}

// A bucket's sum runs over whole diagonals.  A warp has a unit: 256 neighbouring keys, eight a
// lane, up to 256 queries, some sequences of one worker.  It goes down the queries with the
// running sums of 256 diagonals in registers: from one query to the next a diagonal moves on
// by one key, so the sums move by one register (or lane), the last lane's leaves the window and
// a new one begins.  The diagonals' sums end in shared memory and are added up per bucket, in
// an order that depends on the sizes alone.  One read of the gradients, an addition a value: bound
// by bytes, 64 x 16 x 512 x 512 of 16 workers bf16 in 92 us, 5.9 TB/s, fp32 168, 6.4 TB/s.  511 x 513
// of them bf16 in 161 (loaded value by value, 32 keys apart a lane: 763); one sequence each of 4
// workers of 16 x 2048 x 2048 in 112 us, 4.8 TB/s.
// VEC: all rows of keys begin on 16-byte boundaries; else the pieces of 16 bytes that hold them do,
// and the values move over by less than a lane.  Pieces may hold values beside the unit's, which
// are masked.  EDGE: some pieces reach beyond the first or last value of all, whose rows are looked
// for in the units that have any (512 x 513 of them behind a stride of 520 bf16 121 us a pass, 113 without the
// checks; 511 x 513 dense the same; a kernel of its own, since aligned ones of 2048 x 2048 took 115 in it, not 109).
template <typename T, bool VEC, bool EDGE>
__global__ void __launch_bounds__(kBiasThreads, kBiasGradCtas) bias_grad_kernel(const __grid_constant__ BiasGradArgs a, const __grid_constant__ BiasOut o) {
  pdl_enter();
  __shared__ float diagonals[kBiasWarps][kBiasRows + kBiasKeys];
  __shared__ float sums[kBiasWarps][kMaxBuckets];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t h = blockIdx.y;
  const int k = blockIdx.z;
  const int units = a.row_units * a.key_units * a.batch_units;
  const int unit = blockIdx.x * kBiasWarps + warp;
  float* mine = diagonals[warp];
  for (int b = lane; b < a.total; b += 32) sums[warp][b] = 0.f;
  const int64_t b0 = a.off[k] + static_cast<int64_t>(unit / (a.row_units * a.key_units)) * a.per_unit;
  const int nb = unit < units ? static_cast<int>(max(static_cast<int64_t>(0), min(a.off[k + 1] - b0, static_cast<int64_t>(a.per_unit)))) : 0;
  if (nb > 0) {
    const int r = unit % (a.row_units * a.key_units);
    const int64_t q0 = static_cast<int64_t>(r / a.key_units) * a.rows, k0 = static_cast<int64_t>(r % a.key_units) * a.width;
    const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), a.queries - q0));
    const int width = static_cast<int>(min(static_cast<int64_t>(a.width), a.keys - k0));
    const T* p = static_cast<const T*>(a.d) + b0 * a.stride_b + h * a.stride_h + q0 * a.stride_q + k0;
    // Rows of keys come in groups, two of them on their way: some sequences' of one query, or, where
    // there are few sequences (FEW), of some queries.
    constexpr int kGroup = sizeof(T) == 2 ? 4 : 2, kWords = sizeof(T) * 2;
    struct Group {
      uint32_t row[kGroup][kWords];
      int off[VEC ? 1 : kGroup];  // values of a row's first 16 bytes that are before its keys
    } ahead[2];
    const int mine_left = max(0, min(8, width - lane * 8));
    uint32_t mask[kWords];  // of the lane's values that exist
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int left = sizeof(T) == 4 ? mine_left - i : mine_left - 2 * i;
      mask[i] = left <= 0 ? 0u : sizeof(T) == 2 && left == 1 ? 0xFFFFu : 0xFFFFFFFFu;
    }
    const T *const begin = static_cast<const T*>(a.d), *const end = static_cast<const T*>(a.end);
    // where all pieces of a row are whole
    const T* const whole_from = reinterpret_cast<const T*>((reinterpret_cast<uintptr_t>(begin) + 15) & ~uintptr_t(15));
    const T* const whole_to = reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(end) & ~uintptr_t(15));
    // Pieces of 16 bytes that hold a value of the row (and may hold others').
    auto load = [&](Group& g, int s, const T* at, bool on) {
      int off = 0;
      if constexpr (!VEC) g.off[s] = off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15) / static_cast<int>(sizeof(T));
      const uint4* from = reinterpret_cast<const uint4*>(at - off) + lane * (kWords / 4);
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const bool there = on && lane * 8 + i * (16 / static_cast<int>(sizeof(T))) - off < width;
        const uint4 x = there ? load_piece(from + i, begin, end) : make_uint4(0u, 0u, 0u, 0u);
        g.row[s][4 * i] = x.x, g.row[s][4 * i + 1] = x.y, g.row[s][4 * i + 2] = x.z, g.row[s][4 * i + 3] = x.w;
      }
    };
    // The same of a row that may reach into the first or last piece of all.
    auto load_beyond = [&](Group& g, int s, const T* at, bool on) {
      if (at >= whole_from && at + width <= whole_to) return load(g, s, at, on);
      int off = 0;
      if constexpr (!VEC) g.off[s] = off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15) / static_cast<int>(sizeof(T));
      const uint4* from = reinterpret_cast<const uint4*>(at - off) + lane * (kWords / 4);
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const bool there = on && lane * 8 + i * (16 / static_cast<int>(sizeof(T))) - off < width;
        const uint4 x = there ? load_edge(from + i, begin, end) : make_uint4(0u, 0u, 0u, 0u);
        g.row[s][4 * i] = x.x, g.row[s][4 * i + 1] = x.y, g.row[s][4 * i + 2] = x.z, g.row[s][4 * i + 3] = x.w;
      }
    };
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    auto add = [&](const Group& g, int s) {
      uint32_t w[kWords];
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = g.row[s][i];
      } else {
        // the lane's words and the next lane's, moved over by `off` values (the same for the warp):
        // by two words, by one, by half
        constexpr int kMore = sizeof(T) == 4 ? 3 : 4;
        const int off = g.off[s], words = sizeof(T) == 4 ? off : off >> 1;
        uint32_t x[kWords + kMore];
#pragma unroll
        for (int i = 0; i < kWords; ++i) x[i] = g.row[s][i];
#pragma unroll
        for (int i = 0; i < kMore; ++i) x[kWords + i] = __shfl_down_sync(0xFFFFFFFFu, x[i], 1);
#pragma unroll
        for (int i = 0; i < kWords + kMore - 2; ++i) x[i] = words & 2 ? x[i + 2] : x[i];
#pragma unroll
        for (int i = 0; i < kWords + kMore - 3; ++i) x[i] = words & 1 ? x[i + 1] : x[i];
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = sizeof(T) == 4 ? x[i] : __funnelshift_r(x[i], x[i + 1], off & 1 ? 16 : 0);
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] &= mask[i];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        F2 x;
        if constexpr (sizeof(T) == 4) x = f2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]));
        else x = f2(__uint_as_float(w[e >> 1] << 16), __uint_as_float(w[e >> 1] & 0xFFFF0000u));
        const float2 y = parts(add2(f2(acc[e], acc[e + 1]), x));
        acc[e] = y.x;
        acc[e + 1] = y.y;
      }
    };
    int done = 0;  // queries
    // On to the next query: a slot is where a diagonal's key stands in the window at the last one.
    auto next_query = [&] {
      if (++done == rows) return;
      if (lane == 31) mine[kBiasKeys - 1 + rows - done] = acc[7];
      const float in = __shfl_up_sync(0xFFFFFFFFu, acc[7], 1);
#pragma unroll
      for (int e = 7; e > 0; --e) acc[e] = acc[e - 1];
      acc[0] = lane == 0 ? 0.f : in;
    };
    auto sweep = [&](auto few, auto edge) {
      constexpr bool FEW = decltype(few)::value;
      const int per_query = (nb + kGroup - 1) / kGroup, all = rows * nb;
      const int count = FEW ? (all + kGroup - 1) / kGroup : rows * per_query;
      const T* at = p;
      int ready = 0, row = 0, at_b = 0;  // groups fetched; the next row's (FEW), and sequence
      auto fetch = [&](Group& g) {
        if (ready >= count) return;
        ++ready;
#pragma unroll
        for (int s = 0; s < kGroup; ++s) {
          if constexpr (FEW) {
            if constexpr (decltype(edge)::value) load_beyond(g, s, at, row < all);
            else load(g, s, at, row < all);
            ++row;
            if (++at_b == nb) at_b = 0, at = p += a.stride_q;
            else at += a.stride_b;
          } else {
            if constexpr (decltype(edge)::value) load_beyond(g, s, at + s * a.stride_b, at_b + s < nb);
            else load(g, s, at + s * a.stride_b, at_b + s < nb);
          }
        }
        if constexpr (!FEW) {
          at_b += kGroup;
          at += kGroup * a.stride_b;
          if (at_b >= nb) at_b = 0, at = p += a.stride_q;
        }
      };
      int b = 0, taken = 0;  // of the query's sequences (groups of them); rows (FEW)
      auto take = [&](const Group& g) {
#pragma unroll
        for (int s = 0; s < kGroup; ++s) {
          if (FEW && taken == all) break;
          add(g, s);
          if constexpr (FEW) {
            ++taken;
            if (++b == nb) b = 0, next_query();
          }
        }
        if constexpr (!FEW) {
          if (++b == per_query) b = 0, next_query();
        }
      };
      fetch(ahead[0]);
      fetch(ahead[1]);
      for (int i = 0; i < count; i += 2) {
        Group now = ahead[0];
        fetch(ahead[0]);
        take(now);
        if (i + 1 >= count) break;
        now = ahead[1];
        fetch(ahead[1]);
        take(now);
      }
    };
    // (strides are not negative: the unit's first row begins first, its last ends last)
    if (EDGE && (p < whole_from || p + (nb - 1) * a.stride_b + (rows - 1) * a.stride_q + width > whole_to)) {
      if (nb <= 2) sweep(std::true_type{}, std::bool_constant<EDGE>{});
      else sweep(std::false_type{}, std::bool_constant<EDGE>{});
    } else {
      if (nb <= 2) sweep(std::true_type{}, std::false_type{});
      else sweep(std::false_type{}, std::false_type{});
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) mine[lane * 8 + e] = acc[e];
    __syncwarp();
    // mine[i]: key k0 + i against the unit's last query
    const int64_t rel0 = k0 - (q0 + rows - 1) - a.offset;
    const int slots = kBiasKeys + rows - 1;
    const int n = a.buckets.n;
    auto range = [&](int bucket, int& lo, int& hi) {  // slots of a bucket
      const bool ahead = bucket >= n;
      const int j = ahead ? bucket - n : bucket;
      const int64_t near = a.buckets.border[j], far = j + 1 < n ? a.buckets.border[j + 1] : INT64_MAX;
      int64_t first, last;  // of the relative positions, and one past it
      if (ahead) first = max(near, static_cast<int64_t>(1)), last = far;
      else first = far == INT64_MAX ? INT64_MIN : 1 - far, last = 1 - near;
      if (!a.buckets.both && j == 0) last = INT64_MAX;
      auto slot = [&](int64_t rel) {
        return rel <= rel0 ? 0 : rel >= rel0 + slots ? slots : static_cast<int>(rel - rel0);
      };
      lo = slot(first);
      hi = slot(last);
    };
    // short buckets by a lane each, long ones by the warp
    constexpr int kShort = 16;
    for (int c = 0; c < a.total; c += 32) {
      int lo = 0, hi = 0;
      if (c + lane < a.total) range(c + lane, lo, hi);
      float s = 0.f;
      if (hi - lo <= kShort)
        for (int i = lo; i < hi; ++i) s += mine[i];
      unsigned longs = __ballot_sync(0xFFFFFFFFu, hi - lo > kShort);
      for (; longs; longs &= longs - 1) {
        const int from = __ffs(longs) - 1;
        const int l = __shfl_sync(0xFFFFFFFFu, lo, from), e = __shfl_sync(0xFFFFFFFFu, hi, from);
        float v = 0.f;
        for (int i = l + lane; i < e; i += 32) v += mine[i];
        v = warp_sum(v);
        if (lane == from) s = v;
      }
      if (c + lane < a.total) sums[warp][c + lane] = s;
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.total; b += kBiasThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBiasWarps; ++w) s += sums[w][b];
    if (a.partials == nullptr) put_bucket(o, k, h, b, s);
    else a.partials[((k * a.heads + h) * a.groups + blockIdx.x) * a.total + b] = s;
  }
}

// Adds the CTAs' sums of one worker and head, in their order within eight rows of them.
__global__ void __launch_bounds__(256) bias_join_kernel(const __grid_constant__ BiasOut o) {
  pdl_enter();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = blockIdx.z;
  const int64_t h = blockIdx.y;
  const int b = blockIdx.x * 32 + lane;
  const float* p = o.partials + (k * o.heads + h) * o.groups * static_cast<int64_t>(o.total);
  float s = 0.f;
  if (b < o.total) {
#pragma unroll 4
    for (int g = warp; g < o.groups; g += 8) s += p[static_cast<int64_t>(g) * o.total + b];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp > 0 || b >= o.total) return;
#pragma unroll
  for (int j = 1; j < 8; ++j) s += red[j][lane];
  put_bucket(o, k, h, b, s);
}

// ----------------------------------------------------------------------------- host side

// base^power times what is there, in whole numbers of any length.
void multiply(std::vector<uint32_t>& x, uint64_t by) {
  const uint64_t parts[2] = {by & 0xFFFFFFFFu, by >> 32};
  std::vector<uint32_t> out(x.size() + 3, 0u);
  for (int h = 0; h < 2; ++h) {
    uint64_t carry = 0;
    for (size_t i = 0; i < x.size() || carry; ++i) {
      const uint64_t v = out[i + h] + carry + (i < x.size() ? parts[h] * x[i] : 0);
      out[i + h] = static_cast<uint32_t>(v);
      carry = v >> 32;
    }
  }
  while (out.size() > 1 && out.back() == 0) out.pop_back();
  x.swap(out);
}
std::vector<uint32_t> power_product(uint64_t a, int i, uint64_t b, int j) {  // a^i b^j
  std::vector<uint32_t> x(1, 1u);
  for (; i > 0; --i) multiply(x, a);
  for (; j > 0; --j) multiply(x, b);
  return x;
}
bool at_least(const std::vector<uint32_t>& a, const std::vector<uint32_t>& b) {
  if (a.size() != b.size()) return a.size() > b.size();
  for (size_t i = a.size(); i-- > 0;)
    if (a[i] != b[i]) return a[i] > b[i];
  return true;
}

// a^i b^j <= d^k, in 128 bits where they hold both sides (in a vector's digits a call with 32
// buckets up to 128 took 3 us longer, up to 4096 in one direction 10).
bool product_at_most(uint64_t a, int i, uint64_t b, int j, uint64_t d, int k) {
  using Wide = unsigned __int128;
  auto times = [](Wide& x, uint64_t f, int n) {
    for (; n > 0 && x <= ~Wide(0) / f; --n) x *= f;
    return n == 0;
  };
  Wide left = 1, right = 1;
  if (times(left, a, i) && times(left, b, j) && times(right, d, k)) return left <= right;
  return at_least(power_product(d, k, 1, 0), power_product(a, i, b, j));
}

// The borders of one direction.  Bucket e + i begins at the smallest d with
// (n - e) ln(d / e) >= i ln(D / e): where d is not plainly on one side, (d / e)^(n - e) is
// compared with (D / e)^i in whole numbers: d^(n - e) with D^i e^(n - e - i), exponents over their
// greatest common divisor.
void borders(Buckets& b, int64_t max_distance) {
  const int e = b.n / 2, p = b.n - e;
  for (int j = 0; j <= e; ++j) b.border[j] = j;
  for (int i = 1; i < p; ++i) {
    const double x = e * std::exp(std::log(static_cast<double>(max_distance) / e) * i / p);
    int64_t d = std::llround(x);
    if (std::fabs(x - static_cast<double>(d)) < 1e-12 * x) {  // (x is off by 2e-14 at most)
      const int g = std::gcd(i, p);
      if (!product_at_most(max_distance, i / g, e, (p - i) / g, d, p / g)) ++d;
    } else {
      d = static_cast<int64_t>(std::ceil(x));
    }
    b.border[e + i] = d;
  }
}

// Fills the buckets of a call; what is wrong with it.
adasum_status_t make_buckets(Buckets& b, int buckets, int both, int64_t max_distance) {
  if (buckets > kMaxBuckets || max_distance > INT32_MAX) return ADASUM_ERR_UNSUPPORTED;
  if (buckets < 1 || (both && buckets % 2)) return ADASUM_ERR_INVALID_ARG;
  b.both = both != 0;
  b.n = both ? buckets / 2 : buckets;
  if (b.n < 2 || max_distance <= b.n / 2) return ADASUM_ERR_INVALID_ARG;
  try {
    borders(b, max_distance);
  } catch (...) {  // (out of host memory)
    return ADASUM_ERR_NO_MEMORY;
  }
  return ADASUM_OK;
}

adasum_status_t check_sizes(int64_t heads, int64_t batch, int64_t queries, int64_t keys, int64_t offset) {
  if (heads < 0 || batch < 0 || queries < 0 || keys < 0) return ADASUM_ERR_INVALID_ARG;
  constexpr int64_t kFar = int64_t(1) << 61;
  if (heads > 65535 || queries > INT32_MAX || keys > INT32_MAX || offset > kFar || offset < -kFar) return ADASUM_ERR_UNSUPPORTED;
  if (batch > 0 && heads > 0 && queries > 0 && keys > 0 && batch > INT64_MAX / 16 / heads / queries / keys)
    return ADASUM_ERR_UNSUPPORTED;
  return ADASUM_OK;
}
// Elements that strided scores reach over; -1: strides that overlap or cannot be addressed.
int64_t span_of(int64_t batch, int64_t heads, int64_t queries, int64_t keys, int64_t sb, int64_t sh, int64_t sq) {
  if ((queries > 1 && sq < keys) || (heads > 1 && sh < 0) || (batch > 1 && sb < 0)) return -1;
  auto far = [](int64_t count, int64_t stride) { return count > 1 && stride > INT64_MAX / 64 / count; };
  if (far(batch, sb) || far(heads, sh) || far(queries, sq)) return -1;
  return (batch > 1 ? (batch - 1) * sb : 0) + (heads > 1 ? (heads - 1) * sh : 0) + (queries > 1 ? (queries - 1) * sq : 0) + keys;
}

template <typename T, bool SCORES>
int launch_bias(const BiasArgs& a, bool vec, bool flat, dim3 grid, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  if (flat) {
    const size_t smem = (flat_diagonals(static_cast<int>(a.keys), E) * 33 / 32 + 1) * sizeof(float);  // (below 35 KB)
    return launch_pdl(bias_flat_kernel<T, E, SCORES>, grid, dim3(kBiasThreads), smem, stream, a);
  }
  return launch_pdl(vec ? bias_kernel<T, E, true, SCORES> : bias_kernel<T, E, false, SCORES>, grid, dim3(kBiasThreads), 0, stream, a);
}

template <typename T>
int launch_bias_grad(const BiasGradArgs& a, const BiasOut& o, bool vec, bool edge, dim3 grid, cudaStream_t stream) {
  return launch_pdl(vec ? (edge ? bias_grad_kernel<T, true, true> : bias_grad_kernel<T, true, false>)
                        : (edge ? bias_grad_kernel<T, false, true> : bias_grad_kernel<T, false, false>),
                    grid, dim3(kBiasThreads), 0, stream, a, o);
}

// Units of one worker and head, and how they are dealt.
struct GradPlan {
  int rows, width, row_units, key_units, batch_units, per_unit, groups;
};
GradPlan plan_grad(const int64_t* offs, int K, int64_t heads, int64_t queries, int64_t keys, bool vec) {
  GradPlan g = {};
  int64_t most = 1;
  for (int k = 0; k < K; ++k) most = std::max(most, offs[k + 1] - offs[k]);
  // At most 16 sequences a unit, so that no running sum gets long; keys in equal parts.  Then
  // queries, 8 to 256: the number for which the waves of CTAs take least, a unit costing its
  // groups of rows and about 24 groups' time for its diagonals' sums.
  g.per_unit = static_cast<int>(std::min<int64_t>(most, 16));
  const int64_t batch_units = (most + g.per_unit - 1) / g.per_unit, widest = vec ? kBiasKeys : kBiasKeys - 8,
                key_units = (keys + widest - 1) / widest;  // (room for pieces that begin before the keys)
  g.width = static_cast<int>(((keys + key_units - 1) / key_units + 7) / 8 * 8);
  const double per_query = g.per_unit <= 2 ? g.per_unit / 4.0 : (g.per_unit + 3) / 4;
  const int64_t slots = static_cast<int64_t>(kBiasGradCtas) * sm_count();
  double least = 1e300;
  for (int rows = kBiasRows; rows >= 8; rows /= 2) {
    const int64_t units = (queries + rows - 1) / rows * key_units * batch_units;
    const int64_t ctas = K * heads * ((units + kBiasWarps - 1) / kBiasWarps);
    const double cost = static_cast<double>((ctas + slots - 1) / slots) * (static_cast<double>(std::min<int64_t>(rows, queries)) * per_query + 24.0);
    if (cost < least) least = cost, g.rows = rows;
  }
  g.row_units = static_cast<int>((queries + g.rows - 1) / g.rows);
  g.key_units = static_cast<int>(key_units);
  g.batch_units = static_cast<int>(std::min<int64_t>(batch_units, INT32_MAX));
  const int64_t units = static_cast<int64_t>(g.row_units) * key_units * batch_units;
  g.groups = units > (int64_t(1) << 30) ? -1 : static_cast<int>((units + kBiasWarps - 1) / kBiasWarps);
  return g;
}

}  // namespace

int take_bias_error() {
  int h = 0;
#ifdef ADASUM_BOUNDS_CHECK
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&h, g_status, sizeof h) != cudaSuccess) return -1;
  if (h != 0 && cudaMemcpyToSymbol(g_status, &zero, sizeof zero) != cudaSuccess) return -1;
#endif
  return h;
}

}  // namespace adasum

using namespace adasum;

extern "C" {

adasum_status_t adasum_relative_position_bias(const void* table, int buckets, int64_t heads, adasum_dtype_t table_dtype,
                                              int bidirectional, int64_t max_distance, int64_t offset, int64_t queries,
                                              int64_t keys, const void* scores, int64_t batch, int64_t stride_b,
                                              int64_t stride_h, int64_t stride_q, adasum_dtype_t dtype, void* out,
                                              adasum_stream_t stream_) {
  EntryScope scope("adasum_relative_position_bias");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!valid_dtype(table_dtype) || (scores != nullptr && !valid_dtype(dtype))) return ADASUM_ERR_INVALID_ARG;
  if (scores == nullptr) batch = 1, dtype = table_dtype;
  if (adasum_status_t st = check_sizes(heads, batch, queries, keys, offset)) return st;
  BiasArgs a = {};
  if (adasum_status_t st = make_buckets(a.buckets, buckets, bidirectional, max_distance)) return st;
  if (heads == 0 || batch == 0 || queries == 0 || keys == 0) return ADASUM_OK;
  if (table == nullptr || out == nullptr) return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype), te = dtype_bytes(table_dtype), n = heads * queries * keys;
  const int64_t span = scores ? span_of(batch, heads, queries, keys, stride_b, stride_h, stride_q) : 0;
  if (span < 0) return ADASUM_ERR_INVALID_ARG;
  const bool dense = (queries == 1 || stride_q == keys) && (heads == 1 || stride_h == queries * keys) && (batch == 1 || stride_b == n);
  BufferSet set;
  set.read(table, buckets * heads * te, te);
  if (scores != nullptr && !(scores == out && dense)) set.read(scores, span * e, e);
  set.write(out, batch * n * e, e);
  if (adasum_status_t st = set.check()) return st;
  a.table = table;
  a.table_dtype = table_dtype;
  a.heads = heads;
  a.batch = batch;
  a.queries = queries;
  a.keys = keys;
  a.offset = offset;
  a.scores = scores;
  a.stride_b = stride_b;
  a.stride_h = stride_h;
  a.stride_q = stride_q;
  a.out = out;
  a.row_groups = queries > 16 ? 8 : queries > 8 ? 4 : queries > 4 ? 2 : 1;
  const bool vec = is_aligned(out, 16) && keys * e % 16 == 0 &&
                   (scores == nullptr || (is_aligned(scores, 16) && (queries == 1 || stride_q * e % 16 == 0) &&
                                          (heads == 1 || stride_h * e % 16 == 0) && (batch == 1 || stride_b * e % 16 == 0)));
  // (the biases of a row's diagonals have to serve enough values: bf16, 16 heads of 2047 x 2047 89 us
  // and value by value 97, four sequences of them 180 and 269; one of 4 x 4095 x 8191 450 and 183)
  const bool flat = !vec && keys <= std::min<int64_t>(kFlatMaxKeys, 2048 * batch) &&
                    (scores == nullptr || (dense && (reinterpret_cast<uintptr_t>(scores) - reinterpret_cast<uintptr_t>(out)) % 16 == 0));
  const int64_t piece = 16 / e, width = 32 * piece, tiles = (keys + width - 1) / width, rows = 4 * a.row_groups;
  const int64_t x = flat ? (queries * keys + piece - 1 + kFlatPieces * piece - 1) / (kFlatPieces * piece)
                         : tiles * ((queries + rows - 1) / rows);
  const int64_t step = flat ? 1 : kBiasWarps / a.row_groups;
  if (x > INT32_MAX) return ADASUM_ERR_UNSUPPORTED;
  // sequences of a CTA: as many as leave eight CTAs an SM, so that the biases serve many of them
  int64_t parts = std::max<int64_t>(1, std::min<int64_t>((batch + step - 1) / step, static_cast<int64_t>(8) * sm_count() / (x * heads)));
  // (or up to eight times as many, if their waves take less, a CTA's biases taking about two sequences' time:
  // 64 x 16 x 512 x 513 bf16 in four parts, 2.8 waves, 167 us a pass, in two, 1.4 waves, 189; where there
  // are many parts one more or less changes little)
  if (flat && parts < 8) {
    const int64_t slots = static_cast<int64_t>(kFlatCtas) * sm_count(), base = parts;
    auto time = [&](int64_t p) { return (x * heads * p + slots - 1) / slots * ((batch + p - 1) / p + 2); };
    for (int64_t p = base + 1; p <= std::min(batch, 8 * base); ++p)
      if (time(p) < time(parts)) parts = p;
  }
  parts = std::max(parts, (batch + (int64_t(1) << 16) - 1) >> 16);
  a.per_cta = (batch + parts - 1) / parts;
  parts = (batch + a.per_cta - 1) / a.per_cta;
  if (parts > 65535) return ADASUM_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(heads), static_cast<unsigned>(parts));
  return counted_launch(stream, scores ? "position_bias_add" : "position_bias", static_cast<double>(batch) * n * e * (scores ? 2 : 1), [&] {
    if (dtype == ADASUM_BF16) return scores ? launch_bias<bf16, true>(a, vec, flat, grid, stream) : launch_bias<bf16, false>(a, vec, flat, grid, stream);
    return scores ? launch_bias<float, true>(a, vec, flat, grid, stream) : launch_bias<float, false>(a, vec, flat, grid, stream);
  });
}

int64_t adasum_relative_position_bias_backward_scratch_bytes(const int64_t* worker_offsets, int K, int64_t heads,
                                                             int64_t queries, int64_t keys, int buckets) {
  if (check_worker_offsets(worker_offsets, K) || buckets < 1 || buckets > kMaxBuckets) return 0;
  if (check_sizes(heads, worker_offsets[K], queries, keys, 0) || heads == 0 || worker_offsets[K] == 0 || queries == 0 || keys == 0) return 0;
  // (whatever the rows' alignment turns out to be)
  const int64_t groups = std::max(plan_grad(worker_offsets, K, heads, queries, keys, true).groups,
                                  plan_grad(worker_offsets, K, heads, queries, keys, false).groups);
  return groups <= 1 ? 0 : (static_cast<int64_t>(K) * heads * groups * buckets * 4 + 255) / 256 * 256;
}

adasum_status_t adasum_relative_position_bias_backward(const void* grad_scores, int64_t heads, int64_t queries, int64_t keys,
                                                       int64_t stride_b, int64_t stride_h, int64_t stride_q,
                                                       adasum_dtype_t dtype, int buckets, int bidirectional,
                                                       int64_t max_distance, int64_t offset, const int64_t* worker_offsets,
                                                       int K, void* const* grads, adasum_dtype_t grad_dtype, int accumulate,
                                                       void* scratch, int64_t scratch_bytes, adasum_stream_t stream_) {
  EntryScope scope("adasum_relative_position_bias_backward");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (adasum_status_t st = check_worker_offsets(worker_offsets, K)) return st;
  if (!valid_dtype(dtype) || !valid_dtype(grad_dtype) || grads == nullptr) return ADASUM_ERR_INVALID_ARG;
  const int64_t batch = worker_offsets[K];
  if (adasum_status_t st = check_sizes(heads, batch, queries, keys, offset)) return st;
  BiasGradArgs a = {};
  BiasOut o = {};
  if (adasum_status_t st = make_buckets(a.buckets, buckets, bidirectional, max_distance)) return st;
  if (heads == 0) return ADASUM_OK;
  const int64_t e = dtype_bytes(dtype), ge = dtype_bytes(grad_dtype);
  const bool some = batch > 0 && queries > 0 && keys > 0;
  const int64_t span = some ? span_of(batch, heads, queries, keys, stride_b, stride_h, stride_q) : 0;
  if (span < 0 || (some && grad_scores == nullptr)) return ADASUM_ERR_INVALID_ARG;
  const int64_t need = adasum_relative_position_bias_backward_scratch_bytes(worker_offsets, K, heads, queries, keys, buckets);
  if (need > 0 && (scratch == nullptr || scratch_bytes < need || !is_aligned(scratch, 256))) return ADASUM_ERR_INVALID_ARG;
  BufferSet set;
  set.read(grad_scores, span * e, e);
  if (need > 0) set.write(scratch, need, 256);
  for (int k = 0; k < K; ++k) {
    if (grads[k] == nullptr) return ADASUM_ERR_INVALID_ARG;
    set.write(o.grads[k] = grads[k], buckets * heads * ge, ge);
  }
  if (adasum_status_t st = set.check()) return st;
  if (!some && accumulate) return ADASUM_OK;
  const bool vec = is_aligned(grad_scores, 16) && (queries <= 1 || stride_q * e % 16 == 0) && (heads == 1 || stride_h * e % 16 == 0) &&
                   (batch <= 1 || stride_b * e % 16 == 0);
  const GradPlan g = plan_grad(worker_offsets, K, heads, some ? queries : 1, some ? keys : 1, vec);
  if (g.groups < 0) return ADASUM_ERR_UNSUPPORTED;
  a.d = grad_scores;
  a.end = static_cast<const char*>(grad_scores) + span * e;
  a.stride_b = stride_b;
  a.stride_h = stride_h;
  a.stride_q = stride_q;
  a.heads = heads;
  a.queries = queries;
  a.keys = keys;
  a.offset = offset;
  a.rows = g.rows;
  a.width = g.width;
  a.row_units = g.row_units;
  a.key_units = g.key_units;
  a.batch_units = some ? g.batch_units : 0;  // (no units: every sum is zero)
  a.per_unit = g.per_unit;
  a.groups = some ? g.groups : 1;
  a.partials = a.groups > 1 ? static_cast<float*>(scratch) : nullptr;
  a.total = buckets;
  std::copy(worker_offsets, worker_offsets + K + 1, a.off);
  o.dtype = grad_dtype;
  o.accumulate = accumulate != 0;
  o.heads = heads;
  o.total = buckets;
  o.groups = a.groups;
  o.partials = a.partials;
  const dim3 grid(static_cast<unsigned>(a.groups), static_cast<unsigned>(heads), static_cast<unsigned>(K));
  const bool edge = some && !(is_aligned(a.d, 16) && is_aligned(a.end, 16));
  adasum_status_t st = counted_launch(stream, "position_bias_grad", static_cast<double>(batch) * heads * queries * keys * e, [&] {
    return dtype == ADASUM_BF16 ? launch_bias_grad<bf16>(a, o, vec, edge, grid, stream) : launch_bias_grad<float>(a, o, vec, edge, grid, stream);
  });
  if (st || a.partials == nullptr) return st;
  return counted_launch(stream, "position_bias_join", 0.0, [&] {
    return launch_pdl(bias_join_kernel, dim3(static_cast<unsigned>((buckets + 31) / 32), static_cast<unsigned>(heads), static_cast<unsigned>(K)),
                      dim3(256), 0, stream, o);
  });
}

}  // extern "C"
