// train_embedding.cu -- token embeddings and the table's gradient, per worker.
//
// The gradient of a table row is the sum of the rows of grad_out whose token it is.  The
// tokens of each worker are sorted (stably, so that equal tokens stay in their order) and
// the sorted list is cut into chunks of equal length, whatever the tokens: one warp sums
// the runs of equal tokens inside one chunk over 256 columns.  A run that lies inside its
// chunk goes straight to the gradient; the pieces of a run that crosses chunks go to
// scratch memory and are joined in order by a last kernel.  So a token that makes up most
// of the batch costs no more than any other, and every sum has a fixed order.
#include "adasum_host.h"
#include "adasum_launch.h"
#include "adasum_train.cuh"

namespace adasum {
namespace {

constexpr int kEmbThreads = 256;
constexpr int kEmbWarps = kEmbThreads / 32;
constexpr int kSlice = 256;  // columns of a warp

struct LookupArgs {
  const void* table;
  int64_t num_rows, cols;
  const void* tokens;
  int token_bytes;
  int64_t n;
  float scale;
  void* out;
  int parts;  // pieces of kLookupVecs * 256 columns per row
};

__device__ __forceinline__ int64_t load_token(const void* tokens, int bytes, int64_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

// One warp copies up to 1024 columns of one token's row, four 16-byte vectors per lane in
// flight; bound by the output's bytes.
constexpr int kLookupVecs = 4;
template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kEmbThreads) lookup_kernel(const LookupArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * kEmbWarps + (threadIdx.x >> 5);
  const uint32_t i = w / static_cast<uint32_t>(a.parts);
  if (i >= a.n) return;
  const int64_t c0 = static_cast<int64_t>(w - i * a.parts) * (kLookupVecs * kSlice);
  const int64_t t = load_token(a.tokens, a.token_bytes, i);
  const bool there = t >= 0 && t < a.num_rows;
  const T* src = static_cast<const T*>(a.table) + (there ? t : 0) * a.cols + c0;
  T* dst = static_cast<T*>(a.out) + static_cast<int64_t>(i) * a.cols + c0;
  const int64_t left = a.cols - c0;
  Raw8<T> r[kLookupVecs];
#pragma unroll
  for (int j = 0; j < kLookupVecs; ++j) r[j] = load8<T, LAYOUT, true>(src + j * kSlice, there ? left - j * kSlice : 0, lane);
#pragma unroll
  for (int j = 0; j < kLookupVecs; ++j) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = there ? a.scale * raw_value<T>(r[j], e) : 0.f;
    store8<T, LAYOUT>(dst + j * kSlice, left - j * kSlice, lane, v);
  }
}

// ------------------------------------------------------------------- the table's gradient

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 8;                             // tokens per thread
constexpr int kSortMost = kSortThreads * kSortItems;      // tokens one CTA sorts by itself
constexpr int kDigits = 256;
constexpr int kMostPasses = 4;

// Tokens per chunk: 32, or 8 when that leaves too few warps to cover the memory's latency
// (a warp reads its chunk's rows eight at a time).
int chunk_tokens(int64_t n, int64_t cols) {
  const int64_t slices = (cols + kSlice - 1) / kSlice;
  return n * slices >= 32 * 4096 ? 32 : 8;
}
int64_t chunk_bound(int64_t n, int64_t cols, int K) { return n / chunk_tokens(n, cols) + K; }
int64_t tile_bound(int64_t n, int K) { return n / kSortMost + K; }

// Regions of the scratch memory.
struct Scratch {
  int64_t keys[2], pos[2], hist, count, list, partials, total;
  Scratch(int64_t n, int64_t cols, int K) {
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
      const int64_t here = at;
      at += (bytes + 255) / 256 * 256;
      return here;
    };
    for (int i = 0; i < 2; ++i) keys[i] = take(4 * n);
    for (int i = 0; i < 2; ++i) pos[i] = take(4 * n);
    hist = take(4 * kMostPasses * kDigits * tile_bound(n, K));
    count = take(4);
    list = take(4 * chunk_bound(n, cols, K));
    partials = take(8 * cols * chunk_bound(n, cols, K));
    total = at;
  }
};

struct SortArgs {
  const void* tokens;
  int token_bytes;
  int num_rows;
  int64_t padding_idx;
  int K;
  int bits;            // per digit
  int shift;           // of this pass
  int pass, passes;
  int ntiles;          // of the multi-CTA sort
  const int *keys_in, *pos_in;   // null in the first pass: the tokens
  int *keys, *pos;
  int* hist;           // [passes][ntiles][kDigits]
  int* join_count;
  void* fill[kMaxK];   // gradients to be zeroed
  int64_t fill_bytes;  // of each (0: accumulate)
  int fill_ctas;
  int64_t off[kMaxK + 1];
  int tile_off[kMaxK + 1];  // first tile of a worker (multi-CTA sort)
};

struct TableGradArgs {
  const void* dy;
  int64_t cols, ld;
  int num_rows;
  float scale;
  int grad_dtype, accumulate;
  int K, chunk, slices;
  int64_t nchunks;
  const int *keys, *pos;
  int *count, *list;
  float* partials;          // [chunk][head, tail][cols]
  void* grads[kMaxK];
  int64_t off[kMaxK + 1];
  int chunk_off[kMaxK + 1];
};

// The worker k with off[k] <= i < off[k+1].
template <typename I, typename A>
__device__ __forceinline__ int worker_of(const A* off, int K, I i) {
  int lo = 0, hi = K;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (static_cast<I>(off[m]) <= i) lo = m;
    else hi = m;
  }
  return lo;
}

// Zeroes this CTA's share of the gradients.
__device__ __forceinline__ void fill_share(const SortArgs& a, int cta) {
  for (int k = 0; k < a.K; ++k) {
    char* p = static_cast<char*>(a.fill[k]);
    const int64_t head = min(static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15), a.fill_bytes);
    const int64_t vecs = (a.fill_bytes - head) / 16, tail = a.fill_bytes - head - vecs * 16;
    uint4* q = reinterpret_cast<uint4*>(p + head);
    const int64_t step = static_cast<int64_t>(a.fill_ctas) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(cta) * blockDim.x + threadIdx.x; i < vecs; i += step)
      __stcs(q + i, make_uint4(0u, 0u, 0u, 0u));
    if (cta == 0 && threadIdx.x < 16) {
      if (static_cast<int64_t>(threadIdx.x) < head) p[threadIdx.x] = 0;
      if (static_cast<int64_t>(threadIdx.x) < tail) p[a.fill_bytes - tail + threadIdx.x] = 0;
    }
  }
}

// Key of token i: the token, or num_rows (sorted last, not summed) when it gets no gradient.
__device__ __forceinline__ int token_key(const SortArgs& a, int64_t i) {
  const int64_t t = load_token(a.tokens, a.token_bytes, i);
  return t >= 0 && t < a.num_rows && t != a.padding_idx ? static_cast<int>(t) : a.num_rows;
}

struct SortSmem {
  int hist[kSortWarps][kDigits];  // then: where a warp's keys of a digit go
  int scan[kDigits / 32];
  int key[kSortMost], pos[kSortMost];
};

// Ranks a CTA's keys by one digit.  Item j of lane l of warp w is number (w * kSortItems +
// j) * 32 + l of `n`; after the call, item j goes to place s.hist[w][digit] + rank[j] of the
// CTA's keys in the digit's order, equal digits staying in their order.  Returns, to thread
// d < kDigits, the number of keys of digit d and of smaller digits.
struct DigitCount {
  int here, before;
};
__device__ __forceinline__ DigitCount block_rank(SortSmem& s, const int (&key)[kSortItems], int (&rank)[kSortItems],
                                                int n, int shift, int bits) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int mask = (1 << bits) - 1;
  for (int d = lane; d < kDigits; d += 32) s.hist[w][d] = 0;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    if (w * kSortItems * 32 + j * 32 >= n) break;  // (uniform over the warp)
    const bool in = w * kSortItems * 32 + j * 32 + lane < n;
    const int d = in ? (key[j] >> shift) & mask : kDigits;
    const unsigned same = __match_any_sync(0xFFFFFFFFu, d);
    const int before = __popc(same & ((1u << lane) - 1u));
    int base = 0;
    if (in) base = s.hist[w][d];
    __syncwarp();
    if (in && before == 0) s.hist[w][d] = base + __popc(same);
    __syncwarp();
    rank[j] = base + before;
  }
  __syncthreads();
  DigitCount c = {0, 0};
  if (threadIdx.x < kDigits) {
    int sum = 0;
#pragma unroll 8
    for (int i = 0; i < kSortWarps; ++i) {
      const int v = s.hist[i][threadIdx.x];
      s.hist[i][threadIdx.x] = sum;
      sum += v;
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += up;
    }
    if (lane == 31) s.scan[w] = incl;
    c.here = sum;
    c.before = incl - sum;
  }
  __syncthreads();
  if (threadIdx.x < kDigits) {
    for (int i = 0; i < w; ++i) c.before += s.scan[i];
#pragma unroll 8
    for (int i = 0; i < kSortWarps; ++i) s.hist[i][threadIdx.x] += c.before;
  }
  __syncthreads();
  return c;
}

// Up to kSortMost tokens per worker: one CTA sorts a worker's in shared memory, all passes;
// meanwhile the other CTAs zero the gradients.
__global__ void __launch_bounds__(kSortThreads) table_sort_kernel(const __grid_constant__ SortArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SortSmem& s = *reinterpret_cast<SortSmem*>(smem_raw);
  const int k = blockIdx.x;
  if (k >= a.K) return fill_share(a, k - a.K);
  if (k == 0 && threadIdx.x == 0) *a.join_count = 0;
  const int64_t base = a.off[k];
  const int n = static_cast<int>(a.off[k + 1] - base);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int key[kSortItems], pos[kSortItems], rank[kSortItems];
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int i = (w * kSortItems + j) * 32 + lane;
    key[j] = i < n ? token_key(a, base + i) : 0;
    pos[j] = i;
    rank[j] = 0;
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    block_rank(s, key, rank, n, shift, a.bits);
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
      const int i = (w * kSortItems + j) * 32 + lane;
      if (i >= n) continue;
      const int to = s.hist[w][(key[j] >> shift) & ((1 << a.bits) - 1)] + rank[j];
      s.key[to] = key[j];
      s.pos[to] = pos[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
      const int i = (w * kSortItems + j) * 32 + lane;
      if (i >= n) continue;
      key[j] = s.key[i];
      pos[j] = s.pos[i];
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int i = (w * kSortItems + j) * 32 + lane;
    if (i >= n) continue;
    a.keys[base + i] = key[j];
    a.pos[base + i] = static_cast<int>(base) + pos[j];
  }
}

// More tokens: tiles of kSortMost.  First the digit counts of every tile (and the zeroing),
__global__ void __launch_bounds__(kSortThreads) table_count_kernel(const __grid_constant__ SortArgs a) {
  pdl_enter();
  __shared__ int hist[kDigits];
  const int tile = blockIdx.x;
  if (tile >= a.ntiles) return fill_share(a, tile - a.ntiles);
  if (tile == 0 && threadIdx.x == 0) *a.join_count = 0;
  const int k = worker_of(a.tile_off, a.K, tile);
  const int64_t lo = a.off[k] + static_cast<int64_t>(tile - a.tile_off[k]) * kSortMost;
  const int n = static_cast<int>(min(a.off[k + 1] - lo, static_cast<int64_t>(kSortMost)));
  if (threadIdx.x < kDigits) {
    hist[threadIdx.x] = 0;
    for (int p = 1; p < a.passes; ++p) a.hist[(static_cast<int64_t>(p) * a.ntiles + tile) * kDigits + threadIdx.x] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kSortThreads) atomicAdd(&hist[token_key(a, lo + i) & ((1 << a.bits) - 1)], 1);
  __syncthreads();
  if (threadIdx.x < kDigits) a.hist[static_cast<int64_t>(tile) * kDigits + threadIdx.x] = hist[threadIdx.x];
}

// then one pass per digit: a tile's keys of digit d go after the worker's keys of smaller
// digits and those of digit d in earlier tiles; on the way the next digit is counted in the
// tiles that the keys arrive in.
__global__ void __launch_bounds__(kSortThreads) table_scatter_kernel(const __grid_constant__ SortArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SortSmem& s = *reinterpret_cast<SortSmem*>(smem_raw);
  const int tile = blockIdx.x, k = worker_of(a.tile_off, a.K, tile);
  const int64_t base = a.off[k], lo = base + static_cast<int64_t>(tile - a.tile_off[k]) * kSortMost;
  const int n = static_cast<int>(min(a.off[k + 1] - lo, static_cast<int64_t>(kSortMost)));
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, mask = (1 << a.bits) - 1;
  int key[kSortItems], pos[kSortItems], rank[kSortItems];
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int i = (w * kSortItems + j) * 32 + lane;
    key[j] = pos[j] = rank[j] = 0;
    if (i < n) {
      key[j] = a.keys_in ? a.keys_in[lo + i] : token_key(a, lo + i);
      pos[j] = a.keys_in ? a.pos_in[lo + i] : static_cast<int>(lo + i);
    }
  }
  const DigitCount c = block_rank(s, key, rank, n, a.shift, a.bits);
  // place of this tile's digit d in the worker's order, minus its place in the tile's
  if (threadIdx.x < kDigits) {
    const int* h = a.hist + static_cast<int64_t>(a.pass) * a.ntiles * kDigits + threadIdx.x;
    int earlier = 0, total = 0;
#pragma unroll 4
    for (int t = a.tile_off[k]; t < a.tile_off[k + 1]; ++t) {
      const int v = h[static_cast<int64_t>(t) * kDigits];
      if (t < tile) earlier += v;
      total += v;
    }
    int incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += up;
    }
    if (lane == 31) s.scan[w] = incl;
    s.key[threadIdx.x] = incl - total + earlier - c.before;
  }
  __syncthreads();
  if (threadIdx.x < kDigits)
    for (int i = 0; i < w; ++i) s.key[threadIdx.x] += s.scan[i];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int i = (w * kSortItems + j) * 32 + lane;
    if (i >= n) continue;
    const int d = (key[j] >> a.shift) & mask;
    const int to = s.hist[w][d] + rank[j] + s.key[d];
    a.keys[base + to] = key[j];
    a.pos[base + to] = pos[j];
    if (a.pass + 1 < a.passes)
      atomicAdd(&a.hist[(static_cast<int64_t>(a.pass + 1) * a.ntiles + a.tile_off[k] + to / kSortMost) * kDigits +
                        ((key[j] >> (a.shift + a.bits)) & mask)], 1);
  }
}

// Writes scale * acc to (or adds it to) 256 columns of a gradient's row.
template <typename G, int LAYOUT>
__device__ __forceinline__ void put_row(const TableGradArgs& a, int k, int row, int64_t c0, int lane, const float (&acc)[8]) {
  G* out = static_cast<G*>(a.grads[k]) + row * a.cols + c0;
  float v[8];
  if (a.accumulate) {
    const Raw8<G> old = load8<G, LAYOUT>(out, a.cols - c0, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(raw_value<G>(old, e), __fmul_rn(a.scale, acc[e]));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = a.scale * acc[e];
  }
  store8<G, LAYOUT>(out, a.cols - c0, lane, v);
}

// Sums inside one chunk of sorted tokens, 256 columns per warp; rows are loaded eight at a
// time.  Bound by grad_out's bytes (each read once) and the gradient rows written.
template <typename T, typename G, int LAYOUT>
__global__ void __launch_bounds__(kEmbThreads) table_sum_kernel(const __grid_constant__ TableGradArgs a) {
  pdl_enter();
  constexpr int B = 8;
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * kEmbWarps + (threadIdx.x >> 5);
  const int64_t chunk = item / static_cast<uint32_t>(a.slices);
  if (chunk >= a.nchunks) return;
  const int64_t c0 = (item - chunk * a.slices) * kSlice;
  const int k = worker_of(a.chunk_off, a.K, chunk);
  const int64_t first = a.off[k], last = a.off[k + 1], lo = first + (chunk - a.chunk_off[k]) * a.chunk;
  const int m = static_cast<int>(min(static_cast<int64_t>(a.chunk), last - lo));
  int key = a.num_rows, pos = 0;
  if (lane < m) {
    key = a.keys[lo + lane];
    pos = a.pos[lo + lane];
  }
  int cur = __shfl_sync(0xFFFFFFFFu, key, 0);
  if (cur == a.num_rows) return;  // nothing but tokens without a gradient
  bool head = lo > first && a.keys[lo - 1] == cur;
  const int next = lo + m < last ? a.keys[lo + m] : a.num_rows;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  auto piece = [&](int slot) {
    store8<float, LAYOUT>(a.partials + (chunk * 2 + slot) * a.cols + c0, a.cols - c0, lane, acc);
  };
  for (int i0 = 0; i0 < m; i0 += B) {
    Raw8<T> r[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int p = __shfl_sync(0xFFFFFFFFu, pos, (i0 + b) & 31), q = __shfl_sync(0xFFFFFFFFu, key, (i0 + b) & 31);
      r[b] = load8<T, LAYOUT>(static_cast<const T*>(a.dy) + p * a.ld + c0, i0 + b < m && q != a.num_rows ? a.cols - c0 : 0, lane);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (i0 + b >= m) break;
      const int q = __shfl_sync(0xFFFFFFFFu, key, i0 + b);
      if (q != cur) {
        if (head) piece(0);
        else if (cur != a.num_rows) put_row<G, LAYOUT>(a, k, cur, c0, lane, acc);
        cur = q;
        head = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += raw_value<T>(r[b], e);
    }
  }
  if (cur == a.num_rows) return;
  const bool tail = next == cur;
  if (!head && !tail) return put_row<G, LAYOUT>(a, k, cur, c0, lane, acc);
  piece(head ? 0 : 1);
  if (!head && c0 == 0 && lane == 0) a.list[atomicAdd(a.count, 1)] = static_cast<int>(chunk);
}

// Joins the pieces of the runs that cross chunks: one CTA per run and 256 columns, its
// warps taking consecutive parts of the pieces.
template <typename G, int LAYOUT>
__global__ void __launch_bounds__(kEmbThreads) table_join_kernel(const __grid_constant__ TableGradArgs a) {
  pdl_enter();
  constexpr int B = 8;
  __shared__ float part[kEmbWarps][kSlice];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t items = static_cast<int64_t>(*a.count) * a.slices;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t chunk = a.list[item / a.slices], c0 = item % a.slices * kSlice;
    const int k = worker_of(a.chunk_off, a.K, chunk);
    const int64_t first = a.off[k], last = a.off[k + 1];
    const int64_t after = first + (chunk + 1 - a.chunk_off[k]) * a.chunk;  // start of the next chunk
    const int key = a.keys[after];
    // how many chunks begin inside the run: the last such beginning, by bisection
    int64_t lo = 0, hi = (last - after + a.chunk - 1) / a.chunk;  // keys[after + lo * chunk] == key, that of hi is not
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (a.keys[after + mid * a.chunk] == key) lo = mid;
      else hi = mid;
    }
    const int64_t pieces = lo + 2;  // the chunk's own tail, and the heads of the following ones
    const int64_t p0 = pieces * w / kEmbWarps, p1 = pieces * (w + 1) / kEmbWarps;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int64_t i0 = p0; i0 < p1; i0 += B) {
      Raw8<float> r[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int64_t i = i0 + b;
        const float* p = a.partials + ((chunk + i) * 2 + (i == 0 ? 1 : 0)) * a.cols + c0;
        r[b] = load8<float, LAYOUT>(p, i < p1 ? a.cols - c0 : 0, lane);
      }
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += raw_value<float>(r[b], e);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[w][e * 32 + lane] = acc[e];
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[e] = part[0][e * 32 + lane];
#pragma unroll
        for (int i = 1; i < kEmbWarps; ++i) acc[e] += part[i][e * 32 + lane];
      }
      put_row<G, LAYOUT>(a, k, key, c0, lane, acc);
    }
    __syncthreads();
  }
}

template <typename T>
int launch_lookup(const LookupArgs& a, bool vec, unsigned grid, cudaStream_t stream) {
  return launch_pdl(vec ? lookup_kernel<T, kVec> : lookup_kernel<T, kStrided>, dim3(grid), dim3(kEmbThreads), 0, stream, a);
}
template <typename T, typename G>
int launch_sum(const TableGradArgs& a, bool vec, unsigned grid, cudaStream_t stream) {
  return launch_pdl(vec ? table_sum_kernel<T, G, kVec> : table_sum_kernel<T, G, kStrided>, dim3(grid), dim3(kEmbThreads), 0,
                    stream, a);
}
template <typename G>
int launch_join(const TableGradArgs& a, bool vec, unsigned grid, cudaStream_t stream) {
  return launch_pdl(vec ? table_join_kernel<G, kVec> : table_join_kernel<G, kStrided>, dim3(grid), dim3(kEmbThreads), 0,
                    stream, a);
}

// Allows a sort kernel its shared memory (once per device and kernel).
int allow_smem(const void* kernel, int which) {
  static bool done[2][64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return static_cast<int>(cudaErrorInvalidDevice);
  if (dev >= 0 && dev < 64 && done[which][dev]) return 0;
  const int rc = static_cast<int>(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortSmem)));
  if (rc == 0 && dev >= 0 && dev < 64) done[which][dev] = true;
  return rc;
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
  const int parts = static_cast<int>((cols + kLookupVecs * kSlice - 1) / (kLookupVecs * kSlice));
  if (n * parts > UINT32_MAX - kEmbWarps) return ADASUM_ERR_UNSUPPORTED;
  const int64_t grid = (n * parts + kEmbWarps - 1) / kEmbWarps;
  const LookupArgs a = {table, num_rows, cols, tokens, token_bytes, n, scale, out, parts};
  const bool vec = is_aligned(table, 16) && is_aligned(out, 16) && cols * e % 16 == 0;
  return counted_launch(stream, "embedding", static_cast<double>(n) * (2 * cols * e + token_bytes), [&] {
    return dtype == ADASUM_BF16 ? launch_lookup<bf16>(a, vec, static_cast<unsigned>(grid), stream)
                                : launch_lookup<float>(a, vec, static_cast<unsigned>(grid), stream);
  });
}

int64_t adasum_embedding_backward_scratch_bytes(int64_t n, int64_t cols, int K) {
  if (n <= 0 || cols <= 0 || K <= 0) return 0;
  return Scratch(n, cols, K).total;
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
  if (cols > INT32_MAX || n >= INT32_MAX || num_rows >= INT32_MAX) return ADASUM_ERR_UNSUPPORTED;
  if (chunk_bound(n, cols, K) * ((cols + kSlice - 1) / kSlice) > UINT32_MAX - kEmbWarps) return ADASUM_ERR_UNSUPPORTED;
  if (num_rows == 0) return ADASUM_OK;
  if (grads == nullptr || (n > 0 && (grad_out == nullptr || tokens == nullptr || ld < cols)))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t need = adasum_embedding_backward_scratch_bytes(n, cols, K);
  if (need > 0 && (scratch == nullptr || scratch_bytes < need || !is_aligned(scratch, 256)))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype), ge = dtype_bytes(grad_dtype);
  SortArgs s = {};
  TableGradArgs a = {};
  BufferSet set;
  set.read(grad_out, span_bytes(n, cols, ld, e));
  set.read(tokens, n * token_bytes);
  set.write(scratch, need);
  bool vec = is_aligned(grad_out, 16) && ld * e % 16 == 0 && cols * ge % 16 == 0 && cols % 4 == 0;
  int64_t most = 0;
  const int chunk = chunk_tokens(n, cols);
  for (int k = 0; k < K; ++k) {
    if (grads[k] == nullptr) return ADASUM_ERR_INVALID_ARG;
    set.write(grads[k], num_rows * cols * ge);
    vec = vec && is_aligned(grads[k], 16);
    const int64_t nk = worker_offsets[k + 1] - worker_offsets[k];
    most = std::max(most, nk);
    s.fill[k] = a.grads[k] = grads[k];
    s.off[k + 1] = a.off[k + 1] = worker_offsets[k + 1];
    s.tile_off[k + 1] = s.tile_off[k] + static_cast<int>((nk + kSortMost - 1) / kSortMost);
    a.chunk_off[k + 1] = a.chunk_off[k] + static_cast<int>((nk + chunk - 1) / chunk);
  }
  if (set.conflict()) return ADASUM_ERR_ALIAS;
  const Scratch at(std::max<int64_t>(n, 0), cols, K);
  char* base = static_cast<char*>(scratch);
  auto ints = [&](int64_t offset) { return n > 0 ? reinterpret_cast<int*>(base + offset) : nullptr; };
  if (n == 0) {  // nothing to sum: zero the gradients, or leave them
    if (accumulate) return ADASUM_OK;
    for (int k = 0; k < K; ++k)
      if (cudaMemsetAsync(grads[k], 0, static_cast<size_t>(num_rows * cols * ge), stream) != cudaSuccess)
        return ADASUM_ERR_CUDA;
    return ADASUM_OK;
  }
  // digits: as few passes of at most 8 bits as the keys 0..num_rows need
  int bits = 1;
  while ((num_rows >> bits) != 0) ++bits;
  s.tokens = tokens;
  s.token_bytes = token_bytes;
  s.num_rows = static_cast<int>(num_rows);
  s.padding_idx = padding_idx;
  s.K = K;
  s.passes = (bits + 7) / 8;
  s.bits = (bits + s.passes - 1) / s.passes;
  s.ntiles = s.tile_off[K];
  s.hist = ints(at.hist);
  s.join_count = ints(at.count);
  s.fill_bytes = accumulate ? 0 : num_rows * cols * ge;
  const int64_t fill_vecs = static_cast<int64_t>(K) * (s.fill_bytes / 16);
  s.fill_ctas = accumulate ? 0 : static_cast<int>(std::min<int64_t>(2 * sm_count(), 1 + fill_vecs / kSortThreads));
  const int sorters = most <= kSortMost ? K : s.ntiles;
  const double fill = static_cast<double>(K) * s.fill_bytes;
  int out = 0;  // which half of the key and position buffers holds the result
  if (most <= kSortMost) {
    s.keys = ints(at.keys[0]);
    s.pos = ints(at.pos[0]);
    if (adasum_status_t st = counted_launch(stream, "table_sort", fill, [&] {
          if (int rc = allow_smem(reinterpret_cast<const void*>(table_sort_kernel), 0)) return rc;
          return launch_pdl(table_sort_kernel, dim3(sorters + s.fill_ctas), dim3(kSortThreads), sizeof(SortSmem), stream, s);
        }))
      return st;
  } else {
    if (adasum_status_t st = counted_launch(stream, "table_count", fill, [&] {
          return launch_pdl(table_count_kernel, dim3(sorters + s.fill_ctas), dim3(kSortThreads), 0, stream, s);
        }))
      return st;
    for (s.pass = 0; s.pass < s.passes; ++s.pass) {
      out = s.pass & 1;
      s.shift = s.pass * s.bits;
      s.keys_in = s.pass > 0 ? ints(at.keys[1 - out]) : nullptr;
      s.pos_in = s.pass > 0 ? ints(at.pos[1 - out]) : nullptr;
      s.keys = ints(at.keys[out]);
      s.pos = ints(at.pos[out]);
      if (adasum_status_t st = counted_launch(stream, "table_scatter", 0.0, [&] {
            if (int rc = allow_smem(reinterpret_cast<const void*>(table_scatter_kernel), 1)) return rc;
            return launch_pdl(table_scatter_kernel, dim3(sorters), dim3(kSortThreads), sizeof(SortSmem), stream, s);
          }))
        return st;
    }
  }
  a.dy = grad_out;
  a.cols = cols;
  a.ld = ld;
  a.num_rows = static_cast<int>(num_rows);
  a.scale = scale;
  a.grad_dtype = static_cast<int>(grad_dtype);
  a.accumulate = accumulate != 0;
  a.K = K;
  a.chunk = chunk;
  a.slices = static_cast<int>((cols + kSlice - 1) / kSlice);
  a.nchunks = a.chunk_off[K];
  a.keys = ints(at.keys[out]);
  a.pos = ints(at.pos[out]);
  a.count = ints(at.count);
  a.list = ints(at.list);
  a.partials = reinterpret_cast<float*>(base + at.partials);
  const int64_t grid = (a.nchunks * a.slices + kEmbWarps - 1) / kEmbWarps;
  const unsigned g = static_cast<unsigned>(grid);
  if (adasum_status_t st = counted_launch(stream, "table_sum", static_cast<double>(n) * (cols * e + 8), [&] {
        if (dtype == ADASUM_BF16)
          return grad_dtype == ADASUM_BF16 ? launch_sum<bf16, bf16>(a, vec, g, stream) : launch_sum<bf16, float>(a, vec, g, stream);
        return grad_dtype == ADASUM_BF16 ? launch_sum<float, bf16>(a, vec, g, stream) : launch_sum<float, float>(a, vec, g, stream);
      }))
    return st;
  const unsigned joiners = static_cast<unsigned>(std::min<int64_t>(a.nchunks * a.slices, 4 * static_cast<int64_t>(sm_count())));
  return counted_launch(stream, "table_join", 0.0, [&] {
    return grad_dtype == ADASUM_BF16 ? launch_join<bf16>(a, vec, joiners, stream) : launch_join<float>(a, vec, joiners, stream);
  });
}

}  // extern "C"
