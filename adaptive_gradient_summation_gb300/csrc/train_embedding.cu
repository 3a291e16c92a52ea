// train_embedding.cu -- token embeddings and the table's gradient, per worker.
//
// The gradient of a table row is the sum of the rows of grad_out whose token it is.  The
// tokens of each worker are sorted (stably, so that equal tokens stay in their order) and
// the sorted list is cut into chunks of equal length, whatever the tokens: one CTA sums the
// runs of equal tokens inside one chunk over 256 columns, its warps taking equal parts.  A
// run that lies inside the chunk goes straight to the gradient; the pieces of a run that
// crosses chunks go to scratch memory and are joined in order by a last kernel.  So a token
// that makes up most of the batch costs no more than any other (65536 equal tokens x 1024
// columns, added, 78 us in a graph, 65536 different ones 93), and every sum has a fixed order.
// Where all workers have at most 256 tokens the CTAs sort themselves and a warp takes a run to
// its end: there one token for all costs more (256 equal tokens x 1024 columns 62 us in a graph,
// 256 different ones 11).
//
// Times in the comments are those of one launch between two events (the library's profiler; 4
// to 6 us of it are the launch), unless they are said to be of a call in a graph of many or of a
// pass, a call among others through the Python binding.
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

// out = scale * table[token], 0 where a token is not in the table.  One warp copies up to 1024
// columns of one token's row, four 16-byte vectors per lane in flight; rows that repeat come
// from L2.  Bound by the output's bytes: 65536 tokens x 2048 bf16 of a table of 50304 rows in
// 57 us, 52 of them the kernel's (268 MB written; two vectors in flight 59.6), 8 tokens in 6.
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
  Raw8<T, LAYOUT> r[kLookupVecs];
#pragma unroll
  for (int j = 0; j < kLookupVecs; ++j) r[j] = load8<T, LAYOUT, true>(src + j * kSlice, there ? slice_left(left, j * kSlice) : 0, lane);
#pragma unroll
  for (int j = 0; j < kLookupVecs; ++j) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = there ? a.scale * raw_value<T, LAYOUT>(r[j], e) : 0.f;
    store8<T, LAYOUT>(dst + j * kSlice, slice_left(left, j * kSlice), lane, v);
  }
}

// ------------------------------------------------------------------- the table's gradient

// A worker's tokens are sorted by one CTA up to kSortMost, else by tiles of all CTAs.  In a
// graph, the whole gradient of one worker x 1024 columns, added: 4096 tokens 21.8 us by one
// CTA, 22.7 by tiles; 8192 tokens 29.8 and 22.5.
constexpr int kSortThreads = 1024, kSortItems = 4;
constexpr int kSortMost = kSortThreads * kSortItems;
constexpr int kTileThreads = 256, kTileItems = 4;         // of a tile of the multi-CTA sort
constexpr int kTile = kTileThreads * kTileItems;
constexpr int kScanTiles = 64;  // of a worker, above which a kernel of its own sums the tiles' counts
constexpr int kDigits = 256;
constexpr int kMostPasses = 4;
constexpr int kSelfSort = kEmbThreads;  // tokens of a worker that the summing CTAs sort themselves
constexpr int kSelfPart = 4;            // ... and of a warp then (8: 128 tokens 5.7 us in a graph, not 4.4)

// Whether the summing CTAs sort their worker's tokens themselves: few tokens for each, and a
// token and its place in 32 bits.  That is one launch and no scratch memory, though every CTA
// of a worker repeats the sort.  In a graph, against sorting in a kernel before: one worker x
// 1024 columns, 128 tokens 4.4 and 11.0 us, 256 tokens 7.4 and 13.4; 256 x 4096 columns 9.0
// and 14.2; a pass of 128 tokens 18.7 and 29.1.  (The sort is by counting, quadratic in the
// tokens, so it ends where a thread no longer has a token each.)
bool self_sorted(const int64_t* offs, int K, int64_t num_rows) {
  for (int k = 0; k < K; ++k)
    if (offs[k + 1] - offs[k] > kSelfSort) return false;
  return num_rows < (1 << 23);
}

// Tokens per warp of a chunk, by the tokens times slices there are: few enough that the warps
// cover the memory's latency, and not so few that what a warp does once weighs.  Added, in a
// graph, with 8, 16 and 32: 8192 tokens x 1024 columns 29.8, 31.4, 34.5 us; 65536 x 256
// 42.6, 36.5, 40.6; 20000 x 1024 36.3, 33.5, 39.5; 65536 x 1024 85.4, 68.1, 65.0.
int warp_tokens(int64_t n, int64_t cols) {
  const int64_t work = n * ((cols + kSlice - 1) / kSlice);
  return work >= 150000 ? 32 : work >= 50000 ? 16 : 8;
}
int64_t chunk_bound(int64_t n, int64_t cols, int K) { return n / (warp_tokens(n, cols) * kEmbWarps) + K; }
int64_t tile_bound(int64_t n, int K) { return n / kTile + K; }

// Regions of the scratch memory.
struct Scratch {
  int64_t keys[2], pos[2], hist, totals, count, list, partials, total;
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
    totals = take(4 * kDigits * static_cast<int64_t>(K));
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
  int* totals;         // [K][kDigits]: null, or hist holds the counts of a worker's earlier tiles
  int* join_count;
  void* fill[kMaxK];   // gradients to be zeroed
  int64_t fill_bytes;  // of each (0: accumulate)
  int64_t fill_pieces; // of each
  int64_t fill_first;  // of this launch's pieces of all
  int64_t off[kMaxK + 1];
  int tile_off[kMaxK + 1];  // first tile of a worker (multi-CTA sort)
};

struct TableGradArgs {
  const void* dy;
  int64_t cols, ld;
  const void* tokens;       // for CTAs that sort themselves
  int64_t padding_idx;
  int token_bytes;
  int num_rows;
  float scale;
  int accumulate;
  int K, part, slices;      // tokens per warp of a chunk
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

// Zeroes piece `piece` of the gradients: a CTA's kFillVecs vectors per thread of one of them.
// Many CTAs that each write one piece and leave, so that pieces are written nearly in their
// order, reach 7.6 TB/s on 1 GB; a grid that stays and strides, whose CTAs drift apart, 6.4.
// (Beside the sort of 16 workers x 4096 tokens 4, 8, 16, 32 vectors: 159, 137, 135, 137 us;
// the whole gradient of 8192 tokens, one table of 30522 x 1024, in a graph: 26.1, 26.3, 30.8, 33.4.)
constexpr int kFillVecs = 8;
__device__ __forceinline__ void fill_piece(const SortArgs& a, int64_t piece) {
  const int k = static_cast<int>(piece / a.fill_pieces);
  const int64_t j = piece - k * a.fill_pieces;
  char* p = static_cast<char*>(a.fill[k]);
  const int64_t head = min(static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15), a.fill_bytes);
  const int64_t vecs = (a.fill_bytes - head) / 16, tail = a.fill_bytes - head - vecs * 16;
  uint4* q = reinterpret_cast<uint4*>(p + head);
  int64_t i = j * kFillVecs * blockDim.x + threadIdx.x;
#pragma unroll
  for (int u = 0; u < kFillVecs; ++u, i += blockDim.x)
    if (i < vecs) __stcs(q + i, make_uint4(0u, 0u, 0u, 0u));
  if (j == 0 && threadIdx.x < 16) {
    if (static_cast<int64_t>(threadIdx.x) < head) p[threadIdx.x] = 0;
    if (static_cast<int64_t>(threadIdx.x) < tail) p[a.fill_bytes - tail + threadIdx.x] = 0;
  }
}

// Key of token i: the token, or num_rows (sorted last, not summed) when it gets no gradient.
template <typename A>
__device__ __forceinline__ int token_key(const A& a, int64_t i) {
  const int64_t t = load_token(a.tokens, a.token_bytes, i);
  return t >= 0 && t < a.num_rows && t != a.padding_idx ? static_cast<int>(t) : a.num_rows;
}

template <int THREADS, int ITEMS>
struct SortSmem {
  static constexpr int kWarps = THREADS / 32, kParts = THREADS / kDigits;
  int hist[kWarps][kDigits];      // then: where a warp's keys of a digit go
  int part[kParts][kDigits];      // counts of a digit in the warps of a part
  int scan[kDigits / 32];
  int key[THREADS * ITEMS], pos[THREADS * ITEMS];
};

// Ranks a CTA's keys by one digit.  Item j of lane l of warp w is number (w * ITEMS + j) * 32
// + l of `n`; after the call, item j goes to place s.hist[w][digit] + rank[j] of the CTA's
// keys in the digit's order, equal digits staying in their order.  Returns, to thread
// d < kDigits, the number of keys of digit d and of smaller digits.
struct DigitCount {
  int here, before;
};
template <int THREADS, int ITEMS>
__device__ __forceinline__ DigitCount block_rank(SortSmem<THREADS, ITEMS>& s, const int (&key)[ITEMS],
                                                int (&rank)[ITEMS], int n, int shift, int bits) {
  constexpr int kRows = 8;  // warps of a part
  static_assert(THREADS / 32 == kRows * (THREADS / kDigits), "eight warps per 256 threads");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int mask = (1 << bits) - 1;
#pragma unroll
  for (int i = 0; i < kDigits / 32; ++i) s.hist[w][i * 32 + lane] = 0;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    if ((w * ITEMS + j) * 32 >= n) break;  // (uniform over the warp)
    const bool in = (w * ITEMS + j) * 32 + lane < n;
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
  // digit d of the eight warps of part p, by thread p * 256 + d
  const int d = threadIdx.x & (kDigits - 1), p = threadIdx.x / kDigits;
  int row[kRows], sum = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) row[i] = s.hist[p * kRows + i][d];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int v = row[i];
    row[i] = sum;
    sum += v;
  }
  s.part[p][d] = sum;
  __syncthreads();
  int total = 0, mine = 0;
#pragma unroll
  for (int i = 0; i < THREADS / kDigits; ++i) {
    if (i == p) mine = total;
    total += s.part[i][d];
  }
  int incl = total;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, incl, i);
    if (lane >= i) incl += up;
  }
  if (p == 0 && lane == 31) s.scan[w] = incl;
  __syncthreads();
  int before = incl - total;
#pragma unroll
  for (int i = 0; i < kDigits / 32; ++i)
    if (i < d / 32) before += s.scan[i];
#pragma unroll
  for (int i = 0; i < kRows; ++i) s.hist[p * kRows + i][d] = row[i] + mine + before;
  __syncthreads();
  return {total, before};
}

// Up to kSortMost tokens per worker: one CTA sorts a worker's in shared memory, all passes;
// meanwhile the other CTAs zero the gradients.  Bound by the bytes zeroed where there are some:
// 16 workers x 4096 tokens, tables of 30522 x 1024 bf16 (1 GB) in 137 us, 7.3 TB/s.
__global__ void __launch_bounds__(kSortThreads) table_sort_kernel(const __grid_constant__ SortArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& s = *reinterpret_cast<SortSmem<kSortThreads, kSortItems>*>(smem_raw);
  const int k = blockIdx.x;
  if (k >= a.K) return fill_piece(a, k - a.K);
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
    block_rank<kSortThreads, kSortItems>(s, key, rank, n, shift, a.bits);
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

// The zeroing alone.
__global__ void __launch_bounds__(kTileThreads) table_fill_kernel(const __grid_constant__ SortArgs a) {
  pdl_enter();
  fill_piece(a, blockIdx.x);
}

// More tokens: tiles of kTile.  First the digit counts of every tile,
__global__ void __launch_bounds__(kTileThreads) table_count_kernel(const __grid_constant__ SortArgs a) {
  pdl_enter();
  static_assert(kTileThreads == kDigits, "a thread per digit");
  __shared__ int hist[kDigits];
  const int tile = blockIdx.x;
  if (tile == 0 && threadIdx.x == 0) *a.join_count = 0;
  const int k = worker_of(a.tile_off, a.K, tile);
  const int64_t lo = a.off[k] + static_cast<int64_t>(tile - a.tile_off[k]) * kTile;
  const int n = static_cast<int>(min(a.off[k + 1] - lo, static_cast<int64_t>(kTile)));
  hist[threadIdx.x] = 0;
  for (int p = 1; p < a.passes; ++p) a.hist[(static_cast<int64_t>(p) * a.ntiles + tile) * kDigits + threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    const int i = j * kTileThreads + threadIdx.x;
    if (i < n) atomicAdd(&hist[token_key(a, lo + i) & ((1 << a.bits) - 1)], 1);
  }
  __syncthreads();
  a.hist[static_cast<int64_t>(tile) * kDigits + threadIdx.x] = hist[threadIdx.x];
}

// then, where a worker has many tiles, before each pass the counts of its earlier tiles in
// place of a tile's own, and their totals: 32 digits of a worker per CTA, its tiles in as many
// parts as a CTA has warps, each read twice (sums, then prefixes).  Without it every tile of a
// pass reads the counts of all the worker's tiles, which is less where they are few and grows
// with their square.  Gradient of 50304 rows x 8 columns added, tokens of one worker, one call
// in a graph, without and with: 65536 47.6 and 47.6 us, 131072 87 and 76, 1048576 431 and 228, 4194304 3100 and
// 799; 16 workers of 65536 each, 64 columns, 261 and 252.
__global__ void __launch_bounds__(kSortThreads) table_scan_kernel(const __grid_constant__ SortArgs a) {
  pdl_enter();
  constexpr int kParts = kSortThreads / 32;
  __shared__ int part[kParts][32];
  const int k = blockIdx.x / (kDigits / 32), lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int d = blockIdx.x % (kDigits / 32) * 32 + lane;
  const int64_t first = a.tile_off[k], tiles = a.tile_off[k + 1] - first;
  const int64_t t0 = first + tiles * w / kParts, t1 = first + tiles * (w + 1) / kParts;
  int* h = a.hist + static_cast<int64_t>(a.pass) * a.ntiles * kDigits + d;
  int sum = 0;
#pragma unroll 8
  for (int64_t t = t0; t < t1; ++t) sum += h[t * kDigits];
  part[w][lane] = sum;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll 8
  for (int i = 0; i < kParts; ++i) {
    const int v = part[i][lane];
    if (i < w) before += v;
    total += v;
  }
  if (w == 0) a.totals[k * kDigits + d] = total;
  for (int64_t t = t0; t < t1; t += 8) {
    int v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = t + i < t1 ? h[(t + i) * kDigits] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (t + i < t1) h[(t + i) * kDigits] = before;
      before += v[i];
    }
  }
}

// then one pass per digit: a tile's keys of digit d go after the worker's keys of smaller
// digits and those of digit d in earlier tiles; on the way the next digit is counted in the
// tiles that the keys arrive in.  Each pass zeroes its part of the gradients beside.
__global__ void __launch_bounds__(kTileThreads) table_scatter_kernel(const __grid_constant__ SortArgs a) {
  pdl_enter();
  __shared__ SortSmem<kTileThreads, kTileItems> s;
  const int tile = blockIdx.x;
  if (tile >= a.ntiles) return fill_piece(a, a.fill_first + tile - a.ntiles);
  const int k = worker_of(a.tile_off, a.K, tile);
  const int64_t base = a.off[k], lo = base + static_cast<int64_t>(tile - a.tile_off[k]) * kTile;
  const int n = static_cast<int>(min(a.off[k + 1] - lo, static_cast<int64_t>(kTile)));
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, mask = (1 << a.bits) - 1;
  int key[kTileItems], pos[kTileItems], rank[kTileItems];
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    const int i = (w * kTileItems + j) * 32 + lane;
    key[j] = pos[j] = rank[j] = 0;
    if (i < n) {
      key[j] = a.keys_in ? a.keys_in[lo + i] : token_key(a, lo + i);
      pos[j] = a.keys_in ? a.pos_in[lo + i] : static_cast<int>(lo + i);
    }
  }
  // (thread d: digit d of the worker's tiles)
  const int* h = a.hist + static_cast<int64_t>(a.pass) * a.ntiles * kDigits + threadIdx.x;
  int earlier = 0, total = 0;
  if (a.totals) {
    earlier = h[static_cast<int64_t>(tile) * kDigits];
    total = a.totals[k * kDigits + threadIdx.x];
  } else {
#pragma unroll 8
    for (int t = a.tile_off[k]; t < a.tile_off[k + 1]; ++t) {
      const int v = h[static_cast<int64_t>(t) * kDigits];
      if (t < tile) earlier += v;
      total += v;
    }
  }
  const DigitCount c = block_rank<kTileThreads, kTileItems>(s, key, rank, n, a.shift, a.bits);
  // place of this tile's digit d in the worker's order, minus its place in the tile's
  int incl = total;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, incl, i);
    if (lane >= i) incl += up;
  }
  if (lane == 31) s.scan[w] = incl;
  __syncthreads();
  int place = incl - total + earlier - c.before;
  for (int i = 0; i < w; ++i) place += s.scan[i];
  s.key[threadIdx.x] = place;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    const int i = (w * kTileItems + j) * 32 + lane;
    if (i >= n) continue;
    const int d = (key[j] >> a.shift) & mask;
    const int to = s.hist[w][d] + rank[j] + s.key[d];
    a.keys[base + to] = key[j];
    a.pos[base + to] = pos[j];
    if (a.pass + 1 < a.passes)
      atomicAdd(&a.hist[(static_cast<int64_t>(a.pass + 1) * a.ntiles + a.tile_off[k] + to / kTile) * kDigits +
                        ((key[j] >> (a.shift + a.bits)) & mask)], 1);
  }
}

// Writes scale * acc to 256 columns of a gradient's row; ADD: added to `old`, its values.
template <typename G, int LAYOUT, bool ADD>
__device__ __forceinline__ void put_row(G* out, float scale, int left, int lane, const F2 (&acc)[4], const Raw8<G, LAYOUT>& old) {
  F2 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mul2(acc[i], f2(scale));
  if constexpr (ADD) {
    F2 o[4];
    unpack8<G, LAYOUT>(old, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (scalar sums: a packed product and sum would be contracted)
      const float2 x = parts(o[i]), y = parts(v[i]);
      v[i] = f2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
    }
  }
  store8<G, LAYOUT>(out, left, lane, v);
}

__device__ __forceinline__ void add8(F2 (&acc)[4], const F2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = add2(acc[i], v[i]);
}

// What a warp found at the ends of its part of a chunk.
enum Ends : int {
  kHead = 1,   // its first run began earlier
  kSpan = 2,   // ... and does not end here either
  kTail = 4,   // its last run begins here and does not end here
};

// Sums inside one chunk of sorted tokens, 256 columns per CTA and a part of the chunk per
// warp.  A lane copies its pieces of the next rows to shared memory ahead of their use (8 or
// 4 rows, 4 KiB a warp), which takes no registers and no exchange between lanes (N = 1: the
// next row is held in registers).  Runs that cross warps are joined through
// shared memory, runs that cross chunks leave their pieces in scratch memory.
// SORT: the CTA sorts its worker's few tokens itself, and a warp takes the runs that begin in
// its part to their end, so that nothing is left to join.
// The bytes are grad_out's, read once, and the gradient rows written; bound by the issue of
// instructions (73% of its slots), since with tokens spread over the table most runs are one
// or two rows, and a row costs its key, its place and a store besides the sum: 65536 rows x
// 1024 bf16 of 16 workers 41 us after the sort (135 MB read), 128 rows with their sort 12 (in a
// graph 4.4).
// (Two slices a warp measured slower.)
template <typename T, typename G, int LAYOUT, bool ADD>
struct SumSmem {
  static constexpr int kAhead = 16 / sizeof(T);  // rows on their way
  static constexpr int kRing = LAYOUT != kStrided ? kEmbWarps : 1, kOld = LAYOUT != kStrided && ADD ? kEmbWarps : 1;
  using Slot = LaneSlot<T, LAYOUT != kStrided ? LAYOUT : kWide<T>>;
  using OldSlot = LaneSlot<G, LAYOUT != kStrided ? LAYOUT : kWide<G>>;
  union {
    struct {
      Slot dy[kRing][kAhead];
      OldSlot old[kOld][kAhead];  // gradient rows to be added to
    } ring;
    float piece[kEmbWarps][2][kSlice];
    uint32_t unsorted[kSelfSort];
  };
};
template <typename T, typename G, int LAYOUT, bool SORT, bool ADD>
__global__ void __launch_bounds__(kEmbThreads) table_sum_kernel(const __grid_constant__ TableGradArgs a) {
  pdl_enter();
  using Smem = SumSmem<T, G, LAYOUT, ADD>;
  constexpr int kAhead = Smem::kAhead;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  __shared__ int ends[kEmbWarps], tail_key[kEmbWarps];
  __shared__ int own_keys[SORT ? kSelfSort : 1], own_pos[SORT ? kSelfSort : 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t chunk = blockIdx.x / static_cast<uint32_t>(a.slices);
  const int64_t c0 = static_cast<int64_t>(blockIdx.x - chunk * a.slices) * kSlice;
  const int left = slice_left(a.cols, c0), cols = static_cast<int>(a.cols);
  const int k = worker_of(a.chunk_off, a.K, static_cast<int>(chunk));
  const int64_t first = a.off[k], last = a.off[k + 1];
  int64_t lo = first + (static_cast<int64_t>(chunk - a.chunk_off[k]) * kEmbWarps + w) * a.part;
  int m = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(a.part), last - lo)));
  // the part's n tokens with a gradient: the sorted keys and rows of SORT's are read from
  // shared memory, others are held one per lane
  int n, key = a.num_rows, at = 0, before = a.num_rows, after = a.num_rows, skip = 0;
  if constexpr (SORT) {
    // a token's place is the number of smaller (key, index) pairs; `ways` threads count it
    const int total = static_cast<int>(last - first);
    const uint32_t i = threadIdx.x;
    const uint32_t word = static_cast<int>(i) < total ? static_cast<uint32_t>(token_key(a, first + i)) << 8 | i : 0xFFFFFFFFu;
    sm.unsorted[i] = word;
    __syncthreads();
    int ways = 1;
    while (ways < 32 && 2 * ways * total <= kEmbThreads) ways *= 2;
    const int mine = threadIdx.x / ways;
    const uint32_t me = mine < total ? sm.unsorted[mine] : 0u;
    int place = 0;
    for (int j = threadIdx.x % ways; 4 * j < total; j += ways) {
      const uint4 q = reinterpret_cast<const uint4*>(sm.unsorted)[j];
      place += (q.x < me) + (q.y < me) + (q.z < me) + (q.w < me);
    }
    for (int d = ways / 2; d > 0; d /= 2) place += __shfl_xor_sync(0xFFFFFFFFu, place, d);
    if (mine < total && threadIdx.x % ways == 0) {
      own_keys[place] = static_cast<int>(me >> 8);
      own_pos[place] = static_cast<int>(first) + static_cast<int>(me & 255u);
    }
    __syncthreads();
    const int from = static_cast<int>(lo - first);
    while (skip < m && from + skip > 0 && own_keys[from + skip] == own_keys[from + skip - 1]) ++skip;
    if (skip == m) return;  // no run begins here
    int end = from + m;
    while (end < total && own_keys[end] == own_keys[end - 1]) ++end;
    skip += from;  // the runs are [skip, end)
    while (end > skip && own_keys[end - 1] == a.num_rows) --end;  // tokens without a gradient are last
    n = end - skip;
  } else {
    if (lane < m) {
      key = a.keys[lo + lane];
      at = a.pos[lo + lane];
    }
    if (m > 0 && lo > first) before = a.keys[lo - 1];
    if (m > 0 && lo + m < last) after = a.keys[lo + m];
    n = __popc(__ballot_sync(0xFFFFFFFFu, key != a.num_rows));
  }
  auto key_of = [&](int i) { return SORT ? own_keys[skip + min(i, n - 1)] : __shfl_sync(0xFFFFFFFFu, key, i & 31); };
  auto row_of = [&](int i) { return SORT ? own_pos[skip + min(i, n - 1)] : __shfl_sync(0xFFFFFFFFu, at, i & 31); };
  if (SORT && n == 0) return;
  const T* dy = static_cast<const T*>(a.dy) + c0;
  G* grad = static_cast<G*>(a.grads[k]) + c0;
  // where a row lies, in units of 8 bytes from dy (the host keeps them within 32 bits; N > 1)
  const uint32_t ld8 = static_cast<uint32_t>(a.ld * static_cast<int>(sizeof(T)) / 8);
  const uint32_t at8 = static_cast<uint32_t>(at) * ld8;
  Raw8<T, LAYOUT> held;
  Raw8<G, LAYOUT> held_old;
  int copied = -1;  // key of the last row whose copy was begun (rows below n only)
  if (!SORT && n > 0 && before == __shfl_sync(0xFFFFFFFFu, key, 0)) copied = before;  // (that run's row is not added to here)
  auto copy = [&](int i) {  // row i of the part, and the gradient row of a run that begins there
    bool begins = false;
    int q = 0;
    if constexpr (ADD) {
      q = key_of(i);
      begins = i < n && q != copied;
      if (i < n) copied = q;
    }
    if constexpr (LAYOUT != kStrided) {
      const uint32_t p8 = SORT ? static_cast<uint32_t>(row_of(i)) * ld8 : __shfl_sync(0xFFFFFFFFu, at8, i & 31);
      if (i < n) sm.ring.dy[w][i % kAhead].copy(reinterpret_cast<const T*>(reinterpret_cast<const uint2*>(dy) + p8), left, lane);
      if (begins) sm.ring.old[w][i % kAhead].copy(grad + static_cast<int64_t>(q) * cols, left, lane);
      cp_async_commit();
    } else {
      held = load8<T, LAYOUT>(dy + static_cast<int64_t>(row_of(i)) * a.ld, i < n ? left : 0, lane);
      if constexpr (ADD) held_old = load8<G, LAYOUT>(grad + static_cast<int64_t>(q) * cols, begins ? left : 0, lane);
    }
  };
  constexpr int kLead = LAYOUT != kStrided ? kAhead : 1;
  for (int i = 0; i < kLead; ++i) copy(i);
  F2 acc[4], head[4];
  Raw8<G, LAYOUT> old = {};
  auto clear = [&](F2 (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f2(0.f);
  };
  clear(acc);
  clear(head);
  auto put = [&](int row) {
    put_row<G, LAYOUT, ADD>(grad + static_cast<int64_t>(row) * cols, a.scale, left, lane, acc, old);
  };
  int cur = n > 0 ? key_of(0) : -1, found = 0;
  bool from_before = !SORT && n > 0 && before == cur, fresh = !from_before;
  for (int i = 0;; ++i) {
    const int q = i < n ? key_of(i) : -1;
    if (q != cur || i == n) {  // the run `cur` ends in this part, or the part ends
      if (n == 0) break;
      const bool goes_on = !SORT && i == n && i == m && after == cur;
      if (from_before) {
        found |= goes_on ? kHead | kSpan : kHead;
#pragma unroll
        for (int e = 0; e < 4; ++e) head[e] = acc[e];
      } else if (goes_on) {
        found |= kTail;
      } else {
        put(cur);
      }
      if (i == n) break;
      cur = q;
      from_before = false;
      fresh = true;
      clear(acc);
    }
    F2 v[4];
    if constexpr (LAYOUT != kStrided) {
      cp_async_wait<kAhead - 1>();
      unpack8<T, LAYOUT>(sm.ring.dy[w][i % kAhead].take(lane), v);
      if constexpr (ADD)
        if (fresh) old = sm.ring.old[w][i % kAhead].take(lane);
    } else {
      unpack8<T, LAYOUT>(held, v);
      if constexpr (ADD)
        if (fresh) old = held_old;
    }
    fresh = false;
    add8(acc, v);
    copy(i + kLead);
  }
  if constexpr (!SORT) {
    // runs that cross warps
    const int64_t chunk_end = lo + static_cast<int64_t>(kEmbWarps - w) * a.part;
    if constexpr (LAYOUT != kStrided) cp_async_wait<0>();
    if (lane == 0) {
      ends[w] = found;
      tail_key[w] = cur;
    }
    if (!__syncthreads_or(found)) return;
    if (found & kHead) sts8(sm.piece[w][0], lane, head);
    if (found & kTail) sts8(sm.piece[w][1], lane, acc);
    __syncthreads();
    for (int slot = 0; slot < 2; ++slot) {
      // slot 0: the run that enters the chunk (warp 0's head); slot 1: a run that begins here
      if (!(ends[w] & (slot ? kTail : kHead)) || (slot == 0 && w > 0)) continue;
      lds8(sm.piece[w][slot], lane, acc);
      bool open = slot == 1 || (ends[w] & kSpan);
      int u = w + 1;
      for (; open && u < kEmbWarps && (ends[u] & kHead); ++u) {
        F2 v[4];
        lds8(sm.piece[u][0], lane, v);
        add8(acc, v);
        open = ends[u] & kSpan;
      }
      open = open && u == kEmbWarps && chunk_end < last;
      if (slot == 0 || open) {
        store8<float, LAYOUT>(a.partials + (static_cast<int64_t>(chunk) * 2 + slot) * a.cols + c0, left, lane, acc);
        if (slot == 1 && c0 == 0 && lane == 0) a.list[atomicAdd(a.count, 1)] = static_cast<int>(chunk);
      } else {
        put(tail_key[w]);
      }
    }
  }
}

// Joins the pieces of the runs that cross chunks: one CTA per run and 256 columns, its
// warps taking consecutive parts of the pieces.  Bound by latency (a run's key, its pieces'
// keys, the pieces): 10 us beside 41 of the sums for 16 workers x 4096 tokens x 1024 columns.
template <typename G, int LAYOUT>
__global__ void __launch_bounds__(kEmbThreads) table_join_kernel(const __grid_constant__ TableGradArgs a) {
  pdl_enter();
  constexpr int B = 4;
  __shared__ float part[kEmbWarps][kSlice];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t items = static_cast<int64_t>(*a.count) * a.slices;
  const int64_t span = static_cast<int64_t>(a.part) * kEmbWarps;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int chunk = a.list[item / a.slices];
    const int64_t c0 = item % a.slices * kSlice;
    const int left = slice_left(a.cols, c0);
    const int k = worker_of(a.chunk_off, a.K, chunk);
    const int64_t last = a.off[k + 1];
    const int64_t after = a.off[k] + (chunk + 1 - a.chunk_off[k]) * span;  // start of the next chunk
    const int key = a.keys[after];
    // the chunk's own tail, and the heads of the following chunks that begin inside the run
    int64_t pieces = 1;
    for (;;) {
      const int64_t i = after + (pieces - 1 + lane) * span;
      const unsigned in = __ballot_sync(0xFFFFFFFFu, i < last && a.keys[i] == key);
      pieces += __popc(in);
      if (in != 0xFFFFFFFFu) break;
    }
    const int64_t p0 = pieces * w / kEmbWarps, p1 = pieces * (w + 1) / kEmbWarps;
    F2 acc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = f2(0.f);
    for (int64_t i0 = p0; i0 < p1; i0 += B) {
      Raw8<float, LAYOUT> r[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int64_t i = i0 + b;
        const float* p = a.partials + ((chunk + i) * 2 + (i == 0 ? 1 : 0)) * a.cols + c0;
        r[b] = load8<float, LAYOUT>(p, i < p1 ? left : 0, lane);
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        F2 v[4];
        unpack8<float, LAYOUT>(r[b], v);
        add8(acc, v);
      }
    }
    sts8(part[w], lane, acc);
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int i = 1; i < kEmbWarps; ++i) {
        F2 v[4];
        lds8(part[i], lane, v);
        add8(acc, v);
      }
      G* out = static_cast<G*>(a.grads[k]) + key * a.cols + c0;
      if (a.accumulate) put_row<G, LAYOUT, true>(out, a.scale, left, lane, acc, load8<G, LAYOUT>(out, left, lane));
      else put_row<G, LAYOUT, false>(out, a.scale, left, lane, acc, Raw8<G, LAYOUT>{});
    }
    __syncthreads();
  }
}

template <typename T>
int launch_lookup(const LookupArgs& a, bool vec, unsigned grid, cudaStream_t stream) {
  return launch_pdl(vec ? lookup_kernel<T, kWide<T>> : lookup_kernel<T, kStrided>, dim3(grid), dim3(kEmbThreads), 0, stream, a);
}
template <typename T, typename G, int LAYOUT, bool SORT, bool ADD>
int launch_sum_as(const TableGradArgs& a, unsigned grid, cudaStream_t stream) {
  auto kernel = table_sum_kernel<T, G, LAYOUT, SORT, ADD>;
  constexpr size_t smem = sizeof(SumSmem<T, G, LAYOUT, ADD>);
  static SmemAllowed allowed;
  if (int rc = allow_smem(kernel, smem, allowed)) return rc;
  return launch_pdl(kernel, dim3(grid), dim3(kEmbThreads), smem, stream, a);
}
template <typename T, typename G, int LAYOUT>
int launch_sum_layout(const TableGradArgs& a, bool sort, unsigned grid, cudaStream_t stream) {
  if (a.accumulate)
    return sort ? launch_sum_as<T, G, LAYOUT, true, true>(a, grid, stream) : launch_sum_as<T, G, LAYOUT, false, true>(a, grid, stream);
  return sort ? launch_sum_as<T, G, LAYOUT, true, false>(a, grid, stream) : launch_sum_as<T, G, LAYOUT, false, false>(a, grid, stream);
}
template <typename T, typename G>
int launch_sum(const TableGradArgs& a, bool vec, bool sort, unsigned grid, cudaStream_t stream) {
  constexpr int kBoth = sizeof(T) + sizeof(G) == 4 ? kVec8 : kVec4;
  return vec ? launch_sum_layout<T, G, kBoth>(a, sort, grid, stream) : launch_sum_layout<T, G, kStrided>(a, sort, grid, stream);
}
template <typename G>
int launch_join(const TableGradArgs& a, bool vec, unsigned grid, cudaStream_t stream) {
  return launch_pdl(vec ? table_join_kernel<G, kVec4> : table_join_kernel<G, kStrided>, dim3(grid), dim3(kEmbThreads), 0,
                    stream, a);
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
  if (cols > INT32_MAX || n > INT32_MAX || num_rows > INT32_MAX || num_rows > INT64_MAX / 8 / cols)
    return ADASUM_ERR_UNSUPPORTED;
  if (n == 0) return ADASUM_OK;
  if ((table == nullptr && num_rows > 0) || tokens == nullptr || out == nullptr) return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype);
  BufferSet set;
  set.read(table, num_rows * cols * e, e);
  set.read(tokens, n * token_bytes, token_bytes);
  set.write(out, n * cols * e, e);
  if (adasum_status_t st = set.check()) return st;
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

int64_t adasum_embedding_backward_scratch_bytes(const int64_t* worker_offsets, int K, int64_t num_rows, int64_t cols) {
  if (check_worker_offsets(worker_offsets, K) || num_rows <= 0 || cols <= 0) return 0;
  const int64_t n = worker_offsets[K];
  return n == 0 || self_sorted(worker_offsets, K, num_rows) ? 0 : Scratch(n, cols, K).total;
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
  if (cols > INT32_MAX || n >= INT32_MAX || num_rows >= INT32_MAX || num_rows > INT64_MAX / 8 / cols)
    return ADASUM_ERR_UNSUPPORTED;
  if ((n / (kSelfPart * kEmbWarps) + K) * ((cols + kSlice - 1) / kSlice) > INT32_MAX) return ADASUM_ERR_UNSUPPORTED;
  if (num_rows == 0) return ADASUM_OK;
  if (grads == nullptr || (n > 0 && (grad_out == nullptr || tokens == nullptr || !valid_ld(n, cols, ld))))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t need = adasum_embedding_backward_scratch_bytes(worker_offsets, K, num_rows, cols);
  if (need > 0 && (scratch == nullptr || scratch_bytes < need || !is_aligned(scratch, 256)))
    return ADASUM_ERR_INVALID_ARG;
  const int64_t e = dtype_bytes(dtype), ge = dtype_bytes(grad_dtype);
  SortArgs s = {};
  TableGradArgs a = {};
  BufferSet set;
  set.read(grad_out, span_bytes(n, cols, ld, e), e);
  set.read(tokens, n * token_bytes, token_bytes);
  set.write(scratch, need, 256);
  // vectors: pieces of eight columns where both types are bf16, else of four, on their own
  // boundaries (and rows of grad_out addressed by 32 bits of 8-byte units)
  const int piece = e + ge == 4 ? 8 : 4;
  bool vec = is_aligned(grad_out, piece * e) && ld % piece == 0 && cols % piece == 0 &&
             span_bytes(n, cols, ld, e) < (int64_t(8) << 32);
  int64_t most = 0;
  for (int k = 0; k < K; ++k) most = std::max(most, worker_offsets[k + 1] - worker_offsets[k]);
  const bool self_sort = self_sorted(worker_offsets, K, num_rows);
  a.part = self_sort ? kSelfPart : warp_tokens(n, cols);
  const int64_t span = static_cast<int64_t>(a.part) * kEmbWarps;
  for (int k = 0; k < K; ++k) {
    if (grads[k] == nullptr) return ADASUM_ERR_INVALID_ARG;
    set.write(grads[k], num_rows * cols * ge, ge);
    vec = vec && is_aligned(grads[k], piece * ge);
    const int64_t nk = worker_offsets[k + 1] - worker_offsets[k];
    s.fill[k] = a.grads[k] = grads[k];
    s.off[k + 1] = a.off[k + 1] = worker_offsets[k + 1];
    s.tile_off[k + 1] = s.tile_off[k] + static_cast<int>((nk + kTile - 1) / kTile);
    a.chunk_off[k + 1] = a.chunk_off[k] + static_cast<int>((nk + span - 1) / span);
  }
  if (adasum_status_t st = set.check()) return st;
  if (n == 0) {  // nothing to sum: zero the gradients, or leave them
    if (accumulate) return ADASUM_OK;
    for (int k = 0; k < K; ++k)
      if (cudaMemsetAsync(grads[k], 0, static_cast<size_t>(num_rows * cols * ge), stream) != cudaSuccess)
        return ADASUM_ERR_CUDA;
    return ADASUM_OK;
  }
  const Scratch at(n, cols, K);
  char* base = need > 0 ? static_cast<char*>(scratch) : nullptr;
  auto ints = [&](int64_t offset) { return base ? reinterpret_cast<int*>(base + offset) : nullptr; };
  // digits: as few passes of at most 8 bits as the keys 0..num_rows need
  int bits = 1;
  while ((num_rows >> bits) != 0) ++bits;
  s.tokens = a.tokens = tokens;
  s.token_bytes = a.token_bytes = token_bytes;
  s.num_rows = a.num_rows = static_cast<int>(num_rows);
  s.padding_idx = a.padding_idx = padding_idx;
  s.K = a.K = K;
  s.passes = (bits + 7) / 8;
  s.bits = (bits + s.passes - 1) / s.passes;
  s.hist = ints(at.hist);
  s.join_count = ints(at.count);
  s.fill_bytes = accumulate ? 0 : num_rows * cols * ge;
  const int64_t piece_bytes = static_cast<int64_t>(!self_sort && most <= kSortMost ? kSortThreads : kTileThreads) * kFillVecs * 16;
  s.fill_pieces = (s.fill_bytes + piece_bytes - 1) / piece_bytes;
  const int64_t pieces = K * s.fill_pieces;
  if (pieces > INT32_MAX / 2) return ADASUM_ERR_UNSUPPORTED;
  const double fill = static_cast<double>(K) * s.fill_bytes;
  int out = 0;  // which half of the key and position buffers holds the result
  if (self_sort) {
    if (!accumulate)
      if (adasum_status_t st = counted_launch(stream, "table_fill", fill, [&] {
            return launch_pdl(table_fill_kernel, dim3(static_cast<unsigned>(pieces)), dim3(kTileThreads), 0, stream, s);
          }))
        return st;
  } else if (most <= kSortMost) {
    s.keys = ints(at.keys[0]);
    s.pos = ints(at.pos[0]);
    if (adasum_status_t st = counted_launch(stream, "table_sort", fill, [&] {
          static SmemAllowed allowed;
          constexpr size_t smem = sizeof(SortSmem<kSortThreads, kSortItems>);
          if (int rc = allow_smem(table_sort_kernel, smem, allowed)) return rc;
          return launch_pdl(table_sort_kernel, dim3(static_cast<unsigned>(K + pieces)), dim3(kSortThreads), smem, stream, s);
        }))
      return st;
  } else {
    s.ntiles = s.tile_off[K];
    s.totals = most > static_cast<int64_t>(kScanTiles) * kTile ? ints(at.totals) : nullptr;
    if (adasum_status_t st = counted_launch(stream, "table_count", 0.0, [&] {
          return launch_pdl(table_count_kernel, dim3(s.ntiles), dim3(kTileThreads), 0, stream, s);
        }))
      return st;
    for (s.pass = 0; s.pass < s.passes; ++s.pass) {
      out = s.pass & 1;
      s.shift = s.pass * s.bits;
      s.keys_in = s.pass > 0 ? ints(at.keys[1 - out]) : nullptr;
      s.pos_in = s.pass > 0 ? ints(at.pos[1 - out]) : nullptr;
      s.keys = ints(at.keys[out]);
      s.pos = ints(at.pos[out]);
      if (s.totals)
        if (adasum_status_t st = counted_launch(stream, "table_scan", 0.0, [&] {
              return launch_pdl(table_scan_kernel, dim3(static_cast<unsigned>(K * (kDigits / 32))), dim3(kSortThreads), 0, stream, s);
            }))
          return st;
      s.fill_first = pieces * s.pass / s.passes;
      const int64_t share = pieces * (s.pass + 1) / s.passes - s.fill_first;
      if (adasum_status_t st = counted_launch(stream, "table_scatter", fill / s.passes, [&] {
            return launch_pdl(table_scatter_kernel, dim3(static_cast<unsigned>(s.ntiles + share)), dim3(kTileThreads), 0, stream, s);
          }))
        return st;
    }
  }
  a.dy = grad_out;
  a.cols = cols;
  a.ld = ld;
  a.scale = scale;
  a.accumulate = accumulate != 0;
  a.slices = static_cast<int>((cols + kSlice - 1) / kSlice);
  a.keys = ints(at.keys[out]);
  a.pos = ints(at.pos[out]);
  a.count = ints(at.count);
  a.list = ints(at.list);
  a.partials = base ? reinterpret_cast<float*>(base + at.partials) : nullptr;
  const int64_t items = static_cast<int64_t>(a.chunk_off[K]) * a.slices;
  const unsigned grid = static_cast<unsigned>(items);
  if (adasum_status_t st = counted_launch(stream, "table_sum", static_cast<double>(n) * (cols * e + 8), [&] {
        if (dtype == ADASUM_BF16)
          return grad_dtype == ADASUM_BF16 ? launch_sum<bf16, bf16>(a, vec, self_sort, grid, stream)
                                           : launch_sum<bf16, float>(a, vec, self_sort, grid, stream);
        return grad_dtype == ADASUM_BF16 ? launch_sum<float, bf16>(a, vec, self_sort, grid, stream)
                                         : launch_sum<float, float>(a, vec, self_sort, grid, stream);
      }))
    return st;
  if (self_sort || most <= span) return ADASUM_OK;  // no run crosses chunks
  const unsigned joiners = static_cast<unsigned>(std::min<int64_t>(items, 4 * static_cast<int64_t>(sm_count())));
  return counted_launch(stream, "table_join", 0.0, [&] {
    return grad_dtype == ADASUM_BF16 ? launch_join<bf16>(a, vec, joiners, stream) : launch_join<float>(a, vec, joiners, stream);
  });
}

}  // extern "C"
