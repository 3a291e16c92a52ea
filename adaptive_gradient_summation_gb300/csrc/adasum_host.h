// adasum_host.h -- host-side helpers of the training operators (train_*.cu): the launch
// count and profiler they share with adasum_api.cu, and their argument checks.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include "../../include/adasum.h"
#include "adasum_internal.h"

namespace adasum {

// Serialises every entry point (the launch count and the profiler's record).
std::mutex& entry_mutex();
// Start event of a launch when the profiler is on (else null), and the record of it.
cudaEvent_t profile_start(cudaStream_t stream);
adasum_status_t profile_launched(int rc, const char* name, cudaEvent_t start, cudaStream_t stream,
                                 double bytes);

// One launch, counted and (when profiling) timed; `f` returns the launch's cudaError_t as
// int.  `bytes`: its algorithmic bytes.
template <typename F>
adasum_status_t counted_launch(cudaStream_t stream, const char* name, double bytes, F&& f) {
  cudaEvent_t e = profile_start(stream);
  return profile_launched(f(), name, e, stream, bytes);
}

// An entry point's lock and NVTX range.
struct EntryScope {
  explicit EntryScope(const char* name) : lock(entry_mutex()) { nvtxRangePushA(name); }
  ~EntryScope() { nvtxRangePop(); }
  EntryScope(const EntryScope&) = delete;
  EntryScope& operator=(const EntryScope&) = delete;
  std::lock_guard<std::mutex> lock;
};

inline bool valid_dtype(int dt) { return dt == kF32 || dt == kBF16; }
inline int64_t dtype_bytes(int dt) { return dt == kBF16 ? 2 : 4; }
inline bool is_aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Buffers of one call, each with the size of its elements.  `bad`: one does not start on an
// element's boundary; `conflict`: a written one overlaps another.
struct BufferSet {
  static constexpr int kMost = 2 * kMaxK + 16;
  struct Range {
    uintptr_t lo, hi;
    bool written;
  } r[kMost];
  int n = 0;
  bool bad = false;

  void read(const void* p, int64_t bytes, int64_t elem) { add(p, bytes, elem, false); }
  void write(const void* p, int64_t bytes, int64_t elem) { add(p, bytes, elem, true); }
  void add(const void* p, int64_t bytes, int64_t elem, bool written) {
    if (p == nullptr || bytes <= 0) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    bad = bad || (lo & static_cast<uintptr_t>(elem - 1)) != 0;
    r[n++] = Range{lo, lo + static_cast<uintptr_t>(bytes), written};
  }
  bool conflict() {
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t end_any = 0, end_written = 0;
    for (int i = 0; i < n; ++i) {
      if (r[i].lo < (r[i].written ? end_any : end_written)) return true;
      end_any = std::max(end_any, r[i].hi);
      if (r[i].written) end_written = std::max(end_written, r[i].hi);
    }
    return false;
  }
  adasum_status_t check() { return bad ? ADASUM_ERR_INVALID_ARG : conflict() ? ADASUM_ERR_ALIAS : ADASUM_OK; }
};

// Whether rows `ld` apart can be addressed, and the bytes a strided input of them spans.
inline bool valid_ld(int64_t rows, int64_t cols, int64_t ld) {
  return ld >= cols && (rows <= 1 || ld <= INT64_MAX / 16 / rows);
}
inline int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  return rows > 0 ? ((rows - 1) * ld + cols) * elem : 0;
}

// worker_offsets of a call: K+1 values from 0, non-decreasing.
inline adasum_status_t check_worker_offsets(const int64_t* offs, int K) {
  if (offs == nullptr || K < 1) return ADASUM_ERR_INVALID_ARG;
  if (K > kMaxK) return ADASUM_ERR_UNSUPPORTED;
  if (offs[0] != 0) return ADASUM_ERR_INVALID_ARG;
  for (int k = 0; k < K; ++k)
    if (offs[k + 1] < offs[k]) return ADASUM_ERR_INVALID_ARG;
  return ADASUM_OK;
}

// SMs of the current device (asked once per device).
inline int sm_count() {
  static std::atomic<int> known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (dev < 0 || dev >= 64) dev = 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Allows a kernel `bytes` of dynamic shared memory where that is (with its static part) more
// than the default 48 KiB; asked of the runtime once per device.  `known` belongs to the
// kernel and its size.
struct SmemAllowed {
  bool on[64] = {};
};
template <typename Kernel>
int allow_smem(Kernel* kernel, size_t bytes, SmemAllowed& known) {
  if (bytes <= 40 * 1024) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return static_cast<int>(cudaErrorInvalidDevice);
  if (dev >= 0 && dev < 64 && known.on[dev]) return 0;
  const cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (rc == cudaSuccess && dev >= 0 && dev < 64) known.on[dev] = true;
  return static_cast<int>(rc);
}

}  // namespace adasum
