// adasum_umma.cuh -- inline-PTX wrappers of the fifth-generation tensor cores (tcgen05), their
// tensor memory (TMEM), and tiled TMA copies, for sm_103a.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "adasum_ptx.cuh"

namespace adasum {

// True in one lane of a whole warp, always the same.  (Instructions of one thread issued under
// `lane == 0` instead cost the copying and multiplying warps about twice the time: the compiler
// does not see that their operands are uniform.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// ------------------------------------------------------------------------ tiled copies

// CTAS = 2: a pair of CTAs on neighbouring SMs (a cluster of two) works on one product of twice
// the rows; the even one, the pair's first, issues the instructions.

// Address of the same place in the pair's first CTA, for barriers there.
template <int CTAS>
__device__ __forceinline__ uint32_t first_of_pair(uint32_t addr) {
  if constexpr (CTAS == 1) return addr;
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// One box of a three-dimensional tensor map into this CTA's shared memory, its bytes counted
// on the barrier at `bar` (of this CTA, or of the pair's first).  x * element size must be a
// multiple of 16 bytes.
template <int CTAS>
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  if constexpr (CTAS == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// Ordinary writes that this thread has seen become visible to its later asynchronous copies.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// ---------------------------------------------------------------------- tensor memory

// Whole warp (CTAS = 2: one of each CTA); COLS a power of two from 32 to 512.  The address comes
// back in *slot.
template <int COLS, int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot) {
  if constexpr (CTAS == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int COLS, int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t addr) {
  if constexpr (CTAS == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS) : "memory");
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// N columns (16 or 32) of this warp's 32 lanes: lane l holds row l of the warp's quarter.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[N]) {
  static_assert(N == 16 || N == 32, "columns of one load");
  uint32_t r[N];
  if constexpr (N == 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16 % N]), "=r"(r[17 % N]), "=r"(r[18 % N]),
          "=r"(r[19 % N]), "=r"(r[20 % N]), "=r"(r[21 % N]), "=r"(r[22 % N]), "=r"(r[23 % N]), "=r"(r[24 % N]), "=r"(r[25 % N]),
          "=r"(r[26 % N]), "=r"(r[27 % N]), "=r"(r[28 % N]), "=r"(r[29 % N]), "=r"(r[30 % N]), "=r"(r[31 % N])
        : "r"(addr)
        : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
// The same times `gain`, added to v.
template <int N>
__device__ __forceinline__ void tmem_add(uint32_t addr, float (&v)[N], float gain) {
  float w[N];
  tmem_load<N>(addr, w);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __fmaf_rn(w[i], gain, v[i]);
}

// ------------------------------------------------------------------- matrix products

// Shared-memory operand of 16-bit elements with the 128-byte swizzle that TMA wrote, as the two
// words of its descriptor.
// K-major: rows of 64 elements along k, 128 bytes apart; 16 along k further: +32 bytes.
// MN-major: blocks of 64 rows of the product, each 64 k-lines of 128 bytes; 16 along k
// further: +2048 bytes.  `block`: bytes between two blocks of 64 (MN-major only).
// (Addresses count in units of 16 bytes, and fit the low word's 14 bits.)
__device__ __forceinline__ uint32_t umma_low(uint32_t addr, uint32_t block) { return (addr >> 4) | ((block >> 4) << 16); }
constexpr uint32_t kUmmaHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
// fp16 operands, fp32 accumulator of 128 * ctas x n; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t umma_idesc(int ctas, int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 * ctas >> 4) << 24);
}
// a, b: low words of the operands' descriptors.
template <int CTAS>
__device__ __forceinline__ void umma_f16(uint32_t tmem, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.u32 p, %4, 0;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(add ? 1u : 0u), "r"(kUmmaHigh)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.u32 p, %4, 0;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(add ? 1u : 0u), "r"(kUmmaHigh)
        : "memory");
}
// Arrives on `bar` (CTAS = 2: on both CTAs' at that place) once this thread's products so far
// are done.
template <int CTAS>
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_addr(bar)),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}
// One arrival on the barrier at `addr`, this CTA's or the pair's first's.
template <int CTAS>
__device__ __forceinline__ void mbar_arrive_at(uint32_t addr) {
  if constexpr (CTAS == 1) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(addr) : "memory");
  else asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Whether the phase is over, with what the pair did before its arrivals visible.
template <int CTAS>
__device__ __forceinline__ bool mbar_try_wait_pair(uint64_t* bar, uint32_t parity) {
  if constexpr (CTAS == 1) return mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

}  // namespace adasum
