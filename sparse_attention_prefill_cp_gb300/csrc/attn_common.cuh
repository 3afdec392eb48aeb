// What the attention kernels over caches share: exponentials and maxima, waits
// without calls, TMEM loads by width, bulk copies of results.
#pragma once

#include "dsa_common.cuh"

namespace dsa {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// mbar_wait without a call, for the loops that hold most of the registers:
// bounded by the same time, the failing site and detail noted in shared memory.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, int32_t *failed, int site, int detail = 0) {
  if (kCluster ? mbar_try_wait_hint_cluster(bar, parity) : mbar_try_wait_hint(bar, parity)) return true;
  const long long t0 = clock64();
  do {
    if (kCluster ? mbar_try_wait_hint_cluster(bar, parity) : mbar_try_wait_hint(bar, parity)) return true;
  } while (clock64() - t0 < kWaitLimitCycles);
  *failed = site << 24 | (detail & 0xffffff);
  return false;
}

// Columns of the warp's own TMEM lanes.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32]) { tmem_st32(taddr, r); }
#define DSA_OUT8(b) "=r"(r[b + 0]), "=r"(r[b + 1]), "=r"(r[b + 2]), "=r"(r[b + 3]), "=r"(r[b + 4]), "=r"(r[b + 5]), \
                    "=r"(r[b + 6]), "=r"(r[b + 7])
#define DSA_IN8(b) "r"(r[b + 0]), "r"(r[b + 1]), "r"(r[b + 2]), "r"(r[b + 3]), "r"(r[b + 4]), "r"(r[b + 5]), \
                   "r"(r[b + 6]), "r"(r[b + 7])
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : DSA_OUT8(0), DSA_OUT8(8)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      DSA_IN8(0), DSA_IN8(8)
      : "memory");
}
#undef DSA_OUT8
#undef DSA_IN8

// The bulk copy of a result out of shared memory.
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// Until this thread's bulk copies are complete, not only read: the join of the
// parts may be resident before this kernel has ended.
__device__ __forceinline__ void bulk_wait_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace dsa
