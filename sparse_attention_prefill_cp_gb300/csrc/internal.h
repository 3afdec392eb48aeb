// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/dsa_cp.h"

namespace dsa {

// Device address of the library's error word on the current device (set up
// once per device); nullptr if the lookup failed (the CUDA error is recorded).
int *device_error_word();

// Record `e` as the last CUDA error of this thread and return DSA_ERR_CUDA.
dsa_status cuda_fail(cudaError_t e);
dsa_status cuda_fail_msg(const char *msg);

// Launch-error check after a kernel launch.
inline dsa_status check_launch() {
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}

// Shared memory beyond 48 KB for a kernel, asked for once per device (a call of it
// costs the host half a microsecond).
template <typename... Params>
cudaError_t allow_smem(void (*kernel)(Params...), int bytes, std::atomic<uint64_t> &devices) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (devices.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch of a kernel that may become resident while the kernel before it in the
// stream still runs: it touches memory only behind griddepcontrol.wait, and reads it
// with plain loads.  A read-only load (__ldg, ld.global.nc) is for what nobody writes
// while the kernel is there; it may be moved ahead of the wait and need not see what
// the kernel before wrote.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                              const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).
// rank <= 3; dims/strides in elements/bytes as the driver API expects
// (strides exclude the innermost dimension).
dsa_status encode_tensor_map(CUtensorMap *map, CUtensorMapDataType dtype, uint32_t rank, const void *base,
                             const uint64_t *dims, const uint64_t *strides_bytes, const uint32_t *box,
                             CUtensorMapSwizzle swizzle);

int num_sms();

// log2 of a page size of the paged latent cache (16, 32, 64 or 128 rows), -1 of any other.
int page_shift(int32_t page_size);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace dsa
