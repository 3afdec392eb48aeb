// Attention over the 4-bit cache, more queries than run at once: the order in
// which they are started.
#include "sparse_attn_int4.cuh"
#include "internal.h"

namespace dsa {
namespace {

// Longest list first.  What runs last in a call is what starts last, so a long
// list behind short ones keeps a few SMs busy alone.  A list's length is the
// last of 32 positions, evenly spread, that holds an entry; it need not be
// exact, and neither it nor the order among equals (shared-memory atomics)
// changes any result.  One block: a warp samples a query, a lane a position;
// then a counting sort over the 33 lengths.  The attention is launched while
// this runs and waits before it reads the order.
__global__ void __launch_bounds__(kInt4MaxOrdered)
    sparse_attn_int4_order_kernel(const int32_t *__restrict__ idx, const int32_t *__restrict__ q_rows, int n, int topk,
                                  int32_t *__restrict__ order) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint8_t length[kInt4MaxOrdered];
  __shared__ int32_t count[64];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kInt4MaxOrdered / 32;
  if (tid < 64) count[tid] = 0;
  const int k = max(static_cast<int>(static_cast<int64_t>(lane + 1) * topk / 32) - 1, 0);
#pragma unroll 1
  for (int i0 = warp; i0 < n; i0 += 8 * kWarps) {
    int e[8], r[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int i = i0 + x * kWarps;
      e[x] = i < n ? __ldg(idx + static_cast<int64_t>(i) * topk + k) : -1;
      r[x] = i < n && q_rows ? __ldg(q_rows + i) : 0;
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int i = i0 + x * kWarps;
      const unsigned used = __ballot_sync(0xffffffffu, e[x] >= 0 && r[x] >= 0);
      if (lane == 0 && i < n) length[i] = static_cast<uint8_t>(32 - __clz(used));
    }
  }
  __syncthreads();
  const int mine = tid < n ? length[tid] : 0;
  int rank = 0;
  if (tid < n) rank = atomicAdd(&count[mine], 1);
  __syncthreads();
  if (tid < n) {
    int start = 0;
    for (int c = mine + 1; c <= 32; ++c) start += count[c];
    order[start + rank] = tid;
  }
}

}  // namespace

dsa_status launch_attn_int4_order(int32_t n, const AttnInt4Params &P, int32_t *order, cudaStream_t stream) {
  sparse_attn_int4_order_kernel<<<1, kInt4MaxOrdered, 0, stream>>>(P.idx, P.q_rows, n, P.topk, order);
  return check_launch();
}

}  // namespace dsa
