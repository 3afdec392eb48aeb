// Attention over the 4-bit cache with its entries split: the join of the parts.
#include "sparse_attn_int4.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kDv = kInt4Dv;

// Join the splits of one query and head: the parts' weights are e^(m_s - m)
// with m their largest, the sum runs in split order.  One block per (query,
// head), a thread on four value columns, the loads of up to N parts in flight
// together (a part without entries was not written: its values are dropped);
// the weights come from one pass of the warps' lanes over the parts' (m, l).
template <int N>
__global__ void __launch_bounds__(128) sparse_attn_int4_join_kernel(const AttnInt4Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the first kernel may still run
  const int query = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, half = threadIdx.x >> 6;
  const int qrow = P.q_rows ? P.q_rows[query] : query;
  if (qrow < 0 || qrow >= P.num_q_rows) return;  // the latter reported by the first kernel
  const int64_t first = static_cast<int64_t>(query) * P.splits * P.H + h;
  const float4 *o = reinterpret_cast<const float4 *>(P.part_o + first * kDv) + threadIdx.x;
  const int64_t step = static_cast<int64_t>(P.H) * (kDv / 4);
  float4 x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = o[min(k, P.splits - 1) * step];
  float2 t = make_float2(-__builtin_huge_valf(), 0.f);
  if (lane < P.splits) t = P.part_ml[2 * (first + static_cast<int64_t>(lane) * P.H) + half];
  const float m = warp_max(t.x);
  const unsigned parts = __ballot_sync(0xffffffffu, t.y != 0.f);
  const float wgt = t.y != 0.f ? ex2(t.x - (m == -__builtin_huge_valf() ? 0.f : m)) : 0.f;
  float l = P.sink ? ex2(P.sink[h] * 1.4426950408889634f - m) : 0.f;
  const float wl = t.y != 0.f ? wgt * t.y : 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float w = __shfl_sync(0xffffffffu, wgt, k);
    l += __shfl_sync(0xffffffffu, wl, k);
    if ((parts >> k) & 1u) {
      acc.x += w * x[k].x;
      acc.y += w * x[k].y;
      acc.z += w * x[k].z;
      acc.w += w * x[k].w;
    }
  }
  const float inv = parts && l != 0.f ? 1.f / l : 0.f;
  const uint2 r = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2 *>(P.out + (static_cast<int64_t>(qrow) * P.H + h) * kDv + 4 * threadIdx.x) = r;
}

}  // namespace

dsa_status launch_attn_int4_join(int32_t n, const AttnInt4Params &P, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n), static_cast<unsigned>(P.H));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = P.splits <= 8    ? cudaLaunchKernelEx(&cfg, sparse_attn_int4_join_kernel<8>, P)
                        : P.splits <= 16 ? cudaLaunchKernelEx(&cfg, sparse_attn_int4_join_kernel<16>, P)
                                         : cudaLaunchKernelEx(&cfg, sparse_attn_int4_join_kernel<32>, P);
  if (e != cudaSuccess) return cuda_fail(e);
  return check_launch();
}

}  // namespace dsa
