// Attention over the paged cache: the join of the parts of queries whose blocks
// lie in more than one unit.
#include "internal.h"
#include "paged_attn.cuh"

namespace dsa {
namespace {

constexpr int kBatch = 8;  // parts whose loads are in flight together

// One block per (unit, head): the query that starts in that unit and ends in a
// later one, if there is one, from its parts in the units' order.  Part 2u + 1 is
// of the query that starts in unit u, part 2u of the one that goes on there.  The
// weights are e^(m_s - m) with m the largest; a thread has four value columns.
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedAttnParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the first kernel may still run
  const int unit = blockIdx.x, h = blockIdx.y;
  const int2 join = P.joins[unit];
  if (join.x < 0) return;
  const int parts = join.y - unit + 1;
  auto part = [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * unit + 1 : 2 * (unit + k)) * P.H + h; };
  float m = -__builtin_huge_valf();
  for (int k0 = 0; k0 < parts; k0 += 32) {
    const int k = k0 + (threadIdx.x & 31);
    m = fmaxf(m, warp_max(k < parts ? P.part_ml[part(k)].x : -__builtin_huge_valf()));
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int k0 = 0; k0 < parts; k0 += kBatch) {
    float4 x[kBatch];
    float2 ml[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t p = part(min(k0 + k, parts - 1));
      x[k] = *(reinterpret_cast<const float4 *>(P.part_o + p * kPagedDv) + threadIdx.x);
      ml[k] = P.part_ml[p];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      // a part of masked rows alone has l = 0; a NaN among its logits is a NaN in l
      if (k0 + k < parts && ml[k].y != 0.f) {
        const float w = ex2(ml[k].x - (m == -__builtin_huge_valf() ? 0.f : m));
        l += w * ml[k].y;
        acc.x += w * x[k].x;
        acc.y += w * x[k].y;
        acc.z += w * x[k].z;
        acc.w += w * x[k].w;
      }
    }
  }
  const bool empty = l == 0.f;
  if (P.sink && !empty) l += ex2(P.sink[h] * 1.4426950408889634f - m);
  const float inv = empty ? 0.f : 1.f / l;
  const uint2 r = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2 *>(P.out + (static_cast<int64_t>(join.x) * P.H + h) * kPagedDv + 4 * threadIdx.x) = r;
}

}  // namespace

dsa_status launch_paged_join(const PagedAttnParams &P, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(P.units), static_cast<unsigned>(P.H));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_join_kernel, P);
  if (e != cudaSuccess) return cuda_fail(e);
  return check_launch();
}

}  // namespace dsa
