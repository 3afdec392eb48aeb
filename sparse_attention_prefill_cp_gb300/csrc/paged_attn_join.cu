// Attention over the paged cache: the join of the parts of queries whose blocks
// lie in more than one unit.
#include "internal.h"
#include "paged_attn.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kTeam = kPagedDv / 4;     // threads on a head's values, four columns each
constexpr int kTeams = kThreads / kTeam;
constexpr int kBatch = 4;               // parts whose loads are in flight together
constexpr int kBlocksPerSm = 2;

// A unit's join is that of the query that starts in it and ends in a later one,
// from the query's parts in the units' order.  Part 2u + 1 is of the query that
// starts in unit u, part 2u of the one that goes on there.  The weights are
// e^(m_s - m) with m the largest.  As many blocks as the SMs hold go through the
// joins, a team of a block a head at a time; where there are so few joins (one
// long request: 74 parts a head) that the blocks would suffice for a head each, a
// block takes a quarter of a head's columns, its warps every 16th part, and their
// sums are added in the warps' order.  The values of the first parts are requested
// before the maximum is known.  What bounds it: the parts, read once, and below
// that two barriers and two dependent loads.
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) paged_join_kernel(const PagedAttnParams P) {
  __shared__ int32_t units[kThreads];
  __shared__ int32_t counts[kWarps];
  __shared__ float4 sums[kWarps][32];
  __shared__ float lsum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the first kernel may still run
  // the units with a join, in order
  const bool has = tid < P.units && P.joins[tid].x >= 0;
  const uint32_t those = __ballot_sync(0xffffffffu, has);
  if (lane == 0) counts[warp] = __popc(those);
  __syncthreads();
  int n = 0, at = __popc(those & ((1u << lane) - 1u));
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    if (k < warp) at += counts[k];
    n += counts[k];
  }
  if (has) units[at] = tid;
  __syncthreads();
  const bool wide = n * P.H <= static_cast<int>(gridDim.x);
  const int team = wide ? warp : tid / kTeam, step = wide ? kWarps : 1, first = wide ? warp : 0;
  const int per = wide ? 4 : 1;  // items of a block's turn: quarters of a head, or one for each team
  const int items = n * P.H * per;
  for (int item = wide ? blockIdx.x : blockIdx.x * kTeams + team; item < items; item += gridDim.x * (wide ? 1 : kTeams)) {
    const int vh = wide ? item >> 2 : item, v = vh / P.H, h = vh - v * P.H;
    const int unit = units[v];
    const int col = wide ? (item & 3) * 32 + lane : tid % kTeam;
    const int2 join = P.joins[unit];
    const int parts = join.y - unit + 1;
    auto part = [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * unit + 1 : 2 * (unit + k)) * P.H + h; };
    float4 x[kBatch];
    float2 ml[kBatch];
    auto request = [&](int k0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t p = part(min(k0 + k * step, parts - 1));
        x[k] = *(reinterpret_cast<const float4 *>(P.part_o + p * kPagedDv) + col);
        ml[k] = P.part_ml[p];
      }
    };
    request(first);
    float m = -__builtin_huge_valf();
    for (int k0 = 0; k0 < parts; k0 += 32) {
      const int k = k0 + lane;
      m = fmaxf(m, warp_max(k < parts ? P.part_ml[part(k)].x : -__builtin_huge_valf()));
    }
    const float base = m == -__builtin_huge_valf() ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int k0 = first; k0 < parts; k0 += kBatch * step) {
      if (k0 != first) request(k0);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        // a part of masked rows alone has l = 0; a NaN among its logits is a NaN in l
        if (k0 + k * step < parts && ml[k].y != 0.f) {
          const float w = ex2(ml[k].x - base);
          l += w * ml[k].y;
          acc.x += w * x[k].x;
          acc.y += w * x[k].y;
          acc.z += w * x[k].z;
          acc.w += w * x[k].w;
        }
      }
    }
    if (wide) {  // an item is the whole block's here, so all threads come by
      sums[warp][lane] = acc;
      if (lane == 0) lsum[warp] = l;
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int t = 1; t < kWarps; ++t) {
          const float4 y = sums[t][lane];
          acc.x += y.x;
          acc.y += y.y;
          acc.z += y.z;
          acc.w += y.w;
          l += lsum[t];
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const bool empty = l == 0.f;
    if (P.sink && !empty) l += ex2(P.sink[h] * 1.4426950408889634f - m);
    const float inv = empty ? 0.f : 1.f / l;
    const uint2 r = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2 *>(P.out + (static_cast<int64_t>(join.x) * P.H + h) * kPagedDv + 4 * col) = r;
  }
}

}  // namespace

dsa_status launch_paged_join(const PagedAttnParams &P, cudaStream_t stream) {
  const int64_t most = (static_cast<int64_t>(P.units) * P.H + kTeams - 1) / kTeams, fit = kBlocksPerSm * num_sms();
  const cudaError_t e = launch_overlapped(paged_join_kernel, dim3(static_cast<unsigned>(most < fit ? most : fit)), kThreads,
                                          0, stream, P);
  return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

}  // namespace dsa
