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

// Part k of the query that starts in `unit`, of head h: part 2u + 1 is of the query
// that starts in unit u, part 2u of the one that goes on there.
__device__ __forceinline__ int64_t part_at(const PagedAttnParams &P, int unit, int h, int k) {
  return static_cast<int64_t>(k == 0 ? 2 * unit + 1 : 2 * (unit + k)) * P.H + h;
}

__device__ __forceinline__ void add_part(float4 &acc, const float4 &x, float w) {
  acc.x += w * x.x;
  acc.y += w * x.y;
  acc.z += w * x.z;
  acc.w += w * x.w;
}

__device__ __forceinline__ void store_head(const PagedAttnParams &P, int query, int h, int col, const float4 &acc, float l,
                                           float m) {
  const bool empty = l == 0.f;
  if (P.sink && !empty) l += ex2(P.sink[h] * 1.4426950408889634f - m);
  const float inv = empty ? 0.f : 1.f / l;
  *reinterpret_cast<uint2 *>(P.out + (static_cast<int64_t>(query) * P.H + h) * kPagedDv + 4 * col) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// What a block's warps share.
struct JoinShared {
  int4 list[kThreads];    // the units with a join, in order: unit, query, last unit
  int32_t counts[kWarps];
  float weight[kThreads], wsum[kWarps], wmax[kWarps];
  float4 sums[kWarps][kTeam];
};

// One head by a whole block, or NC of the four quarters of its columns from quarter
// c0 on: warp w takes parts w, w + 16, ..; their sums are added in the warps' order.
template <int NC>
__device__ __forceinline__ void join_wide(const PagedAttnParams &P, JoinShared &s, int4 join, int h, int c0) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, unit = join.x, parts = join.z - unit + 1;
  float4 x[2][NC];  // of the next two parts
  auto request = [&](float4 (&y)[NC], int k) {
    const float4 *p = reinterpret_cast<const float4 *>(P.part_o + part_at(P, unit, h, min(k, parts - 1)) * kPagedDv);
#pragma unroll
    for (int c = 0; c < NC; ++c) y[c] = p[32 * (c0 + c) + lane];
  };
  request(x[0], warp);
  if (NC < 4) request(x[1], warp + kWarps);
  const float2 ml = tid < parts ? P.part_ml[part_at(P, unit, h, tid)] : make_float2(-__builtin_huge_valf(), 0.f);
  float m = warp_max(ml.x);
  if (lane == 0) s.wmax[warp] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWarps; ++k) m = fmaxf(m, s.wmax[k]);
  const float base = m == -__builtin_huge_valf() ? 0.f : m;
  // a part of masked rows alone has l = 0; a NaN among its logits is a NaN in l
  const float w = ml.y != 0.f ? ex2(ml.x - base) : 0.f;
  s.weight[tid] = w;
  float l = ml.y != 0.f ? w * ml.y : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) s.wsum[warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) l += s.wsum[k];
  float4 acc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = warp; k < parts; k += kWarps) {
    float4 now[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) now[c] = x[0][c];
    if (NC < 4) {
#pragma unroll
      for (int c = 0; c < NC; ++c) x[0][c] = x[1][c];
      request(x[1], k + 2 * kWarps);
    } else {
      request(x[0], k + kWarps);
    }
    const float wk = s.weight[k];
    if (wk != 0.f) {  // a masked part's values are not looked at
#pragma unroll
      for (int c = 0; c < NC; ++c) add_part(acc[c], now[c], wk);
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) s.sums[warp][32 * c + lane] = acc[c];
  __syncthreads();
  if (tid >= 32 * NC) return;
  float4 all = s.sums[0][tid];
#pragma unroll
  for (int t = 1; t < kWarps; ++t) add_part(all, s.sums[t][tid], 1.f);
  store_head(P, join.y, h, 32 * c0 + tid, all, l, m);
}

// A unit's join is that of the query that starts in it and ends in a later one,
// from the query's parts in the units' order.  The weights are e^(m_s - m) with m
// the largest.  As many blocks as the SMs hold go through the joins, a team of a
// block a head at a time; where there are so few joins (one long request: 74 parts
// a head) that the blocks suffice for a head or half a head each, a block takes one
// with all its warps.  Values are requested before the maximum is known.  What
// bounds it: the parts, read once, and below that the barriers and dependent loads
// of one item, 3 us (of 74 parts: by teams 7).
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) paged_join_kernel(const PagedAttnParams P) {
  __shared__ JoinShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the first kernel may still run
  const int2 mine = tid < P.units ? P.joins[tid] : make_int2(-1, -1);
  const uint32_t those = __ballot_sync(0xffffffffu, mine.x >= 0);
  if (lane == 0) s.counts[warp] = __popc(those);
  __syncthreads();
  int n = 0, at = __popc(those & ((1u << lane) - 1u));
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    if (k < warp) at += s.counts[k];
    n += s.counts[k];
  }
  if (mine.x >= 0) s.list[at] = make_int4(tid, mine.x, mine.y, 0);
  __syncthreads();
  const int items = n * P.H, blocks = static_cast<int>(gridDim.x);
  if (items <= blocks) {
    const bool halves = 2 * items <= blocks;
    const int item = halves ? blockIdx.x >> 1 : blockIdx.x;
    if (item >= items) return;
    const int v = item / P.H, h = item - v * P.H;
    if (halves) {
      join_wide<2>(P, s, s.list[v], h, 2 * (blockIdx.x & 1));
    } else {
      join_wide<4>(P, s, s.list[v], h, 0);
    }
    return;
  }
  const int team = tid / kTeam, col = tid % kTeam;
  for (int item = blockIdx.x * kTeams + team; item < items; item += blocks * kTeams) {
    const int v = item / P.H, h = item - v * P.H;
    const int4 join = s.list[v];
    const int unit = join.x, parts = join.z - unit + 1;
    float4 x[kBatch];
    float2 ml[kBatch];
    auto request = [&](int k0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t p = part_at(P, unit, h, min(k0 + k, parts - 1));
        x[k] = *(reinterpret_cast<const float4 *>(P.part_o + p * kPagedDv) + col);
        ml[k] = P.part_ml[p];
      }
    };
    request(0);
    float m = -__builtin_huge_valf();
    for (int k0 = 0; k0 < parts; k0 += 32)
      m = fmaxf(m, warp_max(k0 + lane < parts ? P.part_ml[part_at(P, unit, h, k0 + lane)].x : -__builtin_huge_valf()));
    const float base = m == -__builtin_huge_valf() ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int k0 = 0; k0 < parts; k0 += kBatch) {
      if (k0) request(k0);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + k < parts && ml[k].y != 0.f) {
          const float w = ex2(ml[k].x - base);
          l += w * ml[k].y;
          add_part(acc, x[k], w);
        }
      }
    }
    store_head(P, join.y, h, col, acc, l, m);
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
