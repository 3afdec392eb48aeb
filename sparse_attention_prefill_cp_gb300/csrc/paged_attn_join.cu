// Attention over the paged cache: the join of the parts of queries whose blocks
// lie in more than one unit.
#include "internal.h"
#include "paged_attn.cuh"

namespace dsa {
namespace {

constexpr int kTeam = kPagedDv / 4;     // threads on a head's values, four columns each
constexpr int kTeams = 4;               // of a block
constexpr int kBatch = 4;               // parts whose loads are in flight together
constexpr int kMaxUnits = kTeam * kTeams;

// A unit's join is that of the query that starts in it and ends in a later one,
// from the query's parts in the units' order.  Part 2u + 1 is of the query that
// starts in unit u, part 2u of the one that goes on there.  The weights are
// e^(m_s - m) with m the largest.  A block has four teams: a head each of one
// unit; but where there are so few joins (one long request: 74 parts a head) that
// the blocks suffice for a head each, a block takes one head, its teams every
// fourth part, and their sums are added in the teams' order.  The values of the
// first parts are requested before the maximum is known.  (A block of one team per
// unit and head: 12 us for 75 joins of 128 heads, 19 for one of 74 parts.)
__global__ void __launch_bounds__(kTeam * kTeams, 3) paged_join_kernel(const PagedAttnParams P) {
  __shared__ int32_t units[kMaxUnits];
  __shared__ int32_t counts[kMaxUnits / 32];
  __shared__ float4 sums[kTeams][kTeam];
  __shared__ float lsum[kTeams];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col = tid % kTeam, team = tid / kTeam;
  const int heads4 = (P.H + kTeams - 1) / kTeams;
  int unit = static_cast<int>(blockIdx.x) / heads4, h = (static_cast<int>(blockIdx.x) - unit * heads4) * kTeams + team;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the first kernel may still run
  const bool has = tid < P.units && P.joins[tid].x >= 0;
  int2 join = P.joins[unit];
  const uint32_t those = __ballot_sync(0xffffffffu, has);
  if (lane == 0) counts[warp] = __popc(those);
  __syncthreads();
  int n = 0, at = __popc(those & ((1u << lane) - 1u));
#pragma unroll
  for (int k = 0; k < kMaxUnits / 32; ++k) {
    if (k < warp) at += counts[k];
    n += counts[k];
  }
  const bool wide = static_cast<int64_t>(n) * P.H <= gridDim.x;
  if (wide) {  // the units with a join, in order
    if (has) units[at] = tid;
    __syncthreads();
    const int v = static_cast<int>(blockIdx.x) / P.H;
    if (v >= n) return;
    unit = units[v];
    h = static_cast<int>(blockIdx.x) - v * P.H;
    join = P.joins[unit];
  } else if (join.x < 0 || h >= P.H) {
    return;
  }
  const int parts = join.y - unit + 1;
  auto part = [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * unit + 1 : 2 * (unit + k)) * P.H + h; };
  const int step = wide ? kTeams : 1, first = wide ? team : 0;
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
  if (wide) {
    sums[team][col] = acc;
    if (col == 0) lsum[team] = l;
    __syncthreads();
    if (team > 0) return;
    for (int t = 1; t < kTeams; ++t) {
      const float4 y = sums[t][col];
      acc.x += y.x;
      acc.y += y.y;
      acc.z += y.z;
      acc.w += y.w;
      l += lsum[t];
    }
  }
  const bool empty = l == 0.f;
  if (P.sink && !empty) l += ex2(P.sink[h] * 1.4426950408889634f - m);
  const float inv = empty ? 0.f : 1.f / l;
  const uint2 r = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2 *>(P.out + (static_cast<int64_t>(join.x) * P.H + h) * kPagedDv + 4 * col) = r;
}

}  // namespace

dsa_status launch_paged_join(const PagedAttnParams &P, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(P.units) * static_cast<unsigned>((P.H + kTeams - 1) / kTeams);
  const cudaError_t e = launch_overlapped(paged_join_kernel, dim3(blocks), kTeam * kTeams, 0, stream, P);
  return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

}  // namespace dsa
