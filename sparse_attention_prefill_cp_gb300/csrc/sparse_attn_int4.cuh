// What the two kernels of the attention over the 4-bit cache share: the call's
// parameters, the resolution of index entries, and single-use loads.
#pragma once

#include "attn_common.cuh"
#include "int4_common.cuh"

namespace dsa {

constexpr int kInt4D = 576, kInt4Dv = 512;
constexpr int kInt4MaxHeads = 128;
constexpr int kInt4MaxSplits = 32;
constexpr int kInt4MaxOrdered = 1024;  // queries that are started in order of their lists' lengths

struct AttnInt4Params {
  const uint8_t *cache;    // [cache_rows][row_bytes]
  const int32_t *slots;    // [num_kv_rows] KV row -> cache row (negative: no row), or nullptr: entries are cache rows
  const int32_t *idx;      // [n][topk]
  const int32_t *q_rows;   // [n] row of q and out (negative: none), or nullptr: row i
  const float *sink;       // [H] or nullptr
  const int32_t *order;    // [n] the query that a pair takes as its i-th, or nullptr: i (splits == 1)
  __nv_bfloat16 *out;      // [num_q_rows][H][Dv]
  float *part_o;           // [n * splits][H][Dv] (splits > 1)
  float2 *part_ml;         // [n * splits][H][2]: (m, l) of each half of the value columns (splits > 1)
  float scale_log2;        // softmax_scale * log2(e)
  int32_t H, topk, splits, split_len;  // split_len: entries per split, a multiple of the kernel's block
  int32_t groups, group_heads;         // of sparse_attn_int4_few.cu: groups of 16 or 32 heads
  int32_t num_kv_rows, cache_rows, num_q_rows;
  Int4Geom g;
  int *err;
};

// Launch of the kernel for groups of few heads (n * splits * groups CTAs).
dsa_status launch_attn_int4_few(const void *q, int32_t n, const AttnInt4Params &P, cudaStream_t stream);
constexpr int kInt4FewRows = 128;   // its entries per block

// Launch of the kernel that fills P.order; what is launched next may start
// while it runs.
dsa_status launch_attn_int4_order(int32_t n, const AttnInt4Params &P, int32_t *order, cudaStream_t stream);

// Launch of the kernel that joins the parts of P.splits > 1 splits.
dsa_status launch_attn_int4_join(int32_t n, const AttnInt4Params &P, cudaStream_t stream);

// The cache row that an index entry names (negative: none), unchecked: the
// value of the slot load is not looked at before checked_row.
__device__ __forceinline__ int slot_of(const AttnInt4Params &P, int32_t *bad, int entry, int k) {
  if (!P.slots || entry < 0) return entry;
  if (entry >= P.num_kv_rows) {
    bad[0] = 49;
    bad[1] = k;
    return -1;
  }
  return __ldg(P.slots + entry);
}
__device__ __forceinline__ int checked_row(const AttnInt4Params &P, int32_t *bad, int row, int k) {
  if (row >= P.cache_rows) {
    bad[0] = 50;
    bad[1] = k;
    return -1;
  }
  return row;
}

// Loads of cache bytes, each used once on this SM; volatile, to be issued where
// they stand.  Without `go` nothing is read and r stays: rows that do not
// exist must not all read one address (152 SMs on one row's sectors wait for
// each other: 55 K cycles in the last block of a call).
__device__ __forceinline__ void ld_once(uint4 &r, const void *p, bool go) {
  asm volatile(
      "{\n\t.reg .pred g;\n\tsetp.ne.b32 g, %5, 0;\n\t"
      "@g ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
      : "l"(p), "r"(static_cast<uint32_t>(go)));
}
__device__ __forceinline__ void ld_once_u16(uint32_t &r, const void *p, bool go) {
  asm volatile(
      "{\n\t.reg .pred g;\n\t.reg .u16 t;\n\tsetp.ne.b32 g, %2, 0;\n\tcvt.u16.u32 t, %0;\n\t"
      "@g ld.global.nc.L1::no_allocate.u16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}"
      : "+r"(r)
      : "l"(p), "r"(static_cast<uint32_t>(go)));
}
__device__ __forceinline__ void ld_once_u8(uint32_t &r, const void *p, bool go) {
  asm volatile(
      "{\n\t.reg .pred g;\n\tsetp.ne.b32 g, %2, 0;\n\t"
      "@g ld.global.nc.L1::no_allocate.u8 %0, [%1];\n\t}"
      : "+r"(r)
      : "l"(p), "r"(static_cast<uint32_t>(go)));
}

}  // namespace dsa
