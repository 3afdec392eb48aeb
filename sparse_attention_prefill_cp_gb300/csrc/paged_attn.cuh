// What the kernels of the attention over the paged latent cache share.
#pragma once

#include "attn_common.cuh"

namespace dsa {

constexpr int kPagedD = 576, kPagedDv = 512;
constexpr int kPagedMaxHeads = 128;
constexpr int kPagedRows = 128;  // KV rows per block

struct PagedAttnParams {
  const int32_t *table;    // [batch][max_pages]
  const int32_t *lens;     // [n] positions a query sees (negative: no query)
  const int32_t *blocks;   // [n][nsel] page ordinals, distinct, in any order, or nullptr: all pages
  const int32_t *req;      // [n] row of the table, or nullptr: row i
  const float *sink;       // [H] or nullptr
  __nv_bfloat16 *out;      // [n][H][Dv]
  float *part_o;           // [2 * units][H][Dv]
  float2 *part_ml;         // [2 * units][H]: (m, l), m in log2 units
  int2 *joins;             // [units]: the query that starts in a unit and ends in a later one, and that unit (or -1)
  float scale_log2;        // softmax_scale * log2(e)
  int32_t n, batch, max_pages, nsel, num_pages, page_shift;
  int32_t H, groups, units;  // groups of heads; a unit is a share of the call's blocks
  int *err;
};

// Pages that a query of `len` >= 0 positions sees.
__host__ __device__ __forceinline__ int paged_pages(int len, int max_pages, int shift) {
  const int64_t pages = (static_cast<int64_t>(len) + (1 << shift) - 1) >> shift;
  return static_cast<int>(pages < max_pages ? pages : max_pages);
}

// Whether a query goes through its list of pages, every entry of it; one that
// sees fewer pages than the list has entries goes through its pages instead and
// takes those that the list names, so that nothing depends on where in the list
// the pages that it sees stand.
__host__ __device__ __forceinline__ bool paged_listed(int pages, int nsel) { return nsel > 0 && nsel <= pages; }

// Blocks of 128 rows of a query that sees `len` positions: at least one (its
// rows may all be masked), none where there is no query.
__host__ __device__ __forceinline__ int paged_blocks(int len, int nsel, int max_pages, int shift) {
  if (len < 0) return 0;
  int used = paged_pages(len, max_pages, shift);
  if (paged_listed(used, nsel)) used = nsel;
  const int per = kPagedRows >> shift;
  return used > 0 ? (used + per - 1) / per : 1;
}

// Launch of the kernel that joins the parts of queries that lie in more than one unit.
dsa_status launch_paged_join(const PagedAttnParams &P, cudaStream_t stream);

}  // namespace dsa
