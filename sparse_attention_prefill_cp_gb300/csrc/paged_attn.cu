// MLA attention over the paged latent cache, for any number of queries down to
// one token of one request:
//   l_p = softmax_scale * q[i, h, :] . k_p
//   out[i, h, :] = sum_p e^(l_p - m) k_p[:Dv] / (sum_p e^(l_p - m) + e^(sink_h - m))
// over the positions p < lens[i] of the query's request, or those of them that
// lie in the pages blocks[i] names.  D = 576, Dv = 512, up to 128 heads.
//
// Rows are the M = 128 side of both products, heads the N side:
//   S^T [128 rows x heads]    = K [rows x 576] (K-major A) * Q^T
//   O^T [128 values x heads] += V^T (the same tiles, MN-major A) * P^T,  four times
// so a page's rows go from memory to shared memory once, by TMA, as they lie,
// and the softmax of a head is a sum over TMEM lanes that no other CTA has part
// of.  A CTA takes a group of up to 64 heads: more (128 x 512 fp32) would fill
// an SM's tensor memory with O alone, and fewer would read the rows again.
//
// Work: the call's blocks of 128 rows, of all queries in order, are cut into
// equal shares, a unit each (a CTA per group of heads); a unit goes through its
// share query by query.  A query that lies in one unit is finished there; the
// parts of the others (unnormalised O and (m, l) per head) are joined by a
// second kernel in the order of the units, without atomics.  So ragged lengths
// keep all SMs busy to the end, whatever the lengths are, and the host need not
// know them.
//
// Shared memory: a ring of tiles of 128 value columns (32 KB, what one step of
// O^T needs, handed back as soon as that step is done), one or two tiles of rope
// columns, over which P is written once QK is done, and Q.
//
// Warps: softmax (a warpgroup for every 16 heads, thread = row of the block = TMEM
// lane), MMA issue, TMA.
//
// Softmax: a head's reference m lies within 2^8 of its running maximum; only
// where a logit is above it (and in a query's first block) are the block's
// maxima reduced and O^T and the sums rescaled.  P is rounded to bf16 for the
// MMA (each weight within 2^-8 of itself); logits, sums and O are fp32.  Rows
// behind a query's last position hold anything, NaN included: they are zeroed in
// shared memory, since 0 * NaN would reach O.
//
// What bounds it: with up to 32 heads HBM (64 requests of 8,192 rows, 16 heads: 106
// us with the join, 5.7 TB/s; 64 heads 119 us).  With 128 heads shared memory: a
// block of 64 heads moves 578 KB (operands of QK and PV 415, TMA 147, P 16), 4,520
// cycles, and takes 5,850, since Q and one block fill the 227 KB and nothing of the
// next lands while the softmax runs: 64 requests of 8,192 rows 189 us, 2,048 queries
// of 2,048 rows 1,390 us, 840 TFLOP/s.
#include "internal.h"
#include "paged_attn.cuh"

namespace dsa {
namespace {

constexpr int kD = kPagedD, kDv = kPagedDv, kRows = kPagedRows;
constexpr int kChunkBytes = kRows * 128;     // 64 columns of a block (128B swizzle)
constexpr int kTileBytes = 2 * kChunkBytes;  // 128 value columns
constexpr int kTiles = kDv / 128;            // per block
constexpr int kQChunks = kD / 64;

template <int HP_, int NT_, int NR_>
struct PagedCfg {
  static constexpr int HP = HP_;         // heads (the missing ones are zero rows of Q)
  static constexpr int NT = NT_;         // value tiles
  static constexpr int NR = NR_;         // rope tiles
  static constexpr int HW = 16;          // heads of a softmax warpgroup
  static constexpr int WG = HP / HW;
  static constexpr int kMmaWarp = 4 * WG, kLoadWarp = kMmaWarp + 1;
  static constexpr int kWarps = kLoadWarp + 1, kThreads = 32 * kWarps;
  static constexpr int kSCol = kTiles * HP;  // TMEM: O^T, then two S buffers
  static constexpr int kTmemCols = kSCol + 2 * HP <= 128 ? 128 : kSCol + 2 * HP <= 256 ? 256 : 512;
  static constexpr int kOffTiles = 0;
  static constexpr int kOffRope = NT * kTileBytes;  // and P: [row][64 heads] bf16, HP of them used
  static constexpr int kOffQ = kOffRope + NR * kChunkBytes;
  static constexpr int kOffStat = kOffQ + kQChunks * HP * 128;
  // floats, per warpgroup: -m per warp and head, its rescaling factor, the warps' maxima or sums
  static constexpr int kStatNm = 0, kStatAlpha = 4 * HW, kStatRed = 8 * HW, kStatWg = 12 * HW;
  static constexpr int kOffBar = kOffStat + WG * kStatWg * 4;
  static constexpr int kNumBars = 2 + 2 * NT + 2 * NR + 2 + 2 + 1 + 1;
  static constexpr int kOffMisc = kOffBar + (kNumBars + 1) / 2 * 16;
  // [0] tmem, [1] failed wait, [2..3] bad index, [4] first query, [5] where in it, [8..8+2*kWarps) scan
  static constexpr int kSmemBytes = kOffMisc + (8 + 2 * kWarps) * 4 + 1024;
  static constexpr uint32_t kIdescQK = idesc_bf16(kRows, HP, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16(128, HP, true, true);
  static_assert(kSCol + 2 * HP <= kTmemCols, "TMEM budget");
  static_assert(kOffQ % 1024 == 0 && (HP * 128) % 1024 == 0, "swizzle atoms");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};
using Cfg16 = PagedCfg<16, 5, 2>;
using Cfg32 = PagedCfg<32, 5, 1>;
using Cfg64 = PagedCfg<64, 4, 1>;

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

// OR of a predicate over the four warps of a warpgroup, and a barrier among them.
__device__ __forceinline__ bool wg_or(int wg, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.cta.red.or.pred b, %2, 128, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(1 + wg)
      : "memory");
  return r != 0;
}

// A plain load that stays where it stands: what the compiler makes of a[i] here it
// may also move or repeat, and the kernel of 64 heads then spills 12 bytes (chunk of
// 2,048 queries: 1,394 against 1,385 us).
__device__ __forceinline__ int load_plain(const int32_t *p) {
  int x;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

// A unit's walk through its share: segments of consecutive blocks of one query.
// A query counts a block more than it has, its first: what a segment costs beside
// its blocks (Q, the first block's maxima, the result) is about a block's time, so
// units of many short queries get fewer blocks (64 queries of 1 to 16 blocks and
// 128 heads: 49 -> 41 us).
struct Walk {
  int q, j0, j1, nb, len, row;  // query, blocks [j0, j1) of its nb, positions it sees, its row of the table
  int take;                     // what the segment counts
  int64_t left;                 // of the share from here on
  // the segment at count `o` of query `query`; false: the share is done
  __device__ __forceinline__ bool start(const PagedAttnParams &P, int query, int o) {
    for (q = query; q < P.n && left > 0; ++q, o = 0) {
      len = load_plain(P.lens + q);
      nb = paged_blocks(len, P.nsel, P.max_pages, P.page_shift);
      if (nb == 0) continue;
      take = static_cast<int>(min(static_cast<int64_t>(nb + 1 - o), left));
      j0 = max(o - 1, 0);
      j1 = o + take - 1;
      if (j1 > j0) {
        row = P.req ? load_plain(P.req + q) : q;
        if (row < 0 || row >= P.batch) len = 0;  // reported by the loading warp
        return true;
      }
      left -= take;  // the share ends with the query's extra count
    }
    return false;
  }
  __device__ __forceinline__ bool next(const PagedAttnParams &P) {
    left -= take;
    return start(P, q + 1, 0);
  }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == nb; }
};

// The page of entry e of what a query goes through, its list or its pages, and the
// entry's first position: the page number unchecked, -1 (and no position) where the
// entry names none.  Called by whole warps whose lanes' entries are of one block.
__device__ __forceinline__ int page_of(const PagedAttnParams &P, const Walk &w, int e, int &pos) {
  int at = e;
  pos = INT32_MAX;
  if (P.blocks) {
    const int32_t *list = P.blocks + static_cast<int64_t>(w.q) * P.nsel;
    if (paged_listed(paged_pages(w.len, P.max_pages, P.page_shift), P.nsel)) {
      if (e >= P.nsel) return -1;
      at = load_plain(list + e);
    } else {
      // which of the block's up to eight pages the list names: a bit each
      const uint32_t E = kRows >> P.page_shift, first = e & ~(E - 1);
      uint32_t named = 0;
      for (int k = threadIdx.x & 31; k < P.nsel; k += 32) {
        const uint32_t d = static_cast<uint32_t>(load_plain(list + k)) - first;
        if (d < E) named |= 1u << d;
      }
      if (!(__reduce_or_sync(0xffffffffu, named) >> (e - first) & 1u)) return -1;
    }
  }
  if (at < 0 || at >= P.max_pages || static_cast<int64_t>(at) << P.page_shift >= w.len) return -1;
  pos = at << P.page_shift;
  return load_plain(P.table + static_cast<int64_t>(w.row) * P.max_pages + at);
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                      const PagedAttnParams P) {
  constexpr int HP = C::HP, HW = C::HW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
  uint64_t *q_full = bars;                 // a query's Q landed (TMA)
  uint64_t *q_free = bars + 1;             // its last QK done (MMA commit)
  uint64_t *t_full = bars + 2;             // [NT] a tile's rows landed (TMA)
  uint64_t *t_free = t_full + C::NT;       // [NT] PV is done with it (MMA commit)
  uint64_t *r_full = t_free + C::NT;       // [NR] a block's rope columns landed (TMA)
  uint64_t *pv_done = r_full + C::NR;      // [NR] PV of a block done, its P (the rope tile) free (MMA commit)
  uint64_t *s_full = pv_done + C::NR;      // [2] QK done (MMA commit)
  uint64_t *s_free = s_full + 2;           // [2] S read out of TMEM (softmax warps)
  uint64_t *p_full = s_free + 2;           // P written (softmax warps)
  uint64_t *o_free = p_full + 1;           // a query's O read out of TMEM (softmax warps)
  int32_t *misc = reinterpret_cast<int32_t *>(smem + C::kOffMisc);
  int32_t *failed = misc + 1, *bad = misc + 2;
  uint64_t *scan = reinterpret_cast<uint64_t *>(misc + 8);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = static_cast<int>(blockIdx.x) / P.groups;
  const int h0 = (static_cast<int>(blockIdx.x) - unit * P.groups) * HP;
  const int heads = min(HP, P.H - h0);

  if (tid == 0) {
    misc[1] = misc[2] = misc[3] = 0;
    misc[4] = P.n;
    misc[5] = 0;
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    for (int s = 0; s < C::NT; ++s) {
      mbar_init(&t_full[s], 1);
      mbar_init(&t_free[s], 1);
    }
    for (int s = 0; s < C::NR; ++s) {
      mbar_init(&r_full[s], 1);
      mbar_init(&pv_done[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 4 * C::WG);
    }
    mbar_init(p_full, 4 * C::WG);
    mbar_init(o_free, 4 * C::WG);
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(reinterpret_cast<uint32_t *>(&misc[0]), C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == C::kLoadWarp && lane == 0) {
    tma_prefetch_desc(&q_map);
    tma_prefetch_desc(&kv_map);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the kernel before may still run
  // Where the share starts: the threads sum what consecutive queries count, and
  // the one that holds the share's first count finds its query.
  const int per = (P.n + C::kThreads - 1) / C::kThreads;
  const int i0 = min(tid * per, P.n), i1 = min(i0 + per, P.n);
  int64_t mine = 0;
  auto counts = [&](int i) {
    const int nb = paged_blocks(P.lens[i], P.nsel, P.max_pages, P.page_shift);
    return nb ? nb + 1 : 0;
  };
  for (int i = i0; i < i1; ++i) mine += counts(i);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += a;
  }
  if (lane == 31) scan[warp] = upto;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t total = 0, before = upto - mine;
#pragma unroll
  for (int w = 0; w < C::kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int64_t share = (total + P.units - 1) / P.units;
  const int64_t g0 = min(unit * share, total), g1 = min(g0 + share, total);
  if (g0 < g1 && g0 >= before && g0 < before + mine) {
    int64_t at = before;
    for (int i = i0; i < i1; ++i) {
      const int c = counts(i);
      if (g0 < at + c) {
        misc[4] = i;
        misc[5] = static_cast<int>(g0 - at);
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  Walk walk;
  walk.left = g1 - g0;
  bool more = walk.start(P, misc[4], misc[5]);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join, which waits for this kernel's end
  if (warp == C::kLoadWarp) {
    // ---------------- TMA: lane l of a tile's boxes (chunk of 64 columns, page);
    // the pages of a block are looked up one block ahead.
    const int E = kRows >> P.page_shift;           // pages of a block
    const int e_lane = lane & (E - 1), c_lane = lane / E;
    const uint32_t page_bytes = 128u << P.page_shift;  // of a chunk
    bool ok = true;
    int tile = 0, blk = 0, seg = 0, pos = INT32_MAX;
    int2 join = make_int2(-1, -1);
    auto lookup = [&](int j) { return page_of(P, walk, j * E + e_lane, pos); };
    int page_next = more ? lookup(walk.j0) : -1;
    while (ok && more) {
      if (walk.j0 == 0) {
        const int len = P.lens[walk.q], row = P.req ? P.req[walk.q] : walk.q;
        if (row < 0 || row >= P.batch || len > static_cast<int64_t>(P.max_pages) << P.page_shift) {
          bad[0] = 58;
          bad[1] = walk.q;
        }
        // it ends in a later unit: the share's last segment
        if (walk.j1 < walk.nb) join = make_int2(walk.q, static_cast<int>((g1 - walk.left + walk.take + walk.nb - 1 - walk.j1) / share));
      }
      if (seg > 0) ok = __all_sync(0xffffffffu, wait_for(q_free, (seg - 1) & 1, failed, 80, walk.q));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, kQChunks * HP * 128);
        for (int c = 0; c < kQChunks; ++c) tma_load_3d(smem + C::kOffQ + c * HP * 128, &q_map, 64 * c, h0, walk.q, q_full);
      }
      ++seg;
      const int j1 = walk.j1;
      bool again = false;
      for (int j = walk.j0; j < j1; ++j) {
        // a page number that the table does not have for rows that exist: reported; the softmax masks its rows
        const bool there = page_next >= 0 && page_next < P.num_pages;
        if (!there && pos != INT32_MAX) {
          bad[0] = 57;
          bad[1] = walk.q;
        }
        const int page = there ? page_next : -1;
        const uint32_t here = __ballot_sync(0xffffffffu, there) & ((1u << E) - 1u);
        const uint32_t bytes = static_cast<uint32_t>(__popc(here)) * page_bytes;
        if (j + 1 < j1) {
          page_next = lookup(j + 1);
        } else {
          again = walk.next(P);
          if (again) page_next = lookup(walk.j0);
        }
#pragma unroll 1
        for (int t = 0; t < kTiles; ++t) {
          const int s = tile % C::NT;
          ok = __all_sync(0xffffffffu, wait_for(&t_free[s], ((tile / C::NT) & 1) ^ 1, failed, 81, blk));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&t_full[s], 2 * bytes);
          __syncwarp();
          if (c_lane < 2 && there)
            tma_load_3d(smem + C::kOffTiles + s * kTileBytes + c_lane * kChunkBytes + e_lane * page_bytes, &kv_map,
                        128 * t + 64 * c_lane, 0, page, &t_full[s]);
          ++tile;
        }
        if (!ok) break;
        const int r = blk % C::NR;
        ok = __all_sync(0xffffffffu, wait_for(&pv_done[r], ((blk / C::NR) & 1) ^ 1, failed, 82, blk));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&r_full[r], bytes);
        __syncwarp();
        if (c_lane == 0 && there)
          tma_load_3d(smem + C::kOffRope + r * kChunkBytes + e_lane * page_bytes, &kv_map, kDv, 0, page, &r_full[r]);
        ++blk;
        // the next block on its way to the L2 while this one is worked on
        if ((j + 1 < j1 || again) && page_next >= 0 && page_next < P.num_pages)
          for (int c = c_lane; c < kQChunks; c += 32 / E) tma_prefetch_3d(&kv_map, 64 * c, 0, page_next);
      }
      more = again;
    }
    if (h0 == 0 && lane == 0) P.joins[unit] = join;
    if (!ok && lane == 0) {
      // loads under way land before this CTA's memory goes
      if (seg > 0) wait_for(q_full, (seg - 1) & 1, failed, 83);
      for (int s = 0; s < C::NT; ++s) {
        const int n = (tile - s + C::NT - 1) / C::NT;  // loads into slot s
        if (n > 0) wait_for(&t_full[s], (n - 1) & 1, failed, 83);
      }
      for (int s = 0; s < C::NR; ++s) {
        const int n = (blk - s + C::NR - 1) / C::NR;
        if (n > 0) wait_for(&r_full[s], (n - 1) & 1, failed, 83);
      }
    }
  } else if (warp == C::kMmaWarp) {
    // ---------------- MMA issuer: QK of a block tile by tile as they land, then,
    // when its P is there, PV, which hands the tiles back one by one.  Where a
    // fifth tile has landed its part of the next QK goes before PV.  The whole
    // warp runs the loop and one elected lane issues.
    const bool issuer = elect_one();
    const uint32_t tile_addr = smem_u32(smem + C::kOffTiles);
    const uint64_t k_a = smem_desc(tile_addr, 16, 1024, kLayoutSW128);
    const uint64_t v_a = smem_desc(tile_addr, kChunkBytes, 1024, kLayoutSW128);
    const uint64_t rope_a = smem_desc(smem_u32(smem + C::kOffRope), 16, 1024, kLayoutSW128);
    const uint64_t p_b = smem_desc(smem_u32(smem + C::kOffRope), kChunkBytes, 1024, kLayoutSW128);
    const uint64_t q_b = smem_desc(smem_u32(smem + C::kOffQ), 16, 1024, kLayoutSW128);
    auto all_wait = [&](uint64_t *bar, uint32_t parity, int site, int detail) {
      return __all_sync(0xffffffffu, wait_for(bar, parity, failed, site, detail));
    };
    bool ok = true;
    // QK of block b over tile t
    auto qk_tile = [&](int b, int t) {
      const int g = kTiles * b + t, s = g % C::NT;
      ok = ok && all_wait(&t_full[s], (g / C::NT) & 1, 84, b);
      if (!ok) return;
      tc_fence_after();
      const uint32_t s_tm = tmem + C::kSCol + (b & 1) * HP;
      const uint64_t a = desc_add(k_a, static_cast<uint32_t>(s * kTileBytes) >> 4);
      const uint64_t q = desc_add(q_b, static_cast<uint32_t>(2 * t * HP * 128) >> 4);
      if (issuer) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ss(s_tm, desc_add(a, (k >> 2) * (kChunkBytes >> 4) + (k & 3) * 2),
                 desc_add(q, (k >> 2) * (HP * 128 >> 4) + (k & 3) * 2), C::kIdescQK, t > 0 || k > 0 ? 1u : 0u);
      }
      __syncwarp();
    };
    // the rest of QK of block b from tile t0 on
    auto qk_rest = [&](int b, int t0) {
#pragma unroll 1
      for (int t = t0; ok && t < kTiles; ++t) qk_tile(b, t);
      const int r = b % C::NR;
      ok = ok && all_wait(&r_full[r], (b / C::NR) & 1, 85, b);
      if (!ok) return;
      tc_fence_after();
      const uint32_t s_tm = tmem + C::kSCol + (b & 1) * HP;
      const uint64_t a = desc_add(rope_a, static_cast<uint32_t>(r * kChunkBytes) >> 4);
      if (issuer) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(s_tm, desc_add(a, k * 2), desc_add(q_b, 8 * (HP * 128 >> 4) + k * 2), C::kIdescQK, 1u);
        mma_commit(&s_full[b & 1]);
      }
      __syncwarp();
    };
    int blk = 0, seg = 0;
    for (; ok && more; more = walk.next(P), ++seg) {
      ok = all_wait(q_full, seg & 1, 86, seg);
      if (ok && blk >= 2) ok = all_wait(&s_free[blk & 1], ((blk - 2) >> 1) & 1, 87, blk);
      qk_rest(blk, 0);
      if (!ok) break;
      if (walk.j1 - walk.j0 == 1 && issuer) mma_commit(q_free);
      __syncwarp();
      for (int j = walk.j0; ok && j < walk.j1; ++j, ++blk) {
        int early = 0;
        const bool again = j + 1 < walk.j1;
        if (again) {
          if (blk >= 1) ok = all_wait(&s_free[(blk + 1) & 1], ((blk - 1) >> 1) & 1, 87, blk);
          if (C::NT > kTiles && ok) {
            const int g = kTiles * (blk + 1), s = g % C::NT;
            if (__all_sync(0xffffffffu, mbar_test(&t_full[s], (g / C::NT) & 1))) {
              qk_tile(blk + 1, 0);
              early = 1;
            }
          }
        }
        if (j == walk.j0 && seg > 0) ok = ok && all_wait(o_free, (seg - 1) & 1, 88, blk);
        ok = ok && all_wait(p_full, blk & 1, 89, blk);
        if (!ok) break;
        tc_fence_after();
        const int r = blk % C::NR;
        const uint64_t p = desc_add(p_b, static_cast<uint32_t>(r * kChunkBytes) >> 4);
#pragma unroll 1
        for (int t = 0; t < kTiles; ++t) {
          const int s = (kTiles * blk + t) % C::NT;
          const uint64_t a = desc_add(v_a, static_cast<uint32_t>(s * kTileBytes) >> 4);
          if (issuer) {
#pragma unroll
            for (int k = 0; k < kRows / 16; ++k)
              mma_ss(tmem + t * HP, desc_add(a, k * 128), desc_add(p, k * 128), C::kIdescPV,
                     j > walk.j0 || k > 0 ? 1u : 0u);
            mma_commit(&t_free[s]);
          }
          __syncwarp();
        }
        if (issuer) mma_commit(&pv_done[r]);
        __syncwarp();
        if (again) {
          qk_rest(blk + 1, early);
          if (ok && j + 2 == walk.j1 && issuer) mma_commit(q_free);
          __syncwarp();
        }
      }
    }
  } else {
    // ---------------- softmax: thread = row of the block = TMEM lane; warpgroup
    // wg has heads [wg * HW, (wg + 1) * HW) of the group.  Every decision that
    // guards a tcgen05.ld/st (.sync.aligned) is warp-uniform, and every one that
    // guards a barrier of the four warps is the same in all.
    const int wg = warp >> 2, w = warp & 3, r = tid & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(w * 32) << 16) + wg * HW;
    float *stat = reinterpret_cast<float *>(smem + C::kOffStat) + wg * C::kStatWg;
    float *nm = stat + C::kStatNm + w * HW;        // -m of every head (0 while m is -inf), this warp's copy
    float *alpha = stat + C::kStatAlpha + w * HW;
    float *red = stat + C::kStatRed;               // [4 warps][HW]
    const uint64_t sc2 = f2_pack(P.scale_log2, P.scale_log2);
    const int E_shift = 7 - P.page_shift, e_row = r >> P.page_shift, in_page = r & ((1 << P.page_shift) - 1);
    int page_next = -1;
    bool fits_next = false;
    auto lookup = [&](int j) {  // of row r of block j
      int pos;
      page_next = page_of(P, walk, (j << E_shift) + e_row, pos);
      fits_next = pos != INT32_MAX && pos + in_page < walk.len;
    };
    if (more) lookup(walk.j0);
    bool ok = true;
    int blk = 0;
    while (more && ok) {
      const int j0 = walk.j0, j1 = walk.j1, query = walk.q;
      const bool whole = walk.whole();
      float m = -__builtin_huge_valf(), l[HW];  // m: of head `lane`, the same in all four warps
      bool none = true;                         // some head still has m = -inf
#pragma unroll
      for (int k = 0; k < HW; ++k) l[k] = 0.f;
#pragma unroll 1
      for (int j = j0; j < j1; ++j, ++blk) {
        const bool used = fits_next && page_next >= 0 && page_next < P.num_pages;
        if (j + 1 < j1) {
          lookup(j + 1);
        } else {
          more = walk.next(P);
          if (more) lookup(walk.j0);
        }
        const int rope = blk % C::NR;
        uint8_t *prow = smem + C::kOffRope + rope * kChunkBytes + r * 128;
        ok = __all_sync(0xffffffffu, ok && wait_for(&s_full[blk & 1], (blk >> 1) & 1, failed, 90, blk));
        tc_fence_after();
        // logits against the reference, in log2 units; S stays in TMEM until the block is done, to be read again
        // where the reference has to move
        float t[HW], top = -__builtin_huge_valf();
        auto load_s = [&]() {
          uint32_t x[HW];
          tmem_ld(lane_base + C::kSCol + (blk & 1) * HP, x);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < HW; ++k) t[k] = used ? __uint_as_float(x[k]) : -__builtin_huge_valf();
        };
        auto against = [&]() {
#pragma unroll
          for (int k = 0; k < HW; k += 4) {
            const float4 n4 = *reinterpret_cast<const float4 *>(nm + k);
            f2_unpack(f2_fma(f2_pack(t[k], t[k + 1]), sc2, f2_pack(n4.x, n4.y)), t[k], t[k + 1]);
            f2_unpack(f2_fma(f2_pack(t[k + 2], t[k + 3]), sc2, f2_pack(n4.z, n4.w)), t[k + 2], t[k + 3]);
          }
        };
        load_s();
        if (!none) {
          against();
#pragma unroll
          for (int k = 0; k < HW; k += 2) top = fmax3(top, t[k], t[k + 1]);
        }
        if (wg_or(wg, none || top > 8.f || !ok)) {
          ok = !wg_or(wg, !ok);
          if (!ok) break;
          // the block's maxima: of the warp's rows by head, then of the warps
          float mine_max = -__builtin_huge_valf();
          if (!none) load_s();
#pragma unroll
          for (int k = 0; k < HW; ++k) {
            const float mx = warp_max(t[k]);
            if (lane == k) mine_max = mx;
          }
          if (lane < HW) red[w * HW + lane] = mine_max;
          wg_or(wg, false);
          if (lane < HW) {
            const float *c = red + lane;
            const float mb = fmaxf(fmaxf(c[0], c[HW]), fmaxf(c[2 * HW], c[3 * HW])) * P.scale_log2;
            const float mn = fmaxf(m, mb);
            alpha[lane] = mn > m ? ex2(m - mn) : 1.f;  // both -inf: nothing yet
            m = mn;
            nm[lane] = mn == -__builtin_huge_valf() ? 0.f : -mn;
          }
          none = __any_sync(0xffffffffu, lane < HW && m == -__builtin_huge_valf());
          wg_or(wg, false);  // the maxima have been read
          if (j > j0) {
            // O^T holds PV of the block before: rescale it before this block's accumulates
            ok = __all_sync(0xffffffffu, wait_for(&pv_done[(blk - 1) % C::NR], ((blk - 1) / C::NR) & 1, failed, 91, blk));
            if (ok) {
              tc_fence_after();
#pragma unroll 1
              for (int o = 0; o < kTiles; ++o) {
                uint32_t z[HW];
                tmem_ld(lane_base + o * HP, z);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < HW; ++k) z[k] = __float_as_uint(__uint_as_float(z[k]) * alpha[k]);
                tmem_st(lane_base + o * HP, z);
              }
              tmem_st_wait();
              tc_fence_before();
            }
#pragma unroll
            for (int k = 0; k < HW; ++k) l[k] *= alpha[k];
          }
          __syncwarp();
          load_s();
          against();
        }
#pragma unroll
        for (int k = 0; k < HW; k += 8) {
          uint32_t p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float e0 = ex2(t[k + 2 * e]), e1 = ex2(t[k + 2 * e + 1]);
            p[e] = pack_bf16x2(e0, e1);
            l[k + 2 * e] += e0;
            l[k + 2 * e + 1] += e1;
          }
          const int u = (wg * HW + k) >> 3;
          *reinterpret_cast<uint4 *>(prow + ((u ^ (r & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
        }
        if (!used) {
          // zero the row in this warpgroup's share of the block's value tiles: what is there may be NaN (a lane's units
          // in its own order, so that eight rows fall on eight bank groups: 1 against 8 K cycles a block)
#pragma unroll 1
          for (int o = wg; o < kTiles; o += C::WG) {
            uint8_t *row = smem + C::kOffTiles + (kTiles * blk + o) % C::NT * kTileBytes + r * 128;
#pragma unroll
            for (int u = 0; u < 16; ++u)
              *reinterpret_cast<uint4 *>(row + (u >> 3) * kChunkBytes + (((u ^ r) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s_free[blk & 1]);
          mbar_arrive(p_full);
        }
      }
      ok = __all_sync(0xffffffffu, ok && wait_for(&pv_done[(blk - 1) % C::NR], ((blk - 1) / C::NR) & 1, failed, 92, blk));
      ok = !wg_or(wg, !ok);
      if (!ok) break;
      tc_fence_after();
      // sums over the rows: HW heads over a warp's 32 lanes by halving (lane k ends with head k), then over the warps
#pragma unroll
      for (int s = HW / 2; s >= 1; s >>= 1)
#pragma unroll
        for (int k = 0; k < s; ++k) {
          const bool up = lane & s;
          const float send = up ? l[k] : l[k + s], keep = up ? l[k + s] : l[k];
          l[k] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], 16);
      if (lane < HW) red[w * HW + lane] = l[0];
      wg_or(wg, false);
      const int64_t part = 2 * unit + (j0 > 0 ? 0 : 1);  // of the workspace arrays
      const int hw0 = h0 + wg * HW, mine_heads = min(max(heads - wg * HW, 0), HW);
      float *inv = alpha;  // this warp's copy
      if (lane < HW) {
        float sum = (red[lane] + red[HW + lane]) + (red[2 * HW + lane] + red[3 * HW + lane]);
        if (!whole) {
          if (w == 0 && lane < mine_heads) P.part_ml[part * P.H + hw0 + lane] = make_float2(m, sum);
        } else {
          // rows that are all masked leave sum = 0 and m = -inf: zeros, whatever the sink
          const bool empty = sum == 0.f;
          if (P.sink && lane < mine_heads && !empty) sum += ex2(P.sink[hw0 + lane] * 1.4426950408889634f - m);
          inv[lane] = empty ? 0.f : 1.f / sum;
        }
      }
      wg_or(wg, false);  // the sums have been read, inv is written
      __nv_bfloat16 *out = P.out + (static_cast<int64_t>(query) * P.H + hw0) * kDv;
      float *po = P.part_o + (part * P.H + hw0) * kDv;
#pragma unroll 1
      for (int o = 0; o < kTiles; ++o) {
        uint32_t z[HW];
        tmem_ld(lane_base + o * HP, z);
        tmem_ld_wait();
        if (whole) {
          // a warp stores 32 consecutive values of two heads at a time, a bf16 pair a lane
          const int d = o * 128 + w * 32 + (lane & ~1);
#pragma unroll
          for (int k = 0; k < HW; k += 2) {
            const float a = __uint_as_float(z[k]) * inv[k], b = __uint_as_float(z[k + 1]) * inv[k + 1];
            const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
            const int h = k + (lane & 1);
            if (h < mine_heads)
              *reinterpret_cast<uint32_t *>(out + h * kDv + d) = lane & 1 ? pack_bf16x2(other, b) : pack_bf16x2(a, other);
          }
        } else {
          const int d = o * 128 + w * 32 + lane;
#pragma unroll
          for (int k = 0; k < HW; ++k)
            if (k < mine_heads) po[k * kDv + d] = __uint_as_float(z[k]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *failed) record_error(P.err, DSA_ERR_DEVICE_TIMEOUT, *failed >> 24, *failed & 0xffffff);
  if (tid == 0 && bad[0]) record_error(P.err, DSA_ERR_DEVICE_BOUNDS, bad[0], bad[1]);
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// How a call is divided: groups of 16, 32 or 64 heads, a CTA each per unit, and
// as many units as fit the SMs (no more than there are blocks).  As many heads to a
// group as can be, since each group reads the rows; but where every block can have
// an SM for each of smaller groups, those, whose block is shorter (one token of 128
// heads over 1,024 rows: groups of 64 17.2 us, of 32 13.8, of 16 13.9; of 64 heads,
// 16 requests of 128 rows: 12.6 against 10.7).  Lengths are on the device, so the
// blocks are those of a full table: a wide table keeps the large groups however short
// the requests are.  Heads that a group lacks cost what they would if they were there
// (64 x 8,192 rows: 96 heads 186 us, 128 189).
struct PagedDivision {
  int group_heads, groups, units;
};

PagedDivision divide(int64_t n, int H, int max_pages, int nsel, int shift) {
  const int64_t blocks = n * paged_blocks(INT32_MAX, nsel, max_pages, shift), sms = num_sms();
  PagedDivision d{H <= 16 ? 16 : H <= 32 ? 32 : 64, 0, 0};
  for (int g = 16; g < d.group_heads; g *= 2)
    if (blocks * ((H + g - 1) / g) <= sms) d.group_heads = g;
  d.groups = (H + d.group_heads - 1) / d.group_heads;
  const int64_t fit = sms / d.groups > 0 ? sms / d.groups : 1;  // below the join's 512
  d.units = static_cast<int>(blocks < fit ? blocks : fit);
  return d;
}

size_t workspace_bytes(const PagedDivision &d, int H) {
  return static_cast<size_t>(d.units) * (2 * static_cast<size_t>(H) * (kDv * 4 + 8) + 16);
}

template <class C>
dsa_status launch(const CUtensorMap &kv_map, const void *q, const PagedAttnParams &P, cudaStream_t stream) {
  CUtensorMap q_map;
  const uint64_t dims[3] = {static_cast<uint64_t>(kD), static_cast<uint64_t>(P.H), static_cast<uint64_t>(P.n)};
  const uint64_t strides[2] = {static_cast<uint64_t>(kD) * 2, static_cast<uint64_t>(P.H) * kD * 2};
  const uint32_t box[3] = {64, C::HP, 1};
  dsa_status st = encode_tensor_map(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box,
                                    CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != DSA_OK) return st;
  static std::atomic<uint64_t> devices{0};
  cudaError_t e = allow_smem(paged_attn_kernel<C>, C::kSmemBytes, devices);
  if (e != cudaSuccess) return cuda_fail(e);
  e = launch_overlapped(paged_attn_kernel<C>, dim3(static_cast<unsigned>(P.units * P.groups)), C::kThreads, C::kSmemBytes,
                        stream, q_map, kv_map, P);
  return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_paged_attn_workspace_size(int32_t n, int32_t H, int32_t max_pages, int32_t nsel,
                                                    int32_t page_size, size_t *bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  const int shift = page_shift(page_size);
  if (n < 0 || max_pages < 1 || nsel < 0) return DSA_ERR_SHAPE;
  if (H < 1 || H > kPagedMaxHeads || shift < 0) return DSA_ERR_UNSUPPORTED;
  *bytes = n == 0 ? 0 : workspace_bytes(divide(n, H, max_pages, nsel, shift), H);
  return DSA_OK;
}

extern "C" dsa_status dsa_paged_attn(const void *q, int32_t n, const void *cache, int64_t page_stride,
                                     int64_t row_stride, int32_t num_pages, int32_t page_size,
                                     const int32_t *page_table, int32_t batch, int32_t max_pages, const int32_t *lens,
                                     const int32_t *req, const int32_t *blocks, int32_t nsel, const float *attn_sink,
                                     float softmax_scale, int32_t H, int32_t D, int32_t Dv, void *out,
                                     void *workspace, size_t ws_bytes, dsa_stream_t stream) {
  const int shift = page_shift(page_size);
  if (!(softmax_scale > 0.f) || softmax_scale > 3.4e38f) return DSA_ERR_INVALID_ARG;
  if (n < 0 || num_pages < 1 || batch < 0 || max_pages < 1 || nsel < 0) return DSA_ERR_SHAPE;
  if (static_cast<int64_t>(batch) * max_pages > INT32_MAX || static_cast<int64_t>(max_pages) * 128 > INT32_MAX ||
      static_cast<int64_t>(n) * nsel > INT32_MAX)
    return DSA_ERR_SHAPE;
  if (!req && n > batch) return DSA_ERR_SHAPE;
  if (row_stride < D || row_stride % 8 || page_stride % 8 || (num_pages > 1 && page_stride < row_stride)) return DSA_ERR_SHAPE;
  if (D != kD || Dv != kDv || H < 1 || H > kPagedMaxHeads || shift < 0) return DSA_ERR_UNSUPPORTED;
  if (n == 0) return DSA_OK;
  if (!q || !cache || !page_table || !lens || !out || (blocks != nullptr) != (nsel > 0)) return DSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
  const PagedDivision div = divide(n, H, max_pages, nsel, shift);
  const size_t need = workspace_bytes(div, H);
  if (!workspace || !aligned16(workspace) || ws_bytes < need) return DSA_ERR_WORKSPACE;
  int *err = device_error_word();
  if (!err) return DSA_ERR_CUDA;

  PagedAttnParams P{};
  P.table = page_table;
  P.lens = lens;
  P.blocks = blocks;
  P.req = req;
  P.sink = attn_sink;
  P.out = static_cast<__nv_bfloat16 *>(out);
  P.part_o = static_cast<float *>(workspace);
  P.part_ml = reinterpret_cast<float2 *>(P.part_o + static_cast<int64_t>(2) * div.units * H * kDv);
  P.joins = reinterpret_cast<int2 *>(P.part_ml + static_cast<int64_t>(2) * div.units * H);
  P.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  P.n = n;
  P.batch = batch;
  P.max_pages = max_pages;
  P.nsel = nsel;
  P.num_pages = num_pages;
  P.page_shift = shift;
  P.H = H;
  P.groups = div.groups;
  P.units = div.units;
  P.err = err;

  CUtensorMap kv_map;
  const uint64_t dims[3] = {static_cast<uint64_t>(kD), static_cast<uint64_t>(page_size), static_cast<uint64_t>(num_pages)};
  const uint64_t strides[2] = {static_cast<uint64_t>(row_stride) * 2,
                               static_cast<uint64_t>(num_pages > 1 ? page_stride : row_stride * page_size) * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(page_size), 1};
  dsa_status st = encode_tensor_map(&kv_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, cache, dims, strides, box,
                                    CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != DSA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = div.group_heads == 16   ? launch<Cfg16>(kv_map, q, P, s)
       : div.group_heads == 32 ? launch<Cfg32>(kv_map, q, P, s)
                               : launch<Cfg64>(kv_map, q, P, s);
  if (st != DSA_OK || div.units == 1) return st;
  return launch_paged_join(P, s);
}
