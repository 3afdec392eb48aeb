// MLA sparse attention over the 4-bit latent-KV cache in groups of up to 32
// heads: a tensor-parallel rank's share, or where a few queries of many heads
// would leave SMs idle (what it computes: sparse_attn_int4.cu).
//
// One CTA takes one query, one group of heads and one split of the entries, in
// blocks of 128 rows, D = 576, Dv = 512.  Both products run transposed, rows as the M = 128 side of
// the MMA and heads as N = 16 or 32:
//   S^T [128 rows x heads]    = K [rows x 576] (K-major A) * Q^T
//   O^T [128 values x heads] += V^T (the same tiles, MN-major A) * P^T,  four times
// so few heads do not leave most of an MMA empty (with heads as M = 128 they
// cost what 128 heads do), the accumulators fit one SM's tensor memory, a CTA
// needs no other CTA and S stays fp32 in one place.  An MMA of N = 16 or 32
// takes 45 cycles, the least there is (its math would be 8 or 16), 68 of them a
// block.  Up to 64 heads were built too: with N = 64 the tiles and Q leave no
// room to overlap decoding, softmax and products, and the 2-CTA kernel is as
// fast at 64 heads and nearly twice as fast at 128.
//
// 13 warps: 0-3 softmax (thread = TMEM lane = row of the block), 4 TMA for Q
// and MMA issue, 5-12 decoding, 16 rows of every block each.  Shared memory:
// tiles of 128 value columns (32 KB: what one step of O^T needs, handed back
// to the decoding as soon as that step is done), the rope tile, over which P is
// written once QK is done, Q, and the codes of the rows to come as they lie in
// the cache.
//
// The decoding warps copy their rows' codes to shared memory by cp.async a
// block ahead (loads to registers a block ahead: 78 against 71 us for 152
// queries of 16 heads and 2048 entries) and make bf16 with one
// shift, one LOP3 and one packed fma per two values.  Nothing in the roles'
// loops is a call (a failed wait or a bad index is noted and recorded at the
// end): a call's register conventions cause spills.
//
// Softmax: a head's running reference m lies within 2^8 of its maximum.  Each
// thread compares its row's logits with it, one barrier with an OR over the
// four warps decides, and only where a logit is above (and in the first block)
// are the block's maxima reduced and O^T and the sums rescaled.  P is rounded
// to bf16 for the MMA (each entry within 2^-8 of itself); logits, exponentials'
// sums and O are fp32.
//
// What bounds it: the chain of a block of 128 rows, about 6,400 cycles, half of
// them decoding; the tensor pipe is active 7 % of the time, DRAM 26 %.  152
// queries of 16 heads x 2048 entries: 64 us, 2.2 TB/s of cache bytes; 64
// queries 38 us; 4 queries, 16 parts each and their join, 11 us.
#include "sparse_attn_int4.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kD = kInt4D, kDv = kInt4Dv;
constexpr int kRows = kInt4FewRows;         // rows per block
constexpr int kThreads = 13 * 32;
constexpr int kDecodeWarps = 8, kFirstDecodeWarp = 5;
constexpr int kChunkBytes = kRows * 128;    // 64 columns of a block (128B swizzle)
constexpr int kTileBytes = 2 * kChunkBytes; // 128 value columns
constexpr int kTiles = kDv / 128;           // per block
constexpr int kQChunks = kD / 64;

constexpr int kWarpRows = kRows / kDecodeWarps;
constexpr int kRawCodes = kDv / 2, kRawScales = kDv / kInt4Block;
// a row's codes and scales as they lie in the cache; eight rows' 16-byte units fall on eight bank groups
constexpr int kRawRow = kRawCodes + kRawScales + 16;

template <int HP_>
struct FewCfg {
  static constexpr int HP = HP_;                     // heads (16 or 32; the missing ones are zero rows of Q)
  static constexpr int kSCol = kTiles * HP;          // TMEM: O^T, then two S buffers
  static constexpr int kTmemCols = HP == 32 ? 256 : 128;
  static constexpr int kOffTiles = 0;
  static constexpr int kOffRope = kTiles * kTileBytes;  // and P: [row][64 heads] bf16, HP of them used
  static constexpr int kOffQ = kOffRope + kChunkBytes;
  static constexpr int kOffRaw = kOffQ + kQChunks * HP * 128;
  static constexpr int kOffStat = kOffRaw + kRows * kRawRow;
  // floats: -m per warp and head, its rescaling factor, the warps' maxima or sums
  static constexpr int kStatNm = 0, kStatAlpha = 4 * HP, kStatRed = 8 * HP, kStatFloats = 12 * HP;
  static constexpr int kOffBar = kOffStat + kStatFloats * 4;
  static constexpr int kNumBars = 1 + 2 * kTiles + 1 + 2 + 2 + 2;
  static constexpr int kOffMisc = kOffBar + (kNumBars + 1) / 2 * 16;
  static constexpr int kSmemBytes = kOffMisc + 20 * 4 + 1024;
  static constexpr uint32_t kIdescQK = idesc_bf16(kRows, HP, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16(128, HP, true, true);
  static_assert(kSCol + 2 * HP <= kTmemCols, "TMEM budget");
  static_assert(kOffQ % 1024 == 0 && (HP * 128) % 1024 == 0, "swizzle atoms");
  static_assert(HP * kDv * 4 <= kTiles * kTileBytes, "the fp32 O fits in the tiles");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

// OR of a predicate over the softmax warps, and a barrier among them.
__device__ __forceinline__ bool softmax_or(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.cta.red.or.pred b, 1, 128, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
    sparse_attn_int4_few_kernel(const __grid_constant__ CUtensorMap q_map, const AttnInt4Params P) {
  constexpr int HP = C::HP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
  uint64_t *q_full = bars;                   // Q landed (TMA)
  uint64_t *v_full = bars + 1;               // [kTiles] a tile is decoded (8 decode warps)
  uint64_t *v_empty = v_full + kTiles;       // [kTiles] PV is done with it (MMA commit)
  uint64_t *rope_full = v_empty + kTiles;    // a block's rope columns are there (4 softmax warps)
  uint64_t *s_full = rope_full + 1;          // [2] QK done (MMA commit)
  uint64_t *s_free = s_full + 2;             // [2] S read out of TMEM (4 softmax warps)
  uint64_t *p_full = s_free + 2;             // P written (4 softmax warps)
  uint64_t *pv_done = p_full + 1;            // PV of a block done, its P (the rope tile) free (MMA commit)
  float *stat = reinterpret_cast<float *>(smem + C::kOffStat);
  // [0] tmem, [1] failed wait, [2..3] bad index, [4..16] last used entry per warp
  int32_t *misc = reinterpret_cast<int32_t *>(smem + C::kOffMisc);
  int32_t *failed = misc + 1, *bad = misc + 2, *last_used = misc + 4;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = static_cast<int>(blockIdx.x) / P.groups;  // query * splits + split
  const int h0 = (static_cast<int>(blockIdx.x) - unit * P.groups) * HP;
  const int heads = min(HP, P.H - h0);
  const int query = unit / P.splits;
  const int k0 = (unit - query * P.splits) * P.split_len;
  const int k1 = min(P.topk, k0 + P.split_len);
  const int32_t *idx_row = P.idx + static_cast<int64_t>(query) * P.topk;
  int qrow = P.q_rows ? P.q_rows[query] : query;
  if (qrow >= P.num_q_rows) {
    if (tid == 0) record_error(P.err, DSA_ERR_DEVICE_BOUNDS, 51, query);
    qrow = -1;
  }

  // Q's TMA first: its latency overlaps the scan of the index row and the set-up
  const bool q_issued = qrow >= 0;
  if (tid == 128) {  // warp 4, lane 0
    mbar_init(q_full, 1);
    fence_mbar_init();
    if (q_issued) {
      tma_prefetch_desc(&q_map);
      mbar_arrive_expect_tx(q_full, kQChunks * HP * 128);
      for (int c = 0; c < kQChunks; ++c)
        tma_load_3d(smem + C::kOffQ + c * HP * 128, &q_map, 64 * c, h0, qrow, q_full);
    }
  }
  if (tid == 0) {
    misc[1] = misc[2] = misc[3] = 0;
    for (int s = 0; s < kTiles; ++s) {
      mbar_init(&v_full[s], kDecodeWarps);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(rope_full, 4);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 4);
    }
    mbar_init(p_full, 4);
    mbar_init(pv_done, 1);
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(reinterpret_cast<uint32_t *>(&misc[0]), C::kTmemCols);
    tmem_relinquish();
  }
  // Decoding and rope copies start here already (roles below): three dependent
  // loads, entry, slot and row, run while the rest is set up.
  const int decoder = warp - kFirstDecodeWarp;
  const int own = decoder >= 0 ? kWarpRows * decoder + (lane & 15) : tid;  // the lane's row of a block
  auto entry_of = [&](int j) {
    const int k = k0 + j * kRows + own;
    return q_issued && k < k1 ? __ldg(idx_row + k) : -1;
  };
  // decoding: four lanes copy a row's 64 bytes of codes of tile t, for rows lane / 4 and 8 + lane / 4 of the warp
  uint8_t *const raw = smem + C::kOffRaw + kWarpRows * decoder * kRawRow;
  const uint32_t raw_to = smem_u32(raw) + (lane >> 2) * kRawRow + 16 * (lane & 3);
  const uint8_t *const raw_from = P.cache + 16 * (lane & 3);
  auto copy = [&](int t, int row0, int row1) {
    cp_async_16(raw_to + 64 * t, raw_from + static_cast<int64_t>(max(row0, 0)) * P.g.row_bytes + 64 * t,
                row0 >= 0 ? 16u : 0u);
    cp_async_16(raw_to + 64 * t + 8 * kRawRow, raw_from + static_cast<int64_t>(max(row1, 0)) * P.g.row_bytes + 64 * t,
                row1 >= 0 ? 16u : 0u);
    cp_async_commit();
  };
  uint4 scales = make_uint4(0u, 0u, 0u, 0u);  // half (lane >> 4) of row lane % 16
  uint32_t exponent = 0;
  auto load = [&](int rr) {
    const uint8_t *src = P.cache + static_cast<int64_t>(max(rr, 0)) * P.g.row_bytes;
    ld_once(scales, src + P.g.scales + 16 * (lane >> 4), rr >= 0);
    ld_once_u8(exponent, src + P.g.exponent, rr >= 0);
  };
  // softmax: the rope columns of the block whose rows are in `row`, eight lanes a row
  int row = -1, row_next = -1, entry = -1;
  const uint32_t rope_tile = smem_u32(smem + C::kOffRope);
  auto rope_copy = [&]() {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int rl = 4 * x + (lane >> 3), r = 32 * warp + rl, u = lane & 7;
      const int rw = __shfl_sync(0xffffffffu, row, rl);
      cp_async_16(rope_tile + r * 128 + ((u ^ (r & 7)) << 4),
                  P.cache + static_cast<int64_t>(max(rw, 0)) * P.g.row_bytes + P.g.rope + 16 * u, rw >= 0 ? 16u : 0u);
    }
    cp_async_commit();
  };
  int32_t early_bad[2] = {0, 0};  // an index out of range, before shared memory is set up
  if (warp != 4) {
    row = entry_of(0);
    row_next = entry_of(1);
    entry = entry_of(2);
    row = checked_row(P, early_bad, slot_of(P, early_bad, row, k0 + own), k0 + own);
    row_next = slot_of(P, early_bad, row_next, k0 + kRows + own);
    if (decoder >= 0) {
      load(row);
      const int row0 = __shfl_sync(0xffffffffu, row, lane >> 2), row1 = __shfl_sync(0xffffffffu, row, 8 + (lane >> 2));
#pragma unroll
      for (int t = 0; t < kTiles; ++t) copy(t, row0, row1);
    } else {
      rope_copy();
    }
  }
  // one past the split's last entry that names a row: the blocks behind it are skipped
  int last = 0;
  if (q_issued)
    for (int k = k0 + tid; k < k1; k += kThreads)
      if (__ldg(idx_row + k) >= 0) last = k + 1 - k0;
  last = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(last)));
  if (lane == 0) last_used[warp] = last;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) last = max(last, last_used[i]);

  if (early_bad[0]) {
    bad[0] = early_bad[0];
    bad[1] = early_bad[1];
  }
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  const int nb = (last + kRows - 1) / kRows;
  const int64_t part = static_cast<int64_t>(unit) * P.H + h0;  // of the workspace arrays
  __nv_bfloat16 *out = P.out + (static_cast<int64_t>(qrow) * P.H + h0) * kDv;

  if (nb == 0) {
    if (P.splits > 1) {
      if (tid < 2 * heads) P.part_ml[2 * part + tid] = make_float2(-__builtin_huge_valf(), 0.f);
    } else if (qrow >= 0) {
      for (int u = tid; u < heads * (kDv / 8); u += kThreads)
        *reinterpret_cast<uint4 *>(out + 8 * u) = make_uint4(0u, 0u, 0u, 0u);
    }
    if (q_issued) wait_for(q_full, 0, failed, 60);  // the Q load issued at the start has landed
    cp_async_wait<0>();
  } else if (warp == 4) {
    // ---------------- MMA issuer, in a fixed order: QK of a block tile by tile
    // as they are decoded, then PV, which hands the tiles back one by one.  The
    // whole warp runs the loops and one elected lane issues: descriptors and
    // addresses then live in uniform registers (alone on the SM, with a commit
    // after every eight, an MMA of N = 16 takes 42 to 45 cycles so; 55 to 59 from
    // a branch of one lane).
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
    bool ok = all_wait(q_full, 0, 61, 0);
#pragma unroll 1
    for (int i = 0; ok && i < nb; ++i) {
      const uint32_t s_tm = tmem + C::kSCol + (i & 1) * HP;
      if (i >= 2) ok = all_wait(&s_free[i & 1], ((i - 2) >> 1) & 1, 62, i);
#pragma unroll 1
      for (int t = 0; t < kTiles; ++t) {
        if (t == kTiles - 1) {  // the rope columns are there before the last tile
          ok = ok && all_wait(rope_full, i & 1, 64, i);
          if (!ok) break;
          tc_fence_after();
          if (issuer) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(s_tm, desc_add(rope_a, k * 2), desc_add(q_b, 8 * (HP * 128 >> 4) + k * 2), C::kIdescQK, 1u);
          }
          __syncwarp();
        }
        ok = ok && all_wait(&v_full[t], i & 1, 63, i);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = desc_add(k_a, static_cast<uint32_t>(t * kTileBytes) >> 4);
        const uint64_t b = desc_add(q_b, static_cast<uint32_t>(2 * t * HP * 128) >> 4);
        if (issuer) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss(s_tm, desc_add(a, (k >> 2) * (kChunkBytes >> 4) + (k & 3) * 2),
                   desc_add(b, (k >> 2) * (HP * 128 >> 4) + (k & 3) * 2), C::kIdescQK, t > 0 || k > 0 ? 1u : 0u);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (issuer) mma_commit(&s_full[i & 1]);
      __syncwarp();
      ok = all_wait(p_full, i & 1, 65, i);
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int t = 0; t < kTiles; ++t) {
        const uint64_t a = desc_add(v_a, static_cast<uint32_t>(t * kTileBytes) >> 4);
        const uint32_t d = tmem + t * HP;
        if (issuer) {
#pragma unroll
          for (int k = 0; k < kRows / 16; ++k)
            mma_ss(d, desc_add(a, k * 128), desc_add(p_b, k * 128), C::kIdescPV, i > 0 || k > 0 ? 1u : 0u);
          mma_commit(&v_empty[t]);
        }
        __syncwarp();
      }
      if (issuer) mma_commit(pv_done);
      __syncwarp();
    }
  } else if (warp >= kFirstDecodeWarp) {
    // ---------------- decoding: warp w takes rows 16w .. 16w + 15 of every
    // block, two rows per lane position (four lanes on a row's 128 columns of a
    // tile, 32 each: 16 bytes of codes, two scales).  The eight lanes of a store
    // phase hold the same unit of eight rows, and fall on eight different bank
    // groups.  A tile's codes are copied for the next block as soon as they are
    // decoded; slots are fetched one block before that, entries two.  An entry
    // that names no row reads nothing; its factors are zero.
    const int w = warp - kFirstDecodeWarp, v = lane >> 3, r8 = lane & 7;
    // the lane's place in a tile for its row 16w + r8 and unit u of its four; the other row is 1024 bytes on
    uint32_t place[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      place[u] = smem_u32(smem + C::kOffTiles) + (v >> 1) * kChunkBytes + (kWarpRows * w + r8) * 128 +
                 (((((v & 1) << 2) | u) ^ r8) << 4);
    bool ok = true;
#pragma unroll 1
    for (int j = 0; ok && j < nb; ++j) {
      row_next = checked_row(P, bad, row_next, k0 + (j + 1) * kRows + own);
      const int row_after = slot_of(P, bad, entry, k0 + (j + 2) * kRows + own);
      entry = entry_of(j + 3);
      const uint32_t factors = row >= 0 ? int4_row_factors(exponent) : 0u;
      const uint32_t fac[2] = {__shfl_sync(0xffffffffu, factors, r8), __shfl_sync(0xffffffffu, factors, 8 + r8)};
      *reinterpret_cast<uint4 *>(raw + (lane & 15) * kRawRow + kRawCodes + 16 * (lane >> 4)) = scales;
      load(row_next);
      const int next0 = __shfl_sync(0xffffffffu, row_next, lane >> 2);
      const int next1 = __shfl_sync(0xffffffffu, row_next, 8 + (lane >> 2));
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        // this tile's codes: outstanding may be those of the tiles after it in this block and before it in the next
        cp_async_wait<kTiles - 1>();
        // the lanes shuffle and read each other's copies, so they go on or give up together
        ok = __all_sync(0xffffffffu, wait_for(&v_empty[t], (j & 1) ^ 1, failed, 67, j));
        if (!ok) break;
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint8_t *src = raw + (8 * g + r8) * kRawRow;
          const uint4 code = *reinterpret_cast<const uint4 *>(src + 64 * t + 16 * v);
          const uint32_t two = *reinterpret_cast<const uint16_t *>(src + kRawCodes + 8 * t + 2 * v);
          const uint32_t f1 = __byte_perm(fac[g], 0, 0x1010), f2 = __byte_perm(fac[g], 0, 0x3232);
          const uint32_t words[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t sc = int4_scale(__byte_perm(two, 0, b == 0 ? 0x4040 : 0x4141), f1, f2);
            const uint32_t sc24 = int4_scale24(sc);
#pragma unroll
            for (int u = 2 * b; u < 2 * b + 2; ++u) {
              uint32_t o[4];
              int4_decode8(words[u], sc, sc24, o);
              st_shared_v4(place[u] + t * kTileBytes + 1024 * g, o[0], o[1], o[2], o[3]);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[t]);
        copy(t, next0, next1);
      }
      if (!ok) break;
      row = row_next;
      row_next = row_after;
    }
    cp_async_wait<0>();
  } else {
    // ---------------- softmax: thread = row of the block = TMEM lane.  Every
    // decision that guards a tcgen05.ld/st (.sync.aligned) is warp-uniform, and
    // every one that guards a barrier of the four warps is the same in all.
    // While the others decode, these warps copy the rope columns (bf16 in the
    // cache) of the next block over P, once its PV is done.
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float *nm = stat + C::kStatNm + warp * HP;        // -m of every head (0 while m is -inf), this warp's copy
    float *alpha = stat + C::kStatAlpha + warp * HP;
    float *red = stat + C::kStatRed;                  // [4 warps][HP]
    float m = -__builtin_huge_valf(), l[HP];          // m: of head `lane`, the same in all four warps
    bool none = true;                                 // some head still has m = -inf
#pragma unroll
    for (int k = 0; k < HP; ++k) l[k] = 0.f;
    const uint64_t sc2 = f2_pack(P.scale_log2, P.scale_log2);
    uint8_t *prow = smem + C::kOffRope + tid * 128;
    auto rope_done = [&]() {
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(rope_full);
    };
    rope_done();
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < nb; ++i) {
      ok = __all_sync(0xffffffffu, ok && wait_for(&s_full[i & 1], (i >> 1) & 1, failed, 68, i));
      tc_fence_after();
      const bool used = row >= 0;
      // logits against the reference, in log2 units; S stays in TMEM until the block is done, to be read again
      // where the reference has to move
      float t[HP], top = -__builtin_huge_valf();
      auto load_s = [&]() {
        uint32_t r[HP];
        tmem_ld(lane_base + C::kSCol + (i & 1) * HP, r);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < HP; ++k) t[k] = used ? __uint_as_float(r[k]) : -__builtin_huge_valf();
      };
      auto against = [&]() {
#pragma unroll
        for (int k = 0; k < HP; k += 4) {
          const float4 n4 = *reinterpret_cast<const float4 *>(nm + k);
          f2_unpack(f2_fma(f2_pack(t[k], t[k + 1]), sc2, f2_pack(n4.x, n4.y)), t[k], t[k + 1]);
          f2_unpack(f2_fma(f2_pack(t[k + 2], t[k + 3]), sc2, f2_pack(n4.z, n4.w)), t[k + 2], t[k + 3]);
        }
      };
      load_s();
      if (!none) {
        against();
#pragma unroll
        for (int k = 0; k < HP; k += 2) top = fmax3(top, t[k], t[k + 1]);
      }
      if (softmax_or(none || top > 8.f || !ok)) {
        ok = !softmax_or(!ok);
        if (!ok) break;
        // the block's maxima: of the warp's rows by head, then of the warps
        float mine = -__builtin_huge_valf();
        if (!none) load_s();
#pragma unroll
        for (int k = 0; k < HP; ++k) {
          const float mx = warp_max(t[k]);
          if (lane == k) mine = mx;
        }
        if (lane < HP) red[warp * HP + lane] = mine;
        softmax_or(false);
        float a = 1.f;
        if (lane < HP) {
          const float *c = red + lane;
          const float mb = fmaxf(fmaxf(c[0], c[HP]), fmaxf(c[2 * HP], c[3 * HP])) * P.scale_log2;
          const float mn = fmaxf(m, mb);
          a = mn > m ? ex2(m - mn) : 1.f;  // both -inf: nothing yet
          m = mn;
          nm[lane] = mn == -__builtin_huge_valf() ? 0.f : -mn;
          alpha[lane] = a;
        }
        none = __any_sync(0xffffffffu, lane < HP && m == -__builtin_huge_valf());
        softmax_or(false);  // the maxima have been read
        if (i > 0) {
          // O^T holds PV(i - 1), which is done (the rope columns waited for it): rescale it before PV(i) accumulates
#pragma unroll 1
          for (int o = 0; o < kTiles; ++o) {
            uint32_t z[HP];
            tmem_ld(lane_base + o * HP, z);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < HP; ++k) z[k] = __float_as_uint(__uint_as_float(z[k]) * alpha[k]);
            tmem_st(lane_base + o * HP, z);
          }
          tmem_st_wait();
          tc_fence_before();
#pragma unroll
          for (int k = 0; k < HP; ++k) l[k] *= alpha[k];
        }
        __syncwarp();
        load_s();
        against();
      }
#pragma unroll
      for (int k = 0; k < HP; k += 8) {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float e0 = ex2(t[k + 2 * e]), e1 = ex2(t[k + 2 * e + 1]);
          p[e] = pack_bf16x2(e0, e1);
          l[k + 2 * e] += e0;
          l[k + 2 * e + 1] += e1;
        }
        const int u = k >> 3;
        *reinterpret_cast<uint4 *>(prow + ((u ^ (tid & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s_free[i & 1]);
        mbar_arrive(p_full);
      }
      row = checked_row(P, bad, row_next, k0 + (i + 1) * kRows + own);
      row_next = slot_of(P, bad, entry, k0 + (i + 2) * kRows + own);
      entry = entry_of(i + 3);
      ok = __all_sync(0xffffffffu, wait_for(pv_done, i & 1, failed, 70, i));
      tc_fence_after();
      if (ok && i + 1 < nb) {
        rope_copy();
        rope_done();
      }
    }
    ok = !softmax_or(!ok);
    if (ok) {
      tc_fence_after();
      // sums over the rows: 32 heads over a warp's 32 lanes by halving (lane k ends with head k), then over the warps
#pragma unroll
      for (int s = HP / 2; s >= 1; s >>= 1)
#pragma unroll
        for (int k = 0; k < s; ++k) {
          const bool up = lane & s;
          const float send = up ? l[k] : l[k + s], keep = up ? l[k + s] : l[k];
          l[k] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
      if (HP < 32) l[0] += __shfl_xor_sync(0xffffffffu, l[0], 16);
      if (lane < HP) red[warp * HP + lane] = l[0];
      softmax_or(false);
      float *inv = alpha;  // this warp's copy
      const int h = lane;
      if (lane < HP) {
        float sum = (red[h] + red[HP + h]) + (red[2 * HP + h] + red[3 * HP + h]);
        if (P.splits > 1) {
          if (warp < 2 && h < heads) P.part_ml[2 * (part + h) + warp] = make_float2(m, sum);
        } else {
          // entries that all lead to no row leave sum = 0 and m = -inf: zeros, whatever the sink
          const bool empty = sum == 0.f;
          if (P.sink && h < heads && !empty) sum += ex2(P.sink[h0 + h] * 1.4426950408889634f - m);
          inv[h] = empty ? 0.f : 1.f / sum;
        }
      }
      __syncwarp();
      // O^T through shared memory (the ring: every PV is done) as rows of 512 values, then one bulk copy
      uint8_t *stage = smem + C::kOffTiles;
#pragma unroll 1
      for (int o = 0; o < kTiles; ++o) {
        uint32_t z[HP];
        tmem_ld(lane_base + o * HP, z);
        tmem_ld_wait();
        const int d = o * 128 + tid;
        if (P.splits > 1) {
#pragma unroll
          for (int k = 0; k < HP; ++k) reinterpret_cast<uint32_t *>(stage)[(k) * kDv + d] = z[k];
        } else {
#pragma unroll
          for (int k = 0; k < HP; ++k)
            reinterpret_cast<__nv_bfloat16 *>(stage)[(k) * kDv + d] =
                __float2bfloat16_rn(__uint_as_float(z[k]) * inv[k]);
        }
      }
      fence_proxy_async_smem();
      softmax_or(false);
      if (tid == 0) {
        if (P.splits > 1) bulk_store(P.part_o + part * kDv, stage, static_cast<uint32_t>(heads) * kDv * 4);
        else bulk_store(out, stage, static_cast<uint32_t>(heads) * kDv * 2);
        bulk_commit();
        bulk_wait_done();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *failed) record_error(P.err, DSA_ERR_DEVICE_TIMEOUT, *failed >> 24, *failed & 0xffffff);
  if (tid == 0 && bad[0]) record_error(P.err, DSA_ERR_DEVICE_BOUNDS, bad[0], bad[1]);
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <class C>
dsa_status launch(const void *q, int32_t n, const AttnInt4Params &P, cudaStream_t stream) {
  CUtensorMap q_map;
  const uint64_t dims[3] = {static_cast<uint64_t>(kD), static_cast<uint64_t>(P.H), static_cast<uint64_t>(P.num_q_rows)};
  const uint64_t strides[2] = {static_cast<uint64_t>(kD) * 2, static_cast<uint64_t>(P.H) * kD * 2};
  const uint32_t box[3] = {64, C::HP, 1};
  dsa_status st = encode_tensor_map(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box,
                                    CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != DSA_OK) return st;
  cudaError_t e =
      cudaFuncSetAttribute(sparse_attn_int4_few_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return cuda_fail(e);
  sparse_attn_int4_few_kernel<C>
      <<<static_cast<unsigned>(n) * P.splits * P.groups, kThreads, C::kSmemBytes, stream>>>(q_map, P);
  return check_launch();
}

}  // namespace

dsa_status launch_attn_int4_few(const void *q, int32_t n, const AttnInt4Params &P, cudaStream_t stream) {
  return P.group_heads == 16 ? launch<FewCfg<16>>(q, n, P, stream) : launch<FewCfg<32>>(q, n, P, stream);
}

}  // namespace dsa
