// MLA sparse attention over the 4-bit latent-KV cache (row format:
// int4_common.cuh), for any number of queries down to one token:
//   l_j = softmax_scale * q[i, h, :] . k_j,  k_j the row that entry j selects
//   out[i, h, :] = sum_j e^(l_j - m) k_j[:Dv] / (sum_j e^(l_j - m) + e^(sink_h - m))
// over the entries of the query's index row that name a row; the others are
// masked wherever they stand, and a query with none gets zeros.
//
// One 2-CTA cluster per query and split of its entries, D = 576, Dv = 512, up
// to 128 heads (the rows of the M = 128 MMA; missing heads are zero rows).
// One fp32 accumulator of 128 heads x 512 values would fill an SM's tensor
// memory, so CTA c owns value columns [256c, 256c + 256) and computes the
// partial QK over latent dims [256c, 256c + 256) + [512 + 32c, 512 + 32c + 32):
// each CTA decodes its half of a row once, and one shared-memory tile serves
// as QK's K-major B and PV's MN-major B.  CTA c does the softmax of heads
// [64c, 64c + 64): it gets its peer's partial S of them, in fp32 (16 KB a block
// of 64 entries), and returns their P and the factor by which the head's O is
// to be rescaled (8.25 KB), so that both halves of a result come from one
// softmax over sums held in 32 bits.  (Exchanging whole partial S tiles in fp32
// and doing every softmax twice: 2,060 against 1,540 us for 2,048 queries; 32 KB
// each way at the link's 13.6 B/clk are 2,400 cycles of a block's time.)  P is bf16
// for the MMA, each entry within 2^-8 of itself; statistics, sums and O are
// fp32.
//
// Tensor memory (512 columns): O (256), two S buffers (2 x 64), the CTA's 256
// main Q dims as bf16 (128).  15 warps: 0-7 softmax in two warpgroups (one
// head row = one TMEM lane per thread; warpgroup w owns columns [32w, 32w + 32)
// of every block of 64 entries; of a warpgroup's four warps two have heads of
// this CTA, two heads of the peer, for which they send S and rescale O), 8 TMA
// for Q then MMA issue, 9 and 14 the copies to the peer, 10-13 the gather.
// Nothing in the roles' loops is a call (a failed wait or a bad index is noted
// and recorded at the end): a call's register conventions made the softmax
// spill, and the gather's loads drove the spilled values out of the small L1
// that 227 KB of shared memory leave.
//
// The gather reads a row's codes, scales and exponent, decodes to bf16 with
// one shift, one LOP3 and one packed fma per two values (no conversion
// instructions: those share a pipe with the softmax's packing) and stores into
// the swizzled tiles.
//
// Splits: with few queries each query's entries are divided among several
// clusters, which leave unnormalised fp32 O halves and (m, l) per head in the
// workspace; a second kernel joins them in split order (no atomics, so the
// result does not depend on timing).
//
// What bounds it: the way of a block from a freed stage to the next, decoding
// (1,500 to 2,100 cycles), QK, partial S to the peer, softmax, P to the peer,
// PV, about 12,000 cycles over four stages: a block of 64 entries every 3,000
// cycles, 1,100 of them MMA work.  76 queries of 128 heads x 2048 entries:
// 63 us, 690 TFLOP/s (58.7 us where all share their rows); 64 queries 62 us;
// 2048 queries 1.54 ms, 758 TFLOP/s (0.40 of the measured bf16 rate).
#include "sparse_attn_int4.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kD = kInt4D, kDv = kInt4Dv;
constexpr int kHeads = kInt4MaxHeads;          // M of the MMAs
constexpr int kBN = 64;              // entries per block
constexpr int kHalf = kBN / 2;       // columns per softmax warpgroup
constexpr int kStages = 4;
constexpr int kNMain = 4;            // 64-wide latent chunks per CTA (128B swizzle), plus one of 32 (64B swizzle)
constexpr int kDvc = 256;            // value columns per CTA
constexpr int kThreads = 480;
constexpr int kMaxTopk = 1 << 30;    // positions in an index row, and a few blocks behind it, are 32-bit
constexpr int kOrderedTopk = 1024;   // lists from this length on are taken longest first (divide)
constexpr int kFirstGatherWarp = 10, kPAgentWarp = 14;
constexpr int kQMain = kNMain * 128 * 128, kQTail = 128 * 64;
constexpr int kStageMain = kNMain * kBN * 128, kStageBytes = kStageMain + kBN * 64;
constexpr int kQKMainSteps = kNMain * 4, kQKSteps = kQKMainSteps + 2, kPVSteps = kBN / 16;
constexpr int kSCol = kDvc, kQCol = kSCol + 2 * kBN, kTmemCols = 512;
// A P tile (bf16, 64 entries a row): per CTA its heads' rows, and beside them their rescaling factors, so that one
// copy takes both to the peer: factors of CTA 0, rows of CTA 0, rows of CTA 1, factors of CTA 1
constexpr int kPRows = kHeads / 2 * 128, kAlphaBytes = kHeads / 2 * 4, kPMsg = kPRows + kAlphaBytes;
constexpr int kPBytes = 2 * kPRows + 1024;
constexpr int kXHalf = kHeads / 2 * kHalf * 4;  // partial S (fp32) of the peer's heads, 32 entries of them
constexpr int kXBytes = 2 * kXHalf;
constexpr int kOffStage = 0;
constexpr int kOffQStage = kOffStage + kStageBytes;  // Q main staged in stages 1..2 at start
constexpr int kOffQTail = kOffStage + kStages * kStageBytes;
constexpr int kOffP = kOffQTail + kQTail + 1024;  // of the rows
constexpr int kOffRecv = kOffP + 2 * kPBytes;
constexpr int kOffStg = kOffRecv + kXBytes;
constexpr int kOffRed = kOffStg + kXBytes;            // floats: block maxima [2 blocks][2 warpgroups][128],
constexpr int kSums = 4 * 128, kInv = 6 * 128;        // sums [2 warpgroups][128], 1 / denominator [128]
constexpr int kOffBar = kOffRed + 7 * 128 * 4;
constexpr int kNumBars = 2 + 2 * kStages + 2 * 3 + 2 * 3 + 1 + 2 * 6 + 3;
// [0] tmem, [1] failed wait, [2..3] bad index, [4..18] last used entry per warp, [20..27] masks
constexpr int kOffMisc = kOffBar + (kNumBars + 1) / 2 * 16;
constexpr int kSmemBytes = kOffMisc + 28 * 4 + 1024;
constexpr uint32_t kIdescQK = idesc_bf16(128, kBN, false, false);
constexpr uint32_t kIdescPV = idesc_bf16(128, kDvc, false, true);
static_assert(kQCol + kNMain * 32 <= kTmemCols, "TMEM budget");
static_assert(kQMain <= 2 * kStageBytes, "Q staging fits in stages 1..2");
static_assert(kStageBytes % 1024 == 0 && kPBytes % 1024 == 0 && kOffQTail % 1024 == 0 && kOffP % 1024 == 0 &&
                  kOffRecv % 1024 == 0,
              "alignment");
constexpr int kPartRow = kDvc * 4 + 16;
static_assert(kHeads * kPartRow <= kStages * kStageBytes, "the fp32 O half fits in the stages");
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

__device__ __forceinline__ float4 ld_shared_v4(uint32_t addr) {
  float4 r;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}

// mbar_test for what the peer's copies complete.
__device__ __forceinline__ bool mbar_test_cluster(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A float into the peer's shared memory.
__device__ __forceinline__ void st_cluster_f32(uint32_t raddr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(raddr), "f"(x) : "memory");
}

__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Multiply TMEM columns [c0, c1) of the warp's lanes by alpha (it runs only
// when a row's max grows by more than 2^8).  Warp-collective.
__device__ __forceinline__ void scale_o(uint32_t lane_base, int c0, int c1, float alpha) {
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    uint32_t r[32];
    tmem_ld32(lane_base + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha);
    tmem_st32(lane_base + c, r);
  }
  tmem_st_wait();
}

__global__ void __launch_bounds__(kThreads, 1)
    sparse_attn_int4_kernel(const __grid_constant__ CUtensorMap qmain_map, const __grid_constant__ CUtensorMap qtail_map,
                            const AttnInt4Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
  uint64_t *q_full = bars;                  // Q staged + tail landed (TMA)
  uint64_t *q_ready = bars + 1;             // Q main copied into TMEM, staging free (8 softmax warps)
  uint64_t *kv_full = bars + 2;             // [kStages] rows decoded (4 gather warps)
  uint64_t *kv_empty = kv_full + kStages;   // [kStages] PV done with the stage (MMA commit)
  uint64_t *s_full = kv_empty + kStages;    // [2] QK done (MMA commit)
  uint64_t *s_free = s_full + 2;            // [2] S read out of TMEM (8 softmax warps)
  uint64_t *red_full = s_free + 2;          // [2] both warpgroups' block maxima written (4 warps)
  uint64_t *recv_full = red_full + 2;       // [2] the peer's partial S of our heads landed, a half (bulk copy)
  uint64_t *staged = recv_full + 2;         // [2] partial S of the peer's heads written, a half (2 warps)
  uint64_t *stg_free = staged + 2;          // [2] the bulk copy has read that half (sender)
  uint64_t *recv_empty = stg_free + 2;      // the peer has read what we sent (one of its threads)
  uint64_t *p_own = recv_empty + 1;         // [2] P of our heads written (4 warps)
  uint64_t *p_sent = p_own + 2;             // [2] the bulk copy has read it (sender)
  uint64_t *p_msg = p_sent + 2;             // [2] P and the rescaling factors of the peer's heads landed (bulk copies)
  uint64_t *o_ready = p_msg + 2;            // [2] O is rescaled for P (8 softmax warps)
  uint64_t *p_empty = o_ready + 2;          // [2] the peer's PV has read the P that we sent (one of its threads)
  uint64_t *pv_done = p_empty + 2;          // [2] PV done, its P tile free (MMA commit)
  uint64_t *sum_full = pv_done + 2;         // both warpgroups' denominators written (4 warps)
  uint64_t *inv_full = sum_full + 1;        // 1 / denominator of all heads written (2 warps of either CTA)
  uint64_t *o_staged = inv_full + 1;        // O rows staged in smem (8 warps)
  int32_t *misc = reinterpret_cast<int32_t *>(smem + kOffMisc);
  int32_t *last_used = misc + 4;
  uint16_t *masks = reinterpret_cast<uint16_t *>(misc + 20);  // [kStages][4]: bit r of half-word w = row 16w + r is used
  float *red = reinterpret_cast<float *>(smem + kOffRed);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t crank = cluster_ctarank(), peer = crank ^ 1u;
  const int unit = static_cast<int>(blockIdx.x >> 1);  // query * splits + split
  int query = unit / P.splits;
  const int k0 = (unit - query * P.splits) * P.split_len;
  if (P.order) {  // splits == 1
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the order is still being made
    query = P.order[unit];
  }
  const int k1 = min(P.topk, k0 + P.split_len);
  const int main_dim0 = static_cast<int>(crank) * kDvc;
  const int tail_dim0 = kDv + 32 * static_cast<int>(crank);
  const int32_t *idx_row = P.idx + static_cast<int64_t>(query) * P.topk;
  int qrow = P.q_rows ? P.q_rows[query] : query;
  if (qrow >= P.num_q_rows) {
    if (tid == 0) record_error(P.err, DSA_ERR_DEVICE_BOUNDS, 51, query);
    qrow = -1;
  }

  // Q's TMA first: its latency overlaps the scan of the index row and the set-up
  const bool q_issued = qrow >= 0;
  if (tid == 256) {  // warp 8, lane 0
    mbar_init(q_full, 1);
    fence_mbar_init();
    if (q_issued) {
      tma_prefetch_desc(&qmain_map);
      mbar_arrive_expect_tx(q_full, kQMain + kQTail);
      for (int i = 0; i < kNMain; ++i)
        tma_load_3d(smem + kOffQStage + i * 16384, &qmain_map, main_dim0 + 64 * i, 0, qrow, q_full);
      tma_load_3d(smem + kOffQTail, &qtail_map, tail_dim0, 0, qrow, q_full);
    }
  }
  if (tid == 0) {
    misc[1] = misc[2] = misc[3] = 0;
    mbar_init(q_ready, 8);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&kv_full[s], 4);
      mbar_init(&kv_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 8);
      mbar_init(&red_full[b], 4);
      mbar_init(&recv_full[b], 1);
      mbar_init(&staged[b], 2);
      mbar_init(&stg_free[b], 1);
      mbar_init(&p_own[b], 4);
      mbar_init(&p_sent[b], 1);
      mbar_init(&p_msg[b], 1);
      mbar_init(&o_ready[b], 8);
      mbar_init(&p_empty[b], 1);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(recv_empty, 1);
    mbar_init(sum_full, 4);
    mbar_init(inv_full, 4);
    mbar_init(o_staged, 8);
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(reinterpret_cast<uint32_t *>(&misc[0]), kTmemCols);
    tmem_relinquish();
  }
  // The gather starts here already (roles below): three dependent loads, entry,
  // slot and row, run while the rest is set up.  Lane l of gather warp w knows
  // row 16w + l % 16 of a block, and loads for row 4q + r4 of it.
  const int own = 16 * (warp - kFirstGatherWarp) + (lane & 15), v = lane >> 2, r4 = lane & 3;
  const uint8_t *const lane_codes = P.cache + main_dim0 / 2 + 16 * v;
  const uint8_t *const lane_scales = P.cache + P.g.scales + main_dim0 / 16 + 2 * v;
  int row = -1, row_next = -1, entry = -1;
  uint4 code[4];
  uint32_t scales[4], exponent = 0;
  auto entry_of = [&](int j) {
    const int k = k0 + j * kBN + own;
    return q_issued && k < k1 ? __ldg(idx_row + k) : -1;
  };
  auto load = [&](int q, int rr) {
    const int rw = __shfl_sync(0xffffffffu, rr, 4 * q + r4);
    const int64_t at = static_cast<int64_t>(max(rw, 0)) * P.g.row_bytes;
    ld_once(code[q], lane_codes + at, rw >= 0);
    ld_once_u16(scales[q], lane_scales + at, rw >= 0);
  };
  auto load_exponent = [&](int rr) {
    ld_once_u8(exponent, P.cache + static_cast<int64_t>(max(rr, 0)) * P.g.row_bytes + P.g.exponent, rr >= 0);
  };
  int32_t early_bad[2] = {0, 0};  // an index out of range, before shared memory is set up
  if (warp >= kFirstGatherWarp && warp < kPAgentWarp) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      code[q] = make_uint4(0u, 0u, 0u, 0u);
      scales[q] = 0;
    }
    row = entry_of(0);
    row_next = entry_of(1);
    entry = entry_of(2);
    row = checked_row(P, early_bad, slot_of(P, early_bad, row, k0 + own), k0 + own);
    row_next = slot_of(P, early_bad, row_next, k0 + kBN + own);
#pragma unroll
    for (int q = 0; q < 4; ++q) load(q, row);
    load_exponent(row);
  }
  // one past the split's last entry that names a row: the blocks behind it are skipped
  int last = 0;
  if (q_issued)
    for (int k = k0 + tid; k < k1; k += kThreads)
      if (__ldg(idx_row + k) >= 0) last = k + 1 - k0;
  last = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(last)));
  if (lane == 0) last_used[warp] = last;
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) last = max(last, last_used[i]);

  int32_t *failed = misc + 1;  // site and detail of a wait that gave up
  int32_t *bad = misc + 2;     // site and position of an index that was out of range
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  const int nb = (last + kBN - 1) / kBN;
  const int64_t part = static_cast<int64_t>(unit) * P.H;  // of the workspace arrays
  __nv_bfloat16 *out_row = P.out + static_cast<int64_t>(qrow) * P.H * kDv + main_dim0;

  if (nb == 0) {
    if (P.splits > 1) {
      if (tid < P.H) P.part_ml[2 * (part + tid) + crank] = make_float2(-__builtin_huge_valf(), 0.f);
    } else if (qrow >= 0) {
      for (int u = tid; u < P.H * (kDvc / 8); u += kThreads)
        *reinterpret_cast<uint4 *>(out_row + static_cast<int64_t>(u / (kDvc / 8)) * kDv + u % (kDvc / 8) * 8) =
            make_uint4(0u, 0u, 0u, 0u);
    }
    if (q_issued) wait_for(q_full, 0, failed, 60);  // the Q load issued at the start has landed
  } else if (warp == 8) {
    // ---------------- MMA issuer, event-driven: QK(j) as soon as its rows are
    // there and its S buffer is free, PV(i) as soon as both CTAs' rows of P(i) are
    // there and O is rescaled for it; each stream in order.  The whole warp runs
    // the loop and one elected lane issues: descriptors and addresses then live
    // in uniform registers (alone on the SM, with a commit after every eight, an
    // MMA of N = 64 takes 48 to 50 cycles so; 55 to 59 from a branch of one lane).
    const bool issuer = elect_one();
    const uint32_t st_addr = smem_u32(smem + kOffStage);
    const uint64_t qk_b0 = smem_desc(st_addr, 16, 1024, kLayoutSW128);
    const uint64_t qk_t0 = smem_desc(st_addr + kStageMain, 16, 512, kLayoutSW64);
    const uint64_t qt_a0 = smem_desc(smem_u32(smem + kOffQTail), 16, 512, kLayoutSW64);
    const uint64_t pv_a0 = smem_desc(smem_u32(smem + kOffP), 16, 1024, kLayoutSW128);
    const uint64_t pv_b0 = smem_desc(st_addr, kBN * 128, 1024, kLayoutSW128);
    const uint32_t s_tm = tmem + kSCol, q_tm = tmem + kQCol;
    bool ok = __all_sync(0xffffffffu, wait_for(q_full, 0, failed, 61) && wait_for(q_ready, 0, failed, 61));
    tc_fence_after();
    int qk = 0, pv = 0;
    long long t_prog = clock64();
    while (ok && pv < nb) {
      bool progressed = false;
      if (qk < nb &&
          __all_sync(0xffffffffu, mbar_test(&kv_full[qk % kStages], (qk / kStages) & 1) &&
                                      (qk < 2 || mbar_test(&s_free[qk & 1], ((qk - 2) >> 1) & 1)))) {
        tc_fence_after();
        const uint32_t d = s_tm + (qk & 1) * kBN;
        const uint32_t so = static_cast<uint32_t>((qk % kStages) * kStageBytes) >> 4;
        const uint64_t kb = desc_add(qk_b0, so), kt = desc_add(qk_t0, so);
        if (issuer) {
#pragma unroll
          for (int k = 0; k < kQKSteps; ++k) {
            if (k < kQKMainSteps) {
              const int i = k >> 2, sub = k & 3;
              mma_ts(d, q_tm + k * 8, desc_add(kb, (i * (kBN * 128) + sub * 32) >> 4), kIdescQK, k > 0 ? 1u : 0u);
            } else {
              const int t = k - kQKMainSteps;
              mma_ss(d, desc_add(qt_a0, t * 2), desc_add(kt, t * 2), kIdescQK, 1u);
            }
          }
          mma_commit(&s_full[qk & 1]);
        }
        __syncwarp();
        ++qk;
        progressed = true;
      }
      if (pv < qk && __all_sync(0xffffffffu, mbar_test(&p_own[pv & 1], (pv >> 1) & 1) &&
                                                     mbar_test(&o_ready[pv & 1], (pv >> 1) & 1) &&
                                                     mbar_test(&p_msg[pv & 1], (pv >> 1) & 1))) {
        tc_fence_after();
        const int bi = pv & 1, si = pv % kStages;
        const uint64_t pb = desc_add(pv_a0, static_cast<uint32_t>(bi * kPBytes) >> 4);
        const uint64_t vb = desc_add(pv_b0, static_cast<uint32_t>(si * kStageBytes) >> 4);
        if (issuer) {
#pragma unroll
          for (int k = 0; k < kPVSteps; ++k)
            mma_ss(tmem, desc_add(pb, k * 2), desc_add(vb, k * 128), kIdescPV, (pv > 0 || k > 0) ? 1u : 0u);
          mma_commit(&pv_done[bi]);
          mma_commit(&kv_empty[si]);
        }
        __syncwarp();
        ++pv;
        progressed = true;
      }
      const long long now = clock64();
      if (progressed) {
        t_prog = now;
      } else if (__any_sync(0xffffffffu, now - t_prog > kWaitLimitCycles)) {
        *failed = 62 << 24 | (pv & 0xffffff);
        ok = false;
      }
    }
  } else if (warp == 9) {
    if (lane == 0) {
      // ---------------- sends the partial S of the peer's heads; the wait that ends
      // last comes last (either way round a wait that is over costs some 170 cycles)
      const uint32_t peer_recv = map_to_cta(smem_u32(smem + kOffRecv), peer);
      const uint32_t peer_full = map_to_cta(smem_u32(recv_full), peer);
      bool ok = true;
      for (int t = 0; ok && t < nb; ++t) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (w == 0 && t >= 1) ok = wait_for<true>(recv_empty, (t - 1) & 1, failed, 64, t);
          ok = ok && wait_for(&staged[w], t & 1, failed, 63, t);
          if (!ok) break;
          bulk_copy_to_peer(peer_recv + w * kXHalf, smem + kOffStg + w * kXHalf, kXHalf, peer_full + 8 * w);
          bulk_commit();
        }
        if (!ok) break;
        bulk_wait_read<1>();
        mbar_arrive(&stg_free[0]);
        bulk_wait_read0();
        mbar_arrive(&stg_free[1]);
      }
      bulk_wait_done();  // after a failed wait a copy may still be under way
    }
  } else if (warp == kPAgentWarp) {
    if (lane == 0) {
      // ---------------- sends P and the rescaling factors of our heads; to the same place in the peer's P tile
      uint8_t *msg = smem + kOffP - kAlphaBytes + crank * kPMsg;
      const uint32_t peer_msg = map_to_cta(smem_u32(msg), peer), peer_full = map_to_cta(smem_u32(p_msg), peer);
      for (int t = 0; t < nb; ++t) {
        const int b = t & 1;
        if (t >= 2 && !wait_for<true>(&p_empty[b], ((t >> 1) & 1) ^ 1, failed, 77, t)) break;
        if (!wait_for(&p_own[b], (t >> 1) & 1, failed, 65, t)) break;
        bulk_copy_to_peer(peer_msg + b * kPBytes, msg + b * kPBytes, kPMsg, peer_full + 8 * b);
        bulk_commit();
        bulk_wait_read0();
        mbar_arrive(&p_sent[b]);
      }
      bulk_wait_done();
    }
  } else if (warp >= kFirstGatherWarp) {
    if (early_bad[0]) {
      bad[0] = early_bad[0];
      bad[1] = early_bad[1];
    }
    // ---------------- gather: four warps, one on each sub-partition, so that
    // none of the softmax warps shares its issue slots with more decoding than
    // the others; warp w takes rows 16w .. 16w + 15 of every block.  Lane l
    // knows row 16w + l % 16; to decode, eight lanes take one row, 32 columns
    // each (one 16-byte load, two scales): lanes of one 8-lane store phase are
    // two neighbours of four rows, and fall on eight different bank groups.
    // The next block's codes and scales are requested before this block's are
    // decoded (row by row as they are: up to 1.5 % slower), so that a freed stage is
    // full again after the decoding alone; slots are fetched one block before
    // that, entries two.  An entry that names no row reads nothing; its factors
    // are zero.
    const int w = warp - kFirstGatherWarp;
    // the lane's place in a stage for row 4q + r4 and unit u of its four, less 512 q: place[(q & 1) * 4 + u]
    uint32_t place[8];
#pragma unroll
    for (int x = 0; x < 8; ++x)
      place[x] = (v >> 1) * (kBN * 128) + (16 * w + r4) * 128 + (((((v & 1) << 2) ^ r4) ^ x) << 4);
#pragma unroll 1
    for (int j = 0; j < nb; ++j) {
      const int s = j % kStages;
      const uint32_t sb = smem_u32(smem + kOffStage + s * kStageBytes);
      const uint32_t used = __ballot_sync(0xffffffffu, row >= 0);
      const uint32_t factors = row >= 0 ? int4_row_factors(exponent) : 0u;
      row_next = checked_row(P, bad, row_next, k0 + (j + 1) * kBN + own);
      load_exponent(row_next);
      const int row_after = slot_of(P, bad, entry, k0 + (j + 2) * kBN + own);
      entry = entry_of(j + 3);
      // stages 1 and 2 held the staged Q until the softmax warps moved it to TMEM;
      // the lanes shuffle below, so they go on or give up together
      const bool go = wait_for(&kv_empty[s], ((j / kStages) & 1) ^ 1, failed, 66, j) &&
                      ((j != 1 && j != 2) || wait_for(q_ready, 0, failed, 67, j));
      if (!__all_sync(0xffffffffu, go)) break;
      if (lane == 0) masks[4 * s + w] = static_cast<uint16_t>(used);
      uint4 now[4];
      uint32_t now_scales[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        now[q] = code[q];
        now_scales[q] = scales[q];
        load(q, row_next);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // the rope columns: bf16 in the cache, four 16-byte units a row for this CTA
        const int rl = 8 * x + (lane >> 2), r = 16 * w + rl, u = lane & 3;
        const int rw = __shfl_sync(0xffffffffu, row, rl);
        cp_async_16(sb + kStageMain + r * 64 + ((u ^ ((r >> 1) & 3)) << 4),
                    P.cache + static_cast<int64_t>(max(rw, 0)) * P.g.row_bytes + P.g.rope + 64 * crank + 16 * u,
                    rw >= 0 ? 16u : 0u);
      }
      cp_async_commit();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t fac = __shfl_sync(0xffffffffu, factors, 4 * q + r4);
        const uint32_t f1 = __byte_perm(fac, 0, 0x1010), f2 = __byte_perm(fac, 0, 0x3232);
        const uint32_t words[4] = {now[q].x, now[q].y, now[q].z, now[q].w};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t sc = int4_scale(__byte_perm(now_scales[q], 0, b == 0 ? 0x4040 : 0x4141), f1, f2);
          const uint32_t sc24 = int4_scale24(sc);
#pragma unroll
          for (int u = 2 * b; u < 2 * b + 2; ++u) {
            uint32_t o[4];
            int4_decode8(words[u], sc, sc24, o);
            st_shared_v4(sb + place[(q & 1) * 4 + u] + 512 * q, o[0], o[1], o[2], o[3]);
          }
        }
      }
      cp_async_wait<0>();
      fence_proxy_async_smem();
      warp_arrive(&kv_full[s], lane);
      row = row_next;
      row_next = row_after;
    }
    cp_async_wait<0>();
  } else {
    // ---------------- softmax: two warpgroups; thread = head row h = TMEM lane,
    // warpgroup w owns columns [32w, 32w + 32) of every block.  Every decision
    // that guards a tcgen05.ld/st (.sync.aligned) is made warp-uniform.  A warp's
    // heads are either this CTA's or the peer's (TMEM lanes belong to a warp's
    // rank in its warpgroup).
    const int h = tid & 127, w = tid >> 7;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    bool ok = __all_sync(0xffffffffu, wait_for(q_full, 0, failed, 68, -1));
    if (ok) {
      // Q main dims: staged rows (128B swizzle) -> TMEM as bf16 pairs, chunks split by warpgroup
      const uint8_t *qs = smem + kOffQStage;
#pragma unroll 1
      for (int i = w; i < kNMain; i += 2) {
        uint32_t r[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint4 x = *reinterpret_cast<const uint4 *>(qs + i * 16384 + h * 128 + ((u ^ (h & 7)) << 4));
          r[4 * u + 0] = x.x;
          r[4 * u + 1] = x.y;
          r[4 * u + 2] = x.z;
          r[4 * u + 3] = x.w;
        }
        tmem_st32(lane_base + kQCol + 32 * i, r);
      }
      tmem_st_wait();
    }
    tc_fence_before();
    warp_arrive(q_ready, lane);

    const bool ours = (warp & 3) >> 1 == static_cast<int>(crank);
    // our row and half of an exchange tile, less the tile's offset: a row of 128 bytes, unit u at u ^ (h & 7)
    const uint32_t x_row = smem_u32(smem) + w * kXHalf + (h & 63) * 128 + ((h & 7) << 4);
    const uint32_t p_row = smem_u32(smem) + h * 128 + ((h & 7) << 4);  // of the P tile
    uint8_t *my_alpha = smem + kOffP + (h < 64 ? -kAlphaBytes : 2 * kPRows) + 4 * (h & 63);
    // our 32 columns of S(j), raw q.k over this CTA's dims; the buffer is then free for QK(j+2)
    auto take_s = [&](int j, float (&x)[32]) {
      uint32_t r[32];
      tmem_ld32(lane_base + kSCol + (j & 1) * kBN + w * kHalf, r);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(r[k]);
      tc_fence_before();
      warp_arrive(&s_free[j & 1], lane);
    };
    if (!ours) {
      // ---- heads of the peer, event-driven: their partial S(js) goes to the peer
      // as soon as it is there and the last one has left; P(jp) and the rescaling
      // factors come back; PV(je) frees its P tile for the peer's next but one.
      const bool first = w == 0 && (h & 63) == 0;  // one thread
      if (first)
        for (int j = 0; j < 2; ++j) mbar_arrive_expect_tx(&p_msg[j], kPMsg);
      int js = 0, jp = 0, je = 0;
      long long t_prog = clock64();
      while (ok && jp < nb) {
        bool progressed = false;
        if (js < nb && __all_sync(0xffffffffu, mbar_test(&s_full[js & 1], (js >> 1) & 1) &&
                                                   (js == 0 || mbar_test(&stg_free[w], (js - 1) & 1)))) {
          float x[32];
          tc_fence_after();
          take_s(js, x);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            st_shared_v4((x_row + kOffStg) ^ (u << 4), __float_as_uint(x[4 * u]), __float_as_uint(x[4 * u + 1]),
                         __float_as_uint(x[4 * u + 2]), __float_as_uint(x[4 * u + 3]));
          fence_proxy_async_smem();  // the bulk copy reads the tile through the async proxy
          warp_arrive(&staged[w], lane);
          ++js;
          progressed = true;
        }
        if (je + 2 < nb && __all_sync(0xffffffffu, mbar_test(&pv_done[je & 1], (je >> 1) & 1))) {
          if (first) mbar_arrive_remote_relaxed(&p_empty[je & 1], peer);
          ++je;
          progressed = true;
        }
        if (__all_sync(0xffffffffu, mbar_test_cluster(&p_msg[jp & 1], (jp >> 1) & 1))) {
          const int b = jp & 1;
          const float alpha = *reinterpret_cast<const float *>(my_alpha + b * kPBytes);
          if (first && jp + 2 < nb) mbar_arrive_expect_tx(&p_msg[b], kPMsg);
          if (jp >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
            ok = __all_sync(0xffffffffu, wait_for(&pv_done[b ^ 1], ((jp - 1) >> 1) & 1, failed, 73, jp));
            if (!ok) break;
            tc_fence_after();
            scale_o(lane_base, w * (kDvc / 2), (w + 1) * (kDvc / 2), alpha);
            tc_fence_before();
          }
          warp_arrive(&o_ready[b], lane);
          ++jp;
          progressed = true;
        }
        const long long now = clock64();
        if (progressed) {
          t_prog = now;
        } else if (__any_sync(0xffffffffu, now - t_prog > kWaitLimitCycles)) {
          *failed = 78 << 24 | (jp & 0xffffff);
          ok = false;
        }
      }
    }
    const uint64_t sc2 = f2_pack(P.scale_log2, P.scale_log2);
    float m_used = -__builtin_huge_valf(), l = 0.f;  // m in log2 units; l over this warpgroup's columns
    // ---- a head of ours
    auto block = [&](int i, const int b) -> bool {
      if ((h & 63) == 0) mbar_arrive_expect_tx(&recv_full[w], kXHalf);
      // the block's rows were complete before its QK, too; their barrier orders the mask word read below
      const bool rows_full = mbar_try_wait_hint(&kv_full[i % kStages], (i / kStages) & 1);
      ok = wait_for(&s_full[b], (i >> 1) & 1, failed, 69, i) && wait_for<true>(&recv_full[w], i & 1, failed, 71, i);
      if (!rows_full) ok = ok && wait_for(&kv_full[i % kStages], (i / kStages) & 1, failed, 71, i);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return false;
      tc_fence_after();
      float x[32];
      take_s(i, x);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float4 t = ld_shared_v4((x_row + kOffRecv) ^ (u << 4));
        f2_unpack(f2_add(f2_pack(x[4 * u], x[4 * u + 1]), f2_pack(t.x, t.y)), x[4 * u], x[4 * u + 1]);
        f2_unpack(f2_add(f2_pack(x[4 * u + 2], x[4 * u + 3]), f2_pack(t.z, t.w)), x[4 * u + 2], x[4 * u + 3]);
      }
      const uint32_t used = reinterpret_cast<const uint32_t *>(masks)[2 * (i % kStages) + w];
      if (used != 0xffffffffu) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (!((used >> k) & 1u)) x[k] = -__builtin_huge_valf();
      }
      float m3[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        m3[q] = fmax3(fmax3(x[8 * q], x[8 * q + 1], x[8 * q + 2]), fmax3(x[8 * q + 3], x[8 * q + 4], x[8 * q + 5]),
                      fmaxf(x[8 * q + 6], x[8 * q + 7]));
      red[(b * 2 + w) * 128 + h] = fmaxf(fmax3(m3[0], m3[1], m3[2]), m3[3]);
      warp_arrive(&red_full[b], lane);
      // PV(i-2) and the copy to the peer have read P(i-2)?
      const uint32_t before = ((i >> 1) & 1) ^ 1;  // parity of block i-2
      const bool p_free =
          __all_sync(0xffffffffu, i < 2 || (mbar_test(&pv_done[b], before) && mbar_test(&p_sent[b], before)));
      ok = __all_sync(0xffffffffu, wait_for(&red_full[b], (i >> 1) & 1, failed, 72, i));
      if (!ok) return false;
      if (w == 0 && (h & 63) == 0) mbar_arrive_remote_relaxed(recv_empty, peer);  // all four warps have read it
      const float mblk = fmaxf(red[(b * 2) * 128 + h], red[(b * 2 + 1) * 128 + h]) * P.scale_log2;  // log2 units
      // lazy rescale: only when some row of the warp saw its max grow by more
      // than 2^8.  Both warpgroups see the same row maxima, so they decide alike.
      float alpha = 1.f;
      const bool moved = __any_sync(0xffffffffu, mblk > m_used + 8.f);
      if (moved) {
        const float m_new = fmaxf(m_used, mblk);
        if (m_new > m_used) alpha = ex2(m_used - m_new);  // else both may be -inf: nothing yet
        l *= alpha;
        m_used = m_new;
      }
      uint32_t packed[16];
      // while no entry has been seen, m is -inf and every x too: any finite m gives e^x = 0
      const float nm = m_used == -__builtin_huge_valf() ? 0.f : -m_used;
      const uint64_t nm2 = f2_pack(nm, nm);
      uint64_t acc[2] = {0, 0};  // +0.0f pairs
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        float t0, t1;
        f2_unpack(f2_fma(f2_pack(x[k], x[k + 1]), sc2, nm2), t0, t1);
        const float e0 = ex2(t0), e1 = ex2(t1);
        packed[k >> 1] = pack_bf16x2(e0, e1);
        acc[(k >> 1) & 1] = f2_add(acc[(k >> 1) & 1], f2_pack(e0, e1));
      }
      float s0, s1, s2, s3;
      f2_unpack(acc[0], s0, s1);
      f2_unpack(acc[1], s2, s3);
      l += (s0 + s1) + (s2 + s3);
      if (!p_free) {
        ok = __all_sync(0xffffffffu, wait_for(&pv_done[b], before, failed, 73, i) &&
                                         wait_for(&p_sent[b], before, failed, 79, i));
        if (!ok) return false;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        st_shared_v4((p_row + kOffP + b * kPBytes) ^ ((w * 4 + u) << 4), packed[4 * u], packed[4 * u + 1],
                     packed[4 * u + 2], packed[4 * u + 3]);
      if (w == 0) *reinterpret_cast<float *>(my_alpha + b * kPBytes) = alpha;
      fence_proxy_async_smem();
      warp_arrive(&p_own[b], lane);
      if (moved && i >= 1) {
        // O holds PV(i-1): rescale this warpgroup's half of it before PV(i) accumulates; P(i) is on its way meanwhile
        ok = __all_sync(0xffffffffu, wait_for(&pv_done[b ^ 1], ((i - 1) >> 1) & 1, failed, 73, i));
        if (!ok) return false;
        tc_fence_after();
        scale_o(lane_base, w * (kDvc / 2), (w + 1) * (kDvc / 2), alpha);
        tc_fence_before();
      }
      warp_arrive(&o_ready[b], lane);
      return true;
    };
    if (ours) {
      for (int i = 0; ok && i < nb; i += 2) {
        ok = block(i, 0);
        if (ok && i + 1 < nb) ok = block(i + 1, 1);
      }
    }
    ok = __all_sync(0xffffffffu, ok && wait_for(&pv_done[(nb - 1) & 1], ((nb - 1) >> 1) & 1, failed, 74, nb));
    if (ours) {
      // the two warpgroups' partial sums of the softmax denominator
      red[kSums + w * 128 + h] = l;
      warp_arrive(sum_full, lane);
      ok = __all_sync(0xffffffffu, wait_for(sum_full, 0, failed, 75) && ok);
      l = red[kSums + h] + red[kSums + 128 + h];
      if (w == 0 && P.splits == 1) {
        // entries that all lead to no row leave l = 0 and m = -inf: zeros, whatever the sink (its power would be
        // e^(-inf + inf) for a sink of -inf); a NaN among the logits is a NaN in l
        const bool none = l == 0.f;
        if (P.sink && h < P.H && !none) l += ex2(P.sink[h] * 1.4426950408889634f - m_used);
        const float inv = none ? 0.f : 1.f / l;
        red[kInv + h] = inv;
        st_cluster_f32(map_to_cta(smem_u32(red + kInv + h), peer), inv);
        warp_arrive(inv_full, lane);
        if (lane == 0) mbar_arrive_remote(inv_full, peer);
      }
    }
    tc_fence_after();
    uint8_t *ost = smem + kOffStage;  // free: every PV is done
    if (P.splits == 1) {
      ok = __all_sync(0xffffffffu, wait_for<true>(inv_full, 0, failed, 75, 1) && ok);
      const float inv = red[kInv + h];
      // normalised rows through shared memory, 16-byte unit u of row h at
      // u ^ (h & 31), so that neither the row-wise writes nor the reads
      // collide; then each warp stores whole 512-byte rows
      if (ok) {
#pragma unroll 1
        for (int c = w * (kDvc / 2); c < (w + 1) * (kDvc / 2); c += 32) {
          uint32_t r[32];
          tmem_ld32(lane_base + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            const int u = (c + k) >> 3;
            *reinterpret_cast<uint4 *>(ost + h * 512 + ((u ^ (h & 31)) << 4)) =
                make_uint4(pack_bf16x2(__uint_as_float(r[k + 0]) * inv, __uint_as_float(r[k + 1]) * inv),
                           pack_bf16x2(__uint_as_float(r[k + 2]) * inv, __uint_as_float(r[k + 3]) * inv),
                           pack_bf16x2(__uint_as_float(r[k + 4]) * inv, __uint_as_float(r[k + 5]) * inv),
                           pack_bf16x2(__uint_as_float(r[k + 6]) * inv, __uint_as_float(r[k + 7]) * inv));
          }
        }
      }
      warp_arrive(o_staged, lane);
      ok = __all_sync(0xffffffffu, wait_for(o_staged, 0, failed, 76) && ok);
      if (ok) {
#pragma unroll 4
        for (int hh = warp; hh < P.H; hh += 8) {
          const uint4 x = *reinterpret_cast<const uint4 *>(ost + hh * 512 + ((lane ^ (hh & 31)) << 4));
          *reinterpret_cast<uint4 *>(out_row + static_cast<int64_t>(hh) * kDv + lane * 8) = x;
        }
      }
    } else {
      // this split's part: O as it is (fp32), a row's 1 KB through shared memory
      // (16 bytes apart, so that the row-wise writes do not collide) and one
      // bulk copy per row
      if (ok) {
#pragma unroll 1
        for (int c = w * (kDvc / 2); c < (w + 1) * (kDvc / 2); c += 32) {
          uint32_t r[32];
          tmem_ld32(lane_base + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<uint4 *>(ost + h * kPartRow + (c + k) * 4) =
                make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
        }
        if (ours && w == 0 && h < P.H)
          reinterpret_cast<float4 *>(P.part_ml)[part + h] = make_float4(m_used, l, m_used, l);
      }
      fence_proxy_async_smem();
      warp_arrive(o_staged, lane);
      if (w == 0 && wait_for(o_staged, 0, failed, 76) && ok && h < P.H) {
        bulk_store(P.part_o + (part + h) * kDv + main_dim0, ost + h * kPartRow, kDvc * 4);
        bulk_commit();
        bulk_wait_done();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *failed) record_error(P.err, DSA_ERR_DEVICE_TIMEOUT, *failed >> 24, *failed & 0xffffff);
  if (tid == 0 && bad[0]) record_error(P.err, DSA_ERR_DEVICE_BOUNDS, bad[0], bad[1]);
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  cluster_sync();  // no CTA leaves while its peer may still touch its smem
}

// How a call is divided: over CTA pairs with all heads (this file), or over
// single CTAs with groups of 16 or 32 heads (sparse_attn_int4_few.cu), and over
// splits of a query's entries.  The times below are what the kernels took, in
// us, for 1 to 256 queries of 2048 entries in 1 to 32 splits, to about 10 %:
//   a wave of pairs       10 + 1.6 per block of  64 entries (any number of heads)
//   a wave of 16-head CTAs 4 + 3.7 per block of 128
//   a wave of 32-head CTAs 4.5 + 4.1 per block of 128
//   joining splits         3 + the parts written and read at 5 TB/s
// Measured with each way forced (pairs / groups of 16 / of 32, us, rows in L2):
//   128 heads,  1 query   15.4 /  11.5 /  13.0    128 heads, 64 queries  59.6 / 230 / 120
//    32 heads, 64 queries 56.5 /  54.4 /  38.3     16 heads, 64 queries  56.2 /  33 /  35
// Pairs win where there are many heads and enough queries for the SMs, groups up
// to 32 heads, and for a query or two of many heads, whose splits alone do not
// fill the SMs.
//
// Two to four waves of pairs over long lists take the queries in the order of
// their lists' lengths (sparse_attn_int4_order.cu; one more load before a pair
// can start, and a small launch).  us for 2048 entries and 128 heads, lengths
// log-uniform to 3000 / all lists full, in the order given -> longest first:
//   152 queries  79.7 -> 64.2 / 124 -> 128     256  111 -> 83 / 245 -> 251
// One wave and a half gains little more than it costs (100 queries 69.3 -> 62.9
// / 117 -> 122), lists of 512 the less (200 queries 51.7 -> 49.2 / 70 -> 75); of
// many waves the last matters little (1000 queries: 311 -> 310 / 853 -> 880),
// and groups of 16 heads pay more for the load (400 queries 86 -> 68 / 180 ->
// 191).
struct Division {
  int splits, split_len, group_heads;  // group_heads 0: pairs
  bool ordered;                        // by the length of the queries' lists
};

Division divide(int64_t n, int H, int topk) {
  struct Way {
    int group_heads, rows;
    double fixed, block;
  };
  const Way ways[3] = {{0, kBN, 10.0, 1.6}, {16, kInt4FewRows, 4.0, 3.7}, {32, kInt4FewRows, 4.5, 4.1}};
  const int sms = num_sms();
  Division best{1, 0, 0, false};
  double best_cost = 1e300;
  for (const Way &w : ways) {
    const int blocks = (topk + w.rows - 1) / w.rows;
    const int groups = w.group_heads ? (H + w.group_heads - 1) / w.group_heads : 1;
    const int units = w.group_heads ? sms : sms > 1 ? sms / 2 : 1;
    for (int s = 1; s <= blocks && s <= kInt4MaxSplits; ++s) {
      const int per = (blocks + s - 1) / s;
      if ((blocks + per - 1) / per != s) continue;  // the same division as a smaller s
      const double waves = static_cast<double>((n * s * groups + units - 1) / units);
      const double parts = static_cast<double>(n * s) * H * (2 * kDv * 4) / 5e6;
      const double cost = waves * (w.fixed + w.block * per) + (s > 1 ? 3.0 + parts : 0.0);
      if (cost < best_cost) {
        best_cost = cost;
        const bool ordered = !w.group_heads && s == 1 && n >= 2 * units && n <= 4 * units && n <= kInt4MaxOrdered &&
                             topk >= kOrderedTopk;
        best = {s, per * w.rows, w.group_heads, ordered};
      }
    }
  }
  return best;
}

size_t workspace_bytes(int64_t n, const Division &d, int H) {
  if (d.ordered) return static_cast<size_t>(n) * 4;
  return d.splits > 1 ? static_cast<size_t>(n) * d.splits * H * (kDv * 4 + 16) : 0;
}

dsa_status launch_pairs(const void *q, int32_t n, const AttnInt4Params &P, cudaStream_t stream) {
  CUtensorMap qmain, qtail;
  const uint64_t dims[3] = {static_cast<uint64_t>(kD), static_cast<uint64_t>(P.H), static_cast<uint64_t>(P.num_q_rows)};
  const uint64_t strides[2] = {static_cast<uint64_t>(kD) * 2, static_cast<uint64_t>(P.H) * kD * 2};
  const uint32_t box_main[3] = {64, kHeads, 1}, box_tail[3] = {32, kHeads, 1};
  dsa_status st = encode_tensor_map(&qmain, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box_main,
                                    CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != DSA_OK) return st;
  st = encode_tensor_map(&qtail, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box_tail,
                         CU_TENSOR_MAP_SWIZZLE_64B);
  if (st != DSA_OK) return st;
  cudaError_t e = cudaFuncSetAttribute(sparse_attn_int4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return cuda_fail(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n) * P.splits * 2u);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = P.order ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, sparse_attn_int4_kernel, qmain, qtail, P);
  if (e != cudaSuccess) return cuda_fail(e);
  return check_launch();
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_sparse_attn_int4kv_workspace_size(int32_t n, int32_t H, int32_t topk, size_t *bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  if (n < 0 || topk < 1 || topk > kMaxTopk) return DSA_ERR_SHAPE;
  if (H < 1 || H > kHeads) return DSA_ERR_UNSUPPORTED;
  *bytes = n == 0 ? 0 : workspace_bytes(n, divide(n, H, topk), H);
  return DSA_OK;
}

extern "C" dsa_status dsa_sparse_attn_int4kv_division(int32_t n, int32_t H, int32_t topk, int32_t *splits,
                                                      int32_t *group_heads, int32_t *longest_first) {
  if (n < 0 || topk < 1 || topk > kMaxTopk) return DSA_ERR_SHAPE;
  if (H < 1 || H > kHeads) return DSA_ERR_UNSUPPORTED;
  const Division d = divide(n, H, topk);
  if (splits) *splits = d.splits;
  if (group_heads) *group_heads = d.group_heads;
  if (longest_first) *longest_first = d.ordered ? 1 : 0;
  return DSA_OK;
}

extern "C" dsa_status dsa_sparse_attn_int4kv(const void *q, int32_t num_q_rows, const int32_t *q_rows, int32_t n,
                                             const void *kv_cache, int32_t num_cache_rows, const int32_t *slots,
                                             int32_t num_kv_rows, const int32_t *topk_idx, int32_t topk,
                                             const float *attn_sink, float softmax_scale, int32_t H, int32_t D,
                                             int32_t Dv, void *out, void *workspace, size_t ws_bytes,
                                             dsa_stream_t stream) {
  if (!(softmax_scale > 0.f) || softmax_scale > 3.4e38f) return DSA_ERR_INVALID_ARG;
  if (n < 0 || num_q_rows < 0 || num_cache_rows < 1 || num_kv_rows < 0 || topk < 1 || topk > kMaxTopk)
    return DSA_ERR_SHAPE;
  if (!q_rows && n > num_q_rows) return DSA_ERR_SHAPE;
  if (D != kD || Dv != kDv || H < 1 || H > kHeads) return DSA_ERR_UNSUPPORTED;
  if (n == 0 || num_q_rows == 0) return DSA_OK;
  if (!q || !kv_cache || !topk_idx || !out) return DSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
  const Division div = divide(n, H, topk);
  const size_t need = workspace_bytes(n, div, H);
  if (need > 0 && (!workspace || !aligned16(workspace) || ws_bytes < need)) return DSA_ERR_WORKSPACE;
  if (static_cast<int64_t>(n) * div.splits * (kHeads / 16) > INT32_MAX) return DSA_ERR_SHAPE;
  int *err = device_error_word();
  if (!err) return DSA_ERR_CUDA;

  AttnInt4Params P{};
  P.cache = static_cast<const uint8_t *>(kv_cache);
  P.slots = slots;
  P.idx = topk_idx;
  P.q_rows = q_rows;
  P.sink = attn_sink;
  P.out = static_cast<__nv_bfloat16 *>(out);
  P.part_o = static_cast<float *>(workspace);
  P.part_ml =
      reinterpret_cast<float2 *>(static_cast<float *>(workspace) + static_cast<int64_t>(n) * div.splits * H * kDv);
  P.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  P.H = H;
  P.topk = topk;
  P.splits = div.splits;
  P.split_len = div.split_len;
  P.group_heads = div.group_heads;
  P.groups = div.group_heads ? (H + div.group_heads - 1) / div.group_heads : 1;
  P.num_kv_rows = num_kv_rows;
  P.cache_rows = num_cache_rows;
  P.num_q_rows = num_q_rows;
  dsa_status st = int4_geom(D, Dv, &P.g);
  if (st != DSA_OK) return st;
  P.err = err;

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (div.ordered) {
    int32_t *order = static_cast<int32_t *>(workspace);
    st = launch_attn_int4_order(n, P, order, s);
    if (st != DSA_OK) return st;
    P.order = order;
  }
  st = div.group_heads ? launch_attn_int4_few(q, n, P, s) : launch_pairs(q, n, P, s);
  if (st != DSA_OK || div.splits == 1) return st;
  return launch_attn_int4_join(n, P, s);
}
