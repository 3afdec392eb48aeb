// Pages worth reading, by a cheap score: for query i and complete page b of its
// request, before the page of the query's own last position,
//   S[i, b] = sum_j w[i, j] relu(q_idx[i, j] . block_keys[page(b)])
// (the lightning-indexer score, of the page's mean key instead of each token's).
// The first keep_first and the last keep_last pages are always taken, then those
// of the highest score, ties to the lower page, up to nsel; ascending, -1 behind.
//
// One CTA takes the queries of a group (four that share a request, or one), 128
// pages at a time: pages as the M = 128 side of the MMA, (query, head) pairs as
// N = 64 each, K = 128, so a page is a TMEM lane and the weighted sum over heads
// is a thread's own loop.  The mean keys of a tile are gathered by cp.async while
// the MMA of the tile before runs and the one before that is summed.  Scores stay
// in shared memory as order-preserving integers; the k-th largest is found bit by
// bit from the counts, and one pass in page order writes the list.
#include "attn_common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kHI = 64, kDI = 128;
constexpr int kRows = 128;                  // pages per tile
constexpr int kThreads = 256;
constexpr int kChunkBytes = kRows * 128;    // 64 of the 128 dims (128B swizzle)
constexpr int kTileBytes = 2 * kChunkBytes;

struct SelectParams {
  const uint4 *q;            // [n][HI][DI] bf16
  const float *w;            // [n][HI]
  const uint4 *keys;         // [num_pages][DI] bf16
  const int32_t *table, *lens, *req;
  int32_t *out;              // [n][nsel]
  int32_t n, HI, batch, max_pages, num_pages, page_shift, nsel, keep_first, keep_last;
  int *err;
};

template <int QT_>
struct SelCfg {
  static constexpr int QT = QT_;  // queries of a group
  static constexpr int N = QT * kHI;
  static constexpr int kOffQ = 2 * kTileBytes;
  static constexpr int kQChunk = N * 128;
  static constexpr int kOffW = kOffQ + 2 * kQChunk;
  static constexpr int kOffBar = kOffW + QT * kHI * 4;
  // [0] tmem, [1] failed, [2..3] bad, [4..7] request, [8..11] pages, [16..31] counts
  static constexpr int kOffMisc = kOffBar + 16;
  static constexpr int kOffKeys = kOffMisc + 128;  // uint32 [QT][max_pages, to whole tiles]
  static constexpr int kTmemCols = 2 * N;
  static constexpr uint32_t kIdesc = idesc_bf16(kRows, N, false, false);
};

// Scores to integers of the same order; a NaN is below every number, 0 is kept
// for pages that do not take part.
__device__ __forceinline__ uint32_t ordered(float s) {
  if (!(s == s)) return 1u;
  const uint32_t u = __float_as_uint(s + 0.f);  // -0 is 0
  const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
  return max(k, 2u);
}

template <class C>
__global__ void __launch_bounds__(kThreads) block_select_kernel(const SelectParams P) {
  constexpr int QT = C::QT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *done = reinterpret_cast<uint64_t *>(smem + C::kOffBar);  // [2] MMA of a tile done
  int32_t *misc = reinterpret_cast<int32_t *>(smem + C::kOffMisc);
  int32_t *failed = misc + 1, *bad = misc + 2;
  float *ws = reinterpret_cast<float *>(smem + C::kOffW);
  uint32_t *keys = reinterpret_cast<uint32_t *>(smem + C::kOffKeys);
  const int ld = (P.max_pages + kRows - 1) / kRows * kRows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i0 = static_cast<int>(blockIdx.x) * QT;

  if (tid == 0) {
    misc[1] = misc[2] = misc[3] = 0;
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(reinterpret_cast<uint32_t *>(&misc[0]), C::kTmemCols);
    tmem_relinquish();
  }
  if (tid < QT) {
    // a query's request and how many pages it sees (no query, or a bad request: none)
    const int i = i0 + tid;
    int row = -1, have = 0;
    if (i < P.n) {
      row = P.req ? P.req[i] : i;
      const int64_t len = P.lens[i], pages = len > 0 ? (len + (1 << P.page_shift) - 1) >> P.page_shift : 0;
      have = static_cast<int>(min(pages, static_cast<int64_t>(P.max_pages)));
      if (len >= 0 && (row < 0 || row >= P.batch || len > static_cast<int64_t>(P.max_pages) << P.page_shift))
        record_error(P.err, DSA_ERR_DEVICE_BOUNDS, 58, i);
      if (row < 0 || row >= P.batch) have = 0;
    }
    misc[4 + tid] = row;
    misc[8 + tid] = have;
  }
  // Q: rows (query, head) of 256 bytes, 16-byte unit u of a 128-byte half at u ^ (row & 7); heads behind HI are zero
#pragma unroll 1
  for (int x = tid; x < C::N * 16; x += kThreads) {
    const int r = x >> 4, u = x & 15, i = i0 + (r >> 6), h = r & 63;
    const bool there = i < P.n && h < P.HI;
    const uint4 *src = P.q + (static_cast<int64_t>(there ? i : 0) * P.HI + (there ? h : 0)) * (kDI / 8) + u;
    cp_async_16(smem_u32(smem + C::kOffQ) + (u >> 3) * C::kQChunk + r * 128 + (((u & 7) ^ (r & 7)) << 4), src,
                there ? 16u : 0u);
  }
  for (int x = tid; x < QT * kHI; x += kThreads) {
    const int i = i0 + x / kHI, h = x % kHI;
    ws[x] = i < P.n && h < P.HI ? P.w[static_cast<int64_t>(i) * P.HI + h] : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  const uint64_t a0 = smem_desc(smem_u32(smem), 16, 1024, kLayoutSW128);
  const uint64_t b0 = smem_desc(smem_u32(smem + C::kOffQ), 16, 1024, kLayoutSW128);

  int tile = 0;  // MMAs issued so far: buffer tile & 1, phase tile >> 1
  bool ok = true;
  // runs of queries with the same request: usually one
  for (int q0 = 0; ok && q0 < QT;) {
    const int row = misc[4 + q0];
    int q1 = q0 + 1, pages = misc[8 + q0];
    while (q1 < QT && misc[4 + q1] == row) pages = max(pages, misc[8 + q1++]);
    const int32_t *trow = P.table + static_cast<int64_t>(max(row, 0)) * P.max_pages;
    bool any = false;  // a query that has to choose
    for (int q = q0; q < q1; ++q) any |= misc[8 + q] > P.nsel;
    const int tiles = any ? (pages + kRows - 1) / kRows : 0;
    auto load = [&](int t, int buf) {
      // a page's key: 16 units by 16 lanes
#pragma unroll
      for (int x = 0; x < kRows * 16 / kThreads; ++x) {
        const int r = x * (kThreads / 16) + (tid >> 4), u = tid & 15, b = t * kRows + r;
        const int page = b < pages ? __ldg(trow + b) : -1;
        const bool there = page >= 0 && page < P.num_pages;
        cp_async_16(smem_u32(smem) + buf * kTileBytes + (u >> 3) * kChunkBytes + r * 128 + (((u & 7) ^ (r & 7)) << 4),
                    P.keys + static_cast<int64_t>(there ? page : 0) * (kDI / 8) + u, there ? 16u : 0u);
      }
      cp_async_commit();
    };
    // the scores of tile t, whose MMA was the n-th
    auto sum = [&](int t, int n) {
      const int b = t * kRows + (warp & 3) * 32 + lane;
      const int page = b < pages ? __ldg(trow + b) : 0;
      const bool there = page >= 0 && page < P.num_pages;
      ok = __all_sync(0xffffffffu, ok && wait_for(&done[n & 1], (n >> 1) & 1, failed, 93, t));
      if (!ok) return;
      tc_fence_after();
      // the two warpgroups take alternate queries, or alternate tiles where there is one query
      for (int q = QT > 1 ? warp >> 2 : 0; q < QT; q += QT > 1 ? 2 : 1) {
        if (QT == 1 ? (t & 1) != (warp >> 2) : q < q0 || q >= q1) continue;
        const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (n & 1) * C::N + q * kHI;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t x[32];
          tmem_ld32(at + 32 * half, x);
          tmem_ld_wait();
          const float *wq = ws + q * kHI + 32 * half;
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 w4 = *reinterpret_cast<const float4 *>(wq + k);
            s[0] += w4.x * fmaxf(__uint_as_float(x[k]), 0.f);
            s[1] += w4.y * fmaxf(__uint_as_float(x[k + 1]), 0.f);
            s[0] += w4.z * fmaxf(__uint_as_float(x[k + 2]), 0.f);
            s[1] += w4.w * fmaxf(__uint_as_float(x[k + 3]), 0.f);
          }
        }
        const int have = misc[8 + q];
        uint32_t key = ordered(s[0] + s[1]);
        if (!there) {
          key = 1u;
          if (b < have) {
            bad[0] = 57;
            bad[1] = i0 + q;
          }
        }
        if (b < P.keep_first || b >= have - P.keep_last) key = 0xffffffffu;
        keys[q * ld + b] = b < have ? key : 0u;
      }
      tc_fence_before();
    };
    if (tiles > 0) load(0, tile & 1);
    for (int t = 0; t < tiles; ++t, ++tile) {
      cp_async_wait<0>();
      fence_proxy_async_smem();
      tc_fence_before();
      // tile t is there; the accumulator of tile t - 2 has been read.  All threads leave together after a failed wait
      if (__syncthreads_or(!ok)) break;
      tc_fence_after();
      if (tid == 0) {
        const uint64_t a = desc_add(a0, static_cast<uint32_t>((tile & 1) * kTileBytes) >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ss(tmem + (tile & 1) * C::N, desc_add(a, (k >> 2) * (kChunkBytes >> 4) + (k & 3) * 2),
                 desc_add(b0, (k >> 2) * (C::kQChunk >> 4) + (k & 3) * 2), C::kIdesc, k > 0 ? 1u : 0u);
        mma_commit(&done[tile & 1]);
      }
      __syncwarp();
      if (t > 0)  // the MMA before has read the other buffer
        ok = __all_sync(0xffffffffu, wait_for(&done[(tile - 1) & 1], ((tile - 1) >> 1) & 1, failed, 93, t));
      if (ok && t + 1 < tiles) load(t + 1, (tile + 1) & 1);
      if (t > 0) sum(t - 1, tile - 1);
    }
    if (ok && tiles > 0) sum(tiles - 1, tile - 1);
    cp_async_wait<0>();
    tc_fence_before();
    ok = !__syncthreads_or(!ok);
    tc_fence_after();
    q0 = q1;
  }

  // ---------------- the choice: a team of warps per query
  constexpr int kTeamWarps = 8 / QT;
  const int q = warp / kTeamWarps, i = i0 + q, member = tid - q * kTeamWarps * 32;
  const int have = misc[8 + q];
  if (ok && i < P.n && P.lens[i] >= 0) {
    int32_t *out = P.out + static_cast<int64_t>(i) * P.nsel;
    if (have <= P.nsel) {
      for (int k = member; k < P.nsel; k += kTeamWarps * 32) out[k] = k < have ? k : -1;
    } else {
      const uint32_t *kq = keys + q * ld;
      int32_t *count = misc + 16;  // [2][8]: partial counts, two sets by turns
      auto team_sum = [&](int c, int turn) {
        c = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(c)));
        if (kTeamWarps == 1) return c;
        if (lane == 0) count[(turn & 1) * 8 + warp] = c;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + q), "r"(kTeamWarps * 32) : "memory");
        int s = 0;
#pragma unroll
        for (int k = 0; k < kTeamWarps; ++k) s += count[(turn & 1) * 8 + q * kTeamWarps + k];
        return s;
      };
      uint32_t cut = 0;  // the largest value that at least nsel keys reach
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = cut | 1u << bit;
        int n = 0;
        for (int b = member; b < have; b += kTeamWarps * 32) n += kq[b] >= c;
        if (team_sum(n, bit) >= P.nsel) cut = c;
      }
      int above = 0;
      for (int b = member; b < have; b += kTeamWarps * 32) above += kq[b] > cut;
      int ties = P.nsel - team_sum(above, 1);  // of the keys equal to the cut, the first so many
      if (member < 32) {
        int at = 0;
        for (int b0 = 0; b0 < have && at < P.nsel; b0 += 32) {
          const uint32_t key = b0 + lane < have ? kq[b0 + lane] : 0u;
          const uint32_t same = __ballot_sync(0xffffffffu, key == cut && b0 + lane < have);
          const uint32_t below = (1u << lane) - 1u;
          const bool take = key > cut || ((same >> lane) & 1u && __popc(same & below) < ties);
          const uint32_t taken = __ballot_sync(0xffffffffu, take);
          if (take) out[at + __popc(taken & below)] = b0 + lane;
          at += __popc(taken);
          ties -= min(ties, __popc(same));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *failed) record_error(P.err, DSA_ERR_DEVICE_TIMEOUT, *failed >> 24, *failed & 0xffffff);
  if (tid == 0 && bad[0]) record_error(P.err, DSA_ERR_DEVICE_BOUNDS, bad[0], bad[1]);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <class C>
size_t smem_bytes(int max_pages) {
  const size_t ld = (static_cast<size_t>(max_pages) + kRows - 1) / kRows * kRows;
  return C::kOffKeys + 4 * ld * C::QT + 1024;
}
constexpr size_t kMaxSmem = 227 * 1024;

template <class C>
dsa_status launch(const SelectParams &P, cudaStream_t stream) {
  const size_t bytes = smem_bytes<C>(P.max_pages);
  cudaError_t e = cudaFuncSetAttribute(block_select_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kMaxSmem));
  if (e != cudaSuccess) return cuda_fail(e);
  block_select_kernel<C><<<static_cast<unsigned>((P.n + C::QT - 1) / C::QT), kThreads, bytes, stream>>>(P);
  return check_launch();
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_block_select(const void *q_idx, const float *w, int32_t n, int32_t HI, int32_t DI,
                                       const void *block_keys, int32_t num_pages, int32_t page_size,
                                       const int32_t *page_table, int32_t batch, int32_t max_pages,
                                       const int32_t *lens, const int32_t *req, int32_t nsel, int32_t keep_first,
                                       int32_t keep_last, int32_t *blocks, dsa_stream_t stream) {
  const int shift = page_shift(page_size);
  if (n < 0 || num_pages < 1 || batch < 0 || max_pages < 1 || nsel < 1 || keep_first < 0 || keep_last < 1 ||
      static_cast<int64_t>(keep_first) + keep_last > nsel)
    return DSA_ERR_SHAPE;
  if (static_cast<int64_t>(batch) * max_pages > INT32_MAX || static_cast<int64_t>(max_pages) * 128 > INT32_MAX ||
      static_cast<int64_t>(n) * nsel > INT32_MAX)
    return DSA_ERR_SHAPE;
  if (!req && n > batch) return DSA_ERR_SHAPE;
  if (HI < 1 || HI > kHI || DI != kDI || shift < 0 || smem_bytes<SelCfg<1>>(max_pages) > kMaxSmem)
    return DSA_ERR_UNSUPPORTED;
  if (n == 0) return DSA_OK;
  if (!q_idx || !w || !block_keys || !page_table || !lens || !blocks) return DSA_ERR_INVALID_ARG;
  if (!aligned16(q_idx) || !aligned16(block_keys)) return DSA_ERR_INVALID_ARG;
  int *err = device_error_word();
  if (!err) return DSA_ERR_CUDA;
  SelectParams P{};
  P.q = static_cast<const uint4 *>(q_idx);
  P.w = w;
  P.keys = static_cast<const uint4 *>(block_keys);
  P.table = page_table;
  P.lens = lens;
  P.req = req;
  P.out = blocks;
  P.n = n;
  P.HI = HI;
  P.batch = batch;
  P.max_pages = max_pages;
  P.num_pages = num_pages;
  P.page_shift = shift;
  P.nsel = nsel;
  P.keep_first = keep_first;
  P.keep_last = keep_last;
  P.err = err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // four queries share a request's keys where queries may share requests, once they fill the SMs
  if (req && n >= 2 * num_sms() && smem_bytes<SelCfg<4>>(max_pages) <= kMaxSmem) return launch<SelCfg<4>>(P, s);
  return launch<SelCfg<1>>(P, s);
}
