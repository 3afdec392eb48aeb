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
// is a thread's own loop.  Warps: sums, a warpgroup for each of four queries or two
// that take the tiles of one by turns; MMA issue; two or four that gather the mean
// keys by cp.async into a ring of tiles, page numbers a tile ahead.  Scores stay
// in shared memory as order-preserving integers, from where the warps of a query
// take them into registers, find the cut from counts and write the list in page
// order.
//
// What bounds it: a group of four queries and 1,024 pages takes 29 K cycles, of
// them 2 K to set up, 4 K to the first tile's MMA, 1.7 K a tile in the sums (1,024
// of MMA; a weight read from shared memory by a warp is 128 bytes into registers,
// 1,024 cycles a tile where none are held: 64 us against 60, and maxima run at half
// rate) and 8 K for the choice; a CTA fills an SM, so nothing hides start and
// choice.  2,048 queries of 1,024 pages 60.4 us, 569 TFLOP/s; 64 requests 10.6 us.
#include "attn_common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kHI = 64, kDI = 128;
constexpr int kRows = 128;                  // pages per tile
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

template <int QT_, int kStages_>
struct SelCfg {
  static constexpr int QT = QT_;  // queries of a group
  static constexpr int N = QT * kHI;
  static constexpr int kStages = kStages_;          // tiles in the ring
  static constexpr int kBufs = 2;                   // accumulators
  static constexpr int kSumWarps = QT == 1 ? 8 : 16, kTeamWarps = kSumWarps / QT;
  static constexpr int kMmaWarp = kSumWarps, kFirstLoadWarp = kMmaWarp + 1;
  static constexpr int kLoadWarps = QT == 1 ? 4 : 2;     // 19 warps leave a thread 96 registers
  static constexpr int kRead = QT == 1 ? 32 : 16;        // columns of an accumulator at a time
  static constexpr int kHeldWeights = QT == 1 ? 0 : 48;  // of a query's 64 in registers (8 bytes spill), the others read
  static constexpr int kThreads = 32 * (kFirstLoadWarp + kLoadWarps);
  static constexpr int kOffQ = kStages * kTileBytes;
  static constexpr int kQChunk = N * 128;
  static constexpr int kOffW = kOffQ + 2 * kQChunk;
  static constexpr int kOffBar = kOffW + QT * kHI * 4;
  static constexpr int kNumBars = 2 * kStages + 2 * kBufs;
  // [0] tmem, [1] failed, [2..3] bad, [4..7] request, [8..11] pages, [16..47] counts
  static constexpr int kOffMisc = kOffBar + (kNumBars + 1) / 2 * 16;
  static constexpr int kOffKeys = kOffMisc + 192;   // uint32 [QT][max_pages, to whole tiles]
  static constexpr int kTmemCols = kBufs * N;
  static constexpr uint32_t kIdesc = idesc_bf16(kRows, N, false, false);
};

// ReLU that keeps a NaN (fmaxf makes it 0).
__device__ __forceinline__ float relu(uint32_t x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(__uint_as_float(x)));
  return y;
}

// Scores to integers of the same order, from that of -inf (0x7fffff) up; a NaN is
// below every number and a page that is none below a NaN; 0 is kept for what does
// not take part, all bits for the pages that are always taken.
constexpr uint32_t kKeyNoPage = 1, kKeyNaN = 2, kKeyForced = 0xffffffffu;
__device__ __forceinline__ uint32_t ordered(float s) {
  if (!(s == s)) return kKeyNaN;
  const uint32_t u = __float_as_uint(s + 0.f);  // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Barrier among the warps of a team.
template <int W>
__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(W * 32) : "memory");
}

// The choice of one query by a team of W warps; `team` numbers the barrier, w the
// warp.  Warp w holds keys [w * per, w * per + per) of kq, a lane every 32nd.  The
// cut, the least key that is taken, is found from counts of the keys that reach a
// value: bit by bit by the team (a barrier each) until at most 32 keys share the
// bits found, then from those alone, one to a lane of every warp.
template <int W>
__device__ __forceinline__ void choose(const uint32_t *kq, int have, int nsel, int team, int w, int lane, int32_t *counts,
                                       uint32_t *near, int32_t *out) {
  constexpr int kHeld = 8;  // keys a lane keeps in registers
  if (have <= nsel) {
    for (int k = w * 32 + lane; k < nsel; k += W * 32) out[k] = k < have ? k : -1;
    return;
  }
  const int per = (have + 32 * W - 1) / (32 * W) * 32, first = w * per, rounds = per / 32;
  uint32_t v[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int b = first + k * 32 + lane;
    v[k] = k < rounds && b < have ? kq[b] : 0u;  // no key is 0
  }
  auto each = [&](auto f) {  // of the lane's keys
#pragma unroll
    for (int k = 0; k < kHeld; ++k) f(v[k]);
    for (int k0 = kHeld; k0 < rounds; k0 += kHeld) {
      uint32_t x[kHeld];
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int b = first + (k0 + k) * 32 + lane;
        x[k] = k0 + k < rounds && b < have ? kq[b] : 0u;
      }
#pragma unroll
      for (int k = 0; k < kHeld; ++k) f(x[k]);
    }
  };
  // the team's counts, a warp each, into c; sets of counts by turns, so that one barrier is enough
  int turn = 0;
  auto team_counts = [&](int n, int4 (&c)[W / 4]) {
    n = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n)));
    int32_t *set = counts + turn * 16 + team * W;
    turn ^= 1;
    if (lane == 0) set[w] = n;
    team_sync<W>(team);
#pragma unroll
    for (int k = 0; k < W / 4; ++k) c[k] = *reinterpret_cast<const int4 *>(set + 4 * k);
  };
  auto total_of = [&](const int4 (&c)[W / 4]) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < W / 4; ++k) n += (c[k].x + c[k].y) + (c[k].z + c[k].w);
    return n;
  };
  auto before_of = [&](const int4 (&c)[W / 4]) {  // of the warps before this one
    int n = 0;
#pragma unroll
    for (int k = 0; k < W / 4; ++k)
      n += (4 * k < w ? c[k].x : 0) + (4 * k + 1 < w ? c[k].y : 0) + (4 * k + 2 < w ? c[k].z : 0);
#pragma unroll
    for (int k = 0; k < W / 4; ++k) n += 4 * k + 3 < w ? c[k].w : 0;
    return n;
  };
  int4 c4[W / 4];
  uint32_t cut = 0;
  int n = have, above = 0, bit = 31;  // keys that reach the cut, and that reach beyond its bits
  for (; bit >= 0 && n != nsel && n - above > 32; --bit) {
    const uint32_t c = cut | 1u << bit;
    int m = 0;
    each([&](uint32_t key) { m += key >= c; });
    team_counts(m, c4);
    m = total_of(c4);
    if (m >= nsel) {
      cut = c;
      n = m;
    } else {
      above = m;
    }
  }
  if (n != nsel && bit >= 0) {
    // the keys with the bits found, in any order: the warps write them down one after another
    int mine = 0;
    auto shares = [&](uint32_t key) { return key != 0u && key >= cut && (key - cut) >> bit <= 1u; };
    each([&](uint32_t key) { mine += shares(key); });
    int at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    at -= mine;
    team_counts(mine, c4);
    const int total = total_of(c4);
    at += before_of(c4);
    uint32_t *list = near + 32 * team;
    each([&](uint32_t key) {
      if (shares(key)) list[at++] = key;
    });
    team_sync<W>(team);
    const uint32_t mykey = lane < total ? list[lane] : 0u;
    for (; bit >= 0 && n != nsel; --bit) {
      const uint32_t c = cut | 1u << bit;
      const int m = above + __popc(__ballot_sync(0xffffffffu, mykey >= c));
      if (m >= nsel) {
        cut = c;
        n = m;
      }
    }
  }
  // keys above the cut are all taken; of those equal to it the first `ties`
  int more = 0, equal = 0;
  each([&](uint32_t key) {
    more += key > cut;
    equal += key == cut;
  });
  team_counts(more, c4);
  int at = before_of(c4), ties = nsel - total_of(c4);
  team_counts(equal, c4);
  const int tied = before_of(c4);
  at += min(tied, ties);
  ties = max(ties - tied, 0);
  const uint32_t below = (1u << lane) - 1u;
  auto write = [&](uint32_t key, int b) {
    const uint32_t same = __ballot_sync(0xffffffffu, key == cut);
    const bool took = key > cut || (key == cut && __popc(same & below) < ties);
    const uint32_t taken = __ballot_sync(0xffffffffu, took);
    if (took) out[at + __popc(taken & below)] = b;
    at += __popc(taken);
    ties -= min(ties, __popc(same));
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (k < rounds) write(v[k], first + k * 32 + lane);
  for (int k = kHeld; k < rounds; ++k) {
    const int b = first + k * 32 + lane;
    write(b < have ? kq[b] : 0u, b);
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads) block_select_kernel(const SelectParams P) {
  constexpr int QT = C::QT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);  // [kStages] a tile's keys are there (load warps)
  uint64_t *k_free = k_full + C::kStages;                              // [kStages] its MMA is done (commit)
  uint64_t *a_full = k_free + C::kStages;                              // [kBufs] an accumulator is complete (commit)
  uint64_t *a_free = a_full + C::kBufs;                                // [kBufs] it has been read (sum warps)
  int32_t *misc = reinterpret_cast<int32_t *>(smem + C::kOffMisc);
  int32_t *failed = misc + 1, *bad = misc + 2;
  float *ws = reinterpret_cast<float *>(smem + C::kOffW);
  uint32_t *keys = reinterpret_cast<uint32_t *>(smem + C::kOffKeys);
  const int ld = (P.max_pages + kRows - 1) / kRows * kRows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i0 = static_cast<int>(blockIdx.x) * QT;

  if (tid == 0) {
    misc[1] = misc[2] = misc[3] = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&k_full[s], C::kLoadWarps);
      mbar_init(&k_free[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&a_full[b], 1);
      mbar_init(&a_free[b], QT == 1 ? 4 : C::kSumWarps);
    }
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(reinterpret_cast<uint32_t *>(&misc[0]), C::kTmemCols);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the kernel before may still run
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Q: rows (query, head) of 256 bytes, 16-byte unit u of a 128-byte half at u ^ (row & 7); heads behind HI are zero
  for (int x = tid; x < C::N * 16; x += C::kThreads) {
    const int r = x >> 4, u = x & 15, i = i0 + (r >> 6), h = r & 63;
    const bool there = i < P.n && h < P.HI;
    const uint4 *src = P.q + (static_cast<int64_t>(there ? i : 0) * P.HI + (there ? h : 0)) * (kDI / 8) + u;
    cp_async_16(smem_u32(smem + C::kOffQ) + (u >> 3) * C::kQChunk + r * 128 + (((u & 7) ^ (r & 7)) << 4), src,
                there ? 16u : 0u);
  }
  cp_async_commit();
  if (warp == C::kFirstLoadWarp && lane < QT) {
    // a query's request and how many pages it sees (no query, or a bad request: none)
    const int i = i0 + lane;
    int row = -1, have = 0;
    if (i < P.n) {
      row = P.req ? P.req[i] : i;
      const int64_t len = P.lens[i], pages = len > 0 ? (len + (1 << P.page_shift) - 1) >> P.page_shift : 0;
      have = static_cast<int>(min(pages, static_cast<int64_t>(P.max_pages)));
      if (len >= 0 && (row < 0 || row >= P.batch || len > static_cast<int64_t>(P.max_pages) << P.page_shift))
        record_error(P.err, DSA_ERR_DEVICE_BOUNDS, 58, i);
      if (row < 0 || row >= P.batch) have = 0;
    }
    misc[4 + lane] = row;
    misc[8 + lane] = have;
  }
  for (int x = tid; x < QT * kHI; x += C::kThreads) {
    const int i = i0 + x / kHI, h = x % kHI;
    ws[x] = i < P.n && h < P.HI ? P.w[static_cast<int64_t>(i) * P.HI + h] : 0.f;
  }
  cp_async_wait<0>();
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);

  // Runs of queries with the same request (usually one): [q0, q1), the pages and the tiles that one of them has to
  // choose from; tiles are numbered through.
  struct Run {
    int q0, q1, pages, tiles;
    const int32_t *row;
  };
  auto run_at = [&](int q0) {
    Run r;
    const int row = misc[4 + q0];
    r.q0 = q0;
    r.q1 = q0 + 1;
    r.pages = misc[8 + q0];
    while (r.q1 < QT && misc[4 + r.q1] == row) r.pages = max(r.pages, misc[8 + r.q1++]);
    r.row = P.table + static_cast<int64_t>(max(row, 0)) * P.max_pages;
    bool any = false;
    for (int q = r.q0; q < r.q1; ++q) any |= misc[8 + q] > P.nsel;
    r.tiles = any ? (r.pages + kRows - 1) / kRows : 0;
    return r;
  };
  bool ok = true;
  int tile = 0;
  if (warp >= C::kFirstLoadWarp) {
    // ---------------- gather: warp w of W takes rows 2W x + 2w + {0, 1} of a tile, x = 0, 1, .., sixteen lanes a row;
    // lane l knows the pages of its rows l, l + 32, .. in that order.  A tile is handed on when the next one's copies
    // are on their way.
    constexpr int W = C::kLoadWarps, kIds = kRows / W / 32;
    const int w = warp - C::kFirstLoadWarp, u = lane & 15;
    const uint32_t to = smem_u32(smem) + (u >> 3) * kChunkBytes;
    bool landed = true;  // the tile before has been handed on
    auto land = [&](int t) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[t % C::kStages]);
    };
    for (int q0 = 0; ok && q0 < QT;) {
      const Run r = run_at(q0);
      int next[kIds];
      auto lookup = [&](int t) {
#pragma unroll
        for (int k = 0; k < kIds; ++k) {
          const int at = 32 * k + lane, b = t * kRows + 2 * W * (at >> 1) + 2 * w + (at & 1);
          next[k] = t < r.tiles && b < r.pages ? r.row[b] : -1;
        }
      };
      lookup(0);
      for (int t = 0; t < r.tiles; ++t, ++tile) {
        int page[kIds];
#pragma unroll
        for (int k = 0; k < kIds; ++k) page[k] = next[k] >= 0 && next[k] < P.num_pages ? next[k] : -1;
        lookup(t + 1);
        const int s = tile % C::kStages;
        // no place for this tile yet: hand the one before on first
        if (!landed && !__all_sync(0xffffffffu, mbar_test(&k_free[s], ((tile / C::kStages) & 1) ^ 1))) {
          cp_async_wait<0>();
          land(tile - 1);
          landed = true;
        }
        ok = __all_sync(0xffffffffu, wait_for(&k_free[s], ((tile / C::kStages) & 1) ^ 1, failed, 93, tile));
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < kRows / W / 2; ++x) {
          const int row = 2 * W * x + 2 * w + (lane >> 4);
          const int pg = __shfl_sync(0xffffffffu, page[x / 16], 2 * (x % 16) + (lane >> 4));
          cp_async_16(to + s * kTileBytes + row * 128 + (((u & 7) ^ (row & 7)) << 4),
                      P.keys + static_cast<int64_t>(max(pg, 0)) * (kDI / 8) + u, pg >= 0 ? 16u : 0u);
        }
        cp_async_commit();
        if (!landed) {
          cp_async_wait<1>();
          land(tile - 1);
        }
        landed = false;
      }
      q0 = r.q1;
    }
    cp_async_wait<0>();
    if (ok && !landed) land(tile - 1);
  } else if (warp == C::kMmaWarp) {
    // ---------------- MMA issue: the whole warp runs the loop, one elected lane issues
    const bool issuer = elect_one();
    const uint64_t a0 = smem_desc(smem_u32(smem), 16, 1024, kLayoutSW128);
    const uint64_t b0 = smem_desc(smem_u32(smem + C::kOffQ), 16, 1024, kLayoutSW128);
    for (int q0 = 0; ok && q0 < QT;) {
      const Run r = run_at(q0);
      for (int t = 0; t < r.tiles; ++t, ++tile) {
        const int s = tile % C::kStages, buf = tile % C::kBufs;
        ok = __all_sync(0xffffffffu, wait_for(&k_full[s], (tile / C::kStages) & 1, failed, 94, tile) &&
                                         wait_for(&a_free[buf], ((tile / C::kBufs) & 1) ^ 1, failed, 95, tile));
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = desc_add(a0, static_cast<uint32_t>(s * kTileBytes) >> 4);
        if (issuer) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss(tmem + buf * C::N, desc_add(a, (k >> 2) * (kChunkBytes >> 4) + (k & 3) * 2),
                   desc_add(b0, (k >> 2) * (C::kQChunk >> 4) + (k & 3) * 2), C::kIdesc, k > 0 ? 1u : 0u);
          mma_commit(&k_free[s]);
          mma_commit(&a_full[buf]);
        }
        __syncwarp();
      }
      q0 = r.q1;
    }
  } else {
    // ---------------- sums: a warpgroup a query of a group, or every second tile of one query
    const int wg = warp >> 2, q = QT == 1 ? 0 : wg;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + q * kHI;
    const float *wq = ws + q * kHI;
    const int have = misc[8 + q];
    uint64_t held[C::kHeldWeights / 2 + 1];
#pragma unroll
    for (int k = 0; k < C::kHeldWeights / 2; ++k) held[k] = f2_pack(wq[2 * k], wq[2 * k + 1]);
    auto release = [&](int buf) {  // the accumulator is in registers
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_free[buf]);
    };
    for (int q0 = 0; ok && q0 < QT;) {
      const Run r = run_at(q0);
      const bool mine = q >= r.q0 && q < r.q1;
      auto page_of = [&](int b) { return mine && b < have ? r.row[b] : 0; };  // a turn ahead
      const int first = QT == 1 ? wg : 0, step = QT == 1 ? C::kBufs : 1;
      int next = page_of(first * kRows + (warp & 3) * 32 + lane);
      for (int t = 0; t < r.tiles; ++t, ++tile) {
        if (QT == 1 && tile % C::kBufs != wg) continue;
        const int buf = tile % C::kBufs, b = t * kRows + (warp & 3) * 32 + lane;
        const int page = next;
        next = page_of(b + step * kRows);
        ok = __all_sync(0xffffffffu, wait_for(&a_full[buf], (tile / C::kBufs) & 1, failed, 96, tile));
        if (!ok) break;
        tc_fence_after();
        if (mine) {
          uint64_t s[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < kHI; c += C::kRead) {
            uint32_t x[C::kRead];
            tmem_ld(lane_base + buf * C::N + c, x);
            tmem_ld_wait();
            if (c == kHI - C::kRead) release(buf);
            if (P.HI < kHI) {  // heads that are none: a zero row of Q, but 0 * inf is no number
#pragma unroll
              for (int k = 0; k < C::kRead; ++k)
                if (c + k >= P.HI) x[k] = 0u;
            }
#pragma unroll
            for (int k = 0; k < C::kRead; k += 4) {
              uint64_t wa, wb;
              if (c + k < C::kHeldWeights) {
                wa = held[(c + k) / 2];
                wb = held[(c + k) / 2 + 1];
              } else {
                const float4 w4 = *reinterpret_cast<const float4 *>(wq + c + k);
                wa = f2_pack(w4.x, w4.y);
                wb = f2_pack(w4.z, w4.w);
              }
              s[0] = f2_fma(wa, f2_pack(relu(x[k]), relu(x[k + 1])), s[0]);
              s[1] = f2_fma(wb, f2_pack(relu(x[k + 2]), relu(x[k + 3])), s[1]);
            }
          }
          float s0, s1, s2, s3;
          f2_unpack(s[0], s0, s1);
          f2_unpack(s[1], s2, s3);
          uint32_t key = ordered((s0 + s1) + (s2 + s3));
          if (page < 0 || page >= P.num_pages) {
            key = kKeyNoPage;
            bad[0] = 57;
            bad[1] = i0 + q;
          }
          if (b < P.keep_first || b >= have - P.keep_last) key = kKeyForced;
          keys[q * ld + b] = key;
        } else {
          release(buf);
        }
      }
      q0 = r.q1;
    }
  }
  tc_fence_before();
  ok = !__syncthreads_or(!ok);
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (warp < C::kSumWarps && ok) {
    const int q = warp / C::kTeamWarps, i = i0 + q;
    if (misc[8 + q] <= P.nsel) {
      // all its pages are taken; those that no tile was scored for are looked at here
      const int32_t *row = P.table + static_cast<int64_t>(max(misc[4 + q], 0)) * P.max_pages;
      for (int k = (warp % C::kTeamWarps) * 32 + lane; k < misc[8 + q]; k += C::kTeamWarps * 32)
        if (row[k] < 0 || row[k] >= P.num_pages) record_error(P.err, DSA_ERR_DEVICE_BOUNDS, 57, i);
    }
    if (i < P.n && P.lens[i] >= 0)
      choose<C::kTeamWarps>(keys + q * ld, misc[8 + q], P.nsel, q, warp % C::kTeamWarps, lane, misc + 16,
                            reinterpret_cast<uint32_t *>(smem), P.out + static_cast<int64_t>(i) * P.nsel);
  }
  if (tid == 0 && *failed) record_error(P.err, DSA_ERR_DEVICE_TIMEOUT, *failed >> 24, *failed & 0xffffff);
  if (tid == 0 && bad[0]) record_error(P.err, DSA_ERR_DEVICE_BOUNDS, bad[0], bad[1]);
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
  static std::atomic<uint64_t> devices{0};
  cudaError_t e = allow_smem(block_select_kernel<C>, static_cast<int>(kMaxSmem), devices);
  if (e != cudaSuccess) return cuda_fail(e);
  e = launch_overlapped(block_select_kernel<C>, dim3(static_cast<unsigned>((P.n + C::QT - 1) / C::QT)), C::kThreads, bytes,
                        stream, P);
  return e == cudaSuccess ? check_launch() : cuda_fail(e);
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
  if (HI < 1 || HI > kHI || DI != kDI || shift < 0 || smem_bytes<SelCfg<1, 2>>(max_pages) > kMaxSmem)
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
  // four queries share a request's keys where queries may share requests and there are more than fit the SMs at once,
  // two CTAs of a query to an SM (625 blocks: 304 queries 13.5 against 12.1 us, 400 13.5 against 21.4); where there are
  // no more queries than SMs a longer ring instead of a second CTA (64 of 1,024 blocks: 10.5 against 11.5 us).  All by
  // the table's width, since lengths are on the device: the scores of four queries fit beside the rest up to 4,096
  // pages, and in a wider table each query gathers its request's keys alone (600 queries of 4,096 pages 47 us, of
  // 4,097 82), however short the requests are
  if (req && n > 2 * num_sms() && smem_bytes<SelCfg<4, 3>>(max_pages) <= kMaxSmem) return launch<SelCfg<4, 3>>(P, s);
  if (n <= num_sms() && smem_bytes<SelCfg<1, 4>>(max_pages) <= kMaxSmem) return launch<SelCfg<1, 4>>(P, s);
  return launch<SelCfg<1, 2>>(P, s);
}
