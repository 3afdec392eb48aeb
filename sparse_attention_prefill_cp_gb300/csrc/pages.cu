// The paged latent cache around the attention: page tables grown and shrunk out
// of a list of free pages, the slots that rows get, and rows written into them.
//
// A page holds P rows; position p of request b lies in slot
// page_table[b][p / P] * P + p % P.
#include "dsa_common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kUpdateThreads = 1024;

struct PagesUpdate {
  int32_t *table, *free_pages, *free_count;
  const int32_t *held, *seq;
  int32_t batch, max_pages, num_pages, page_shift;
  int *err;
};

__device__ __forceinline__ int pages_of(int rows, int shift) {
  return static_cast<int>((static_cast<int64_t>(rows) + (1 << shift) - 1) >> shift);
}

// Sum of (released, grown) pages over the block's threads before this one, and
// in total; both counts of a call fit 32 bits (checked on the host).
__device__ __forceinline__ uint2 scan_pair(uint2 x, uint2 &total, uint2 *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint2 s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, s.x, o), b = __shfl_up_sync(0xffffffffu, s.y, o);
    if (lane >= o) {
      s.x += a;
      s.y += b;
    }
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  uint2 w = warp_sums[lane];  // as many warps as lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, w.x, o), b = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += a;
      w.y += b;
    }
  }
  total.x = __shfl_sync(0xffffffffu, w.x, 31);
  total.y = __shfl_sync(0xffffffffu, w.y, 31);
  const uint32_t bx = __shfl_sync(0xffffffffu, w.x, max(warp - 1, 0)), by = __shfl_sync(0xffffffffu, w.y, max(warp - 1, 0));
  __syncthreads();
  return make_uint2(s.x - x.x + (warp ? bx : 0u), s.y - x.y + (warp ? by : 0u));
}

// Pages of a batch for new lengths.  With R pages released and G taken in all,
// both numbered request by request and page by page, and c free pages before:
//   released page j goes to free[c + R - 1 - j], taken page k comes from
//   free[c + R - 1 - k],
// a stack on which the releases are pushed last request first: what a call took,
// a call with the lengths exchanged gives back to the same places, and the
// result depends on nothing but the inputs.  1,024 requests at a time: a scan
// numbers their pages, then the threads share the pages out evenly, each finding
// its page's request by bisection (a warp a request instead: 27 against 10 us for
// 16 prompts of 68,569 rows taken, named and given back).  Everything is checked before anything is written.
// One block: a step of a decode batch touches a page in P requests, and is a
// launch and four dependent loads long.
__global__ void __launch_bounds__(kUpdateThreads) pages_update_kernel(const PagesUpdate P) {
  __shared__ uint2 warp_sums[32];
  __shared__ int32_t bad[2];
  __shared__ uint32_t start[kUpdateThreads];  // of a request's pages among the chunk's
  __shared__ int32_t page0[kUpdateThreads];   // the first of them
  const int tid = threadIdx.x;
  const int64_t limit = static_cast<int64_t>(P.max_pages) << P.page_shift;
  if (tid == 0) bad[0] = bad[1] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the kernel before may still run
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t count = *P.free_count;
  __syncthreads();
  auto change = [&](int b, int &had, int &need) {
    had = need = 0;
    if (b >= P.batch) return;
    const int h = P.held[b], s = P.seq[b];
    if (h < 0 || s < 0 || h > limit || s > limit) {
      bad[0] = 52;
      bad[1] = b;
      return;
    }
    had = pages_of(h, P.page_shift);
    need = pages_of(s, P.page_shift);
  };
  // the pages of requests b0.. that are released (or taken), numbered in order: do_page(request, page, number);
  // returns their count, and the chunk's count of the other kind in `other`
  auto each_page = [&](int b0, bool released, uint32_t &other, auto do_page) {
    int had, need;
    change(b0 + tid, had, need);
    const int from = released ? need : had, to = released ? had : need;
    uint2 total;
    const uint2 before = scan_pair(make_uint2(max(to - from, 0), max(from - to, 0)), total, warp_sums);
    start[tid] = before.x;
    page0[tid] = from;
    __syncthreads();
    for (uint32_t i = tid; i < total.x; i += kUpdateThreads) {
      int lo = 0;
#pragma unroll
      for (int d = kUpdateThreads / 2; d; d >>= 1)  // the last request that starts at or before i
        if (start[lo + d] <= i) lo += d;
      do_page(b0 + lo, page0[lo] + static_cast<int>(i - start[lo]), i);
    }
    __syncthreads();
    other = total.y;
    return total.x;
  };
  int64_t R = 0, G = 0;
  auto refused = [&]() {
    if (!bad[0] && count >= 0 && count + R <= P.num_pages && G <= count + R) return false;
    if (tid == 0) record_error(P.err, DSA_ERR_DEVICE_BOUNDS, bad[0] ? bad[0] : 54, bad[0] ? bad[1] : static_cast<int>(G));
    return true;
  };
  if (P.batch <= kUpdateThreads) {
    // one look at the lengths and one scan for both kinds (update, slots and update back for 64 requests: 8.6 -> 7.2 us)
    int had, need;
    change(tid, had, need);
    uint2 total;
    const uint2 before = scan_pair(make_uint2(max(had - need, 0), max(need - had, 0)), total, warp_sums);
    R = total.x;
    G = total.y;
    page0[tid] = min(had, need);
    for (int released = 1; released >= 0; --released) {
      const uint32_t n = released ? total.x : total.y;
      if (n == 0) {
        if (released && refused()) return;
        continue;
      }
      start[tid] = released ? before.x : before.y;
      __syncthreads();
      for (int write = released ? 0 : 1; write < 2; ++write) {  // releases are looked over first
        for (uint32_t i = tid; i < n; i += kUpdateThreads) {
          int lo = 0;
#pragma unroll
          for (int d = kUpdateThreads / 2; d; d >>= 1)
            if (start[lo + d] <= i) lo += d;
          int32_t *entry = P.table + static_cast<int64_t>(lo) * P.max_pages + page0[lo] + static_cast<int>(i - start[lo]);
          int32_t *place = P.free_pages + (count + R - 1 - i);
          if (!write) {
            if (*entry < 0 || *entry >= P.num_pages) {
              bad[0] = 53;
              bad[1] = lo;
            }
          } else if (released) {
            *place = *entry;
            *entry = -1;
          } else {
            *entry = *place;
          }
        }
        __syncthreads();
        if (!write && refused()) return;
      }
    }
    if (tid == 0) *P.free_count = static_cast<int32_t>(count + R - G);
    return;
  }
  for (int b0 = 0; b0 < P.batch; b0 += kUpdateThreads) {
    uint32_t grown;
    R += each_page(b0, true, grown, [&](int b, int k, uint32_t) {
      const int page = P.table[static_cast<int64_t>(b) * P.max_pages + k];
      if (page < 0 || page >= P.num_pages) {
        bad[0] = 53;
        bad[1] = b;
      }
    });
    G += grown;
  }
  if (refused()) return;
  // releases, then growth, which may take what was released
  for (int released = 1; released >= 0; --released) {
    if ((released ? R : G) == 0) continue;
    int64_t top = count + R - 1;
    for (int b0 = 0; b0 < P.batch; b0 += kUpdateThreads) {
      uint32_t other;
      top -= each_page(b0, released, other, [&](int b, int k, uint32_t i) {
        int32_t *entry = P.table + static_cast<int64_t>(b) * P.max_pages + k;
        int32_t *place = P.free_pages + (top - i);
        if (released) {
          *place = *entry;
          *entry = -1;
        } else {
          *entry = *place;
        }
      });
    }
  }
  if (tid == 0) *P.free_count = static_cast<int32_t>(count + R - G);
}

constexpr int kSlotThreads = 256;

// Slots of positions first[b] .. seq[b] - 1 of every request, requests in order.
// `per` blocks a request and as many for what lies behind the last; each sums the
// counts of the requests before its own (a few loads a thread, no scan launch).
// Bound by the launch below some 10^5 slots, by the stores above.
__global__ void __launch_bounds__(kSlotThreads)
    pages_slots_kernel(const int32_t *table, int batch, int max_pages, int shift,
                       const int32_t *first, const int32_t *seq, int32_t *slots,
                       int64_t num_slots, int per, int *err) {
  __shared__ int64_t sums[kSlotThreads / 32];
  const int b = static_cast<int>(blockIdx.x) / per, part = static_cast<int>(blockIdx.x) - b * per;
  const int tid = threadIdx.x, lane = tid & 31;
  // of a request: its first position and how many it has (none below 0)
  auto begin = [&](int r) { return first ? max(first[r], 0) : 0; };
  auto count = [&](int r) { return max(max(seq[r], 0) - begin(r), 0); };
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the kernel before may still run
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int64_t start = 0;
  for (int r = tid; r < b; r += kSlotThreads) start += count(r);
#pragma unroll
  for (int o = 16; o; o >>= 1) start += __shfl_xor_sync(0xffffffffu, start, o);
  if (lane == 0) sums[tid >> 5] = start;
  __syncthreads();
  start = 0;
#pragma unroll
  for (int k = 0; k < kSlotThreads / 32; ++k) start += sums[k];
  const int64_t step = static_cast<int64_t>(per) * kSlotThreads;
  if (b == batch) {
    if (start > num_slots && part == 0 && tid == 0) record_error(err, DSA_ERR_DEVICE_BOUNDS, 55, batch);
    for (int64_t t = start + part * kSlotThreads + tid; t < num_slots; t += step) slots[t] = -1;
    return;
  }
  const int p0 = begin(b), n = count(b);
  if (part == 0 && tid == 0 &&
      ((first && first[b] < 0) || seq[b] < 0 || seq[b] > (static_cast<int64_t>(max_pages) << shift)))
    record_error(err, DSA_ERR_DEVICE_BOUNDS, 52, b);
  const int32_t *row = table + static_cast<int64_t>(b) * max_pages;
  for (int64_t i = part * kSlotThreads + tid; i < n && start + i < num_slots; i += step) {
    const int64_t pos = p0 + i, at = pos >> shift;
    const int page = at < max_pages ? row[at] : -1;
    const int64_t slot = (static_cast<int64_t>(page) << shift) + (pos & ((1 << shift) - 1));
    slots[start + i] = page < 0 || slot > INT32_MAX ? -1 : static_cast<int>(slot);
  }
}

struct PagesAppend {
  const uint4 *kv, *k_idx;      // 16-byte units
  const int32_t *slots;
  uint4 *cache, *keys, *means;
  int64_t kv_stride, page_stride, row_stride;  // in 16-byte units
  int32_t n, kv_units, key_units, page_shift, num_pages;
  int *err;
};

constexpr int kAppendWarps = 8;
constexpr int kMaxKeyUnits = 16;  // half a warp

constexpr int kAppendThreads = kAppendWarps * 32;
constexpr int kShortList = 4 * kAppendThreads - 8;  // slots that a block holds, four a thread

// A call's slots by fours, from the first 16-byte boundary on; the up to three ones
// before it and behind the last four stand alone.
struct SlotList {
  const int32_t *slots;
  int n, head, n4, rest;
  __device__ __forceinline__ SlotList(const int32_t *s, int count) : slots(s), n(count) {
    head = min(n, static_cast<int>((0 - (reinterpret_cast<uintptr_t>(s) >> 2)) & 3));
    n4 = (n - head) >> 2;
    rest = head + 4 * n4;
  }
  __device__ __forceinline__ int4 four(int k) const {
    return k < n4 ? reinterpret_cast<const int4 *>(slots + head)[k] : make_int4(-1, -1, -1, -1);
  }
  // the ones that stand alone, x < 6
  __device__ __forceinline__ int single_at(int x) const { return x < head ? x : rest + x - head; }
  __device__ __forceinline__ int single(int x) const { return x < n - rest + head ? slots[single_at(x)] : -1; }
};

// Rows into their slots, a warp a row; the warp that writes a page's last row
// makes the page's mean key.  The keys of the page's rows that this call writes
// come from its input, wherever in its list they stand (another warp may just be
// writing them to the key cache), the others from the key cache; half warp h sums
// rows h, h + 2, .. in fp32, and the halves are added, so a page's key has the same
// bits however its rows arrived.  Where a page's rows stand: a block looks through
// a short list, which its threads hold; in a longer one they are as a rule the P
// rows up to the last, and only where they are not all there the block goes through
// the list.  61 rows 3.5 us (a launch and three dependent loads), 8,000 rows 5.7 us,
// 4.0 TB/s (a launch and its ramp).
template <bool kShort>
__global__ void __launch_bounds__(kAppendThreads) pages_append_kernel(const PagesAppend A) {
  __shared__ int32_t places[kAppendWarps][128];  // of a page's rows in the list, -1: written before
  __shared__ int4 sought[kAppendWarps / 4];      // the page whose rows a warp has to find, or -1
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp;
  const SlotList list(A.slots, A.n);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the kernel before may still run
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int slot = t < A.n ? A.slots[t] : -1;
  int4 held = make_int4(-1, -1, -1, -1);
  int held1 = -1;
  if (kShort && A.k_idx) {
    held = list.four(tid);
    held1 = list.single(tid);
  }
  const int P = 1 << A.page_shift;
  if (slot >> A.page_shift >= A.num_pages) {
    if (lane == 0) record_error(A.err, DSA_ERR_DEVICE_BOUNDS, 56, static_cast<int>(t));
    slot = -1;
  }
  const int page = slot >> A.page_shift, r = slot & (P - 1);
  const uint4 *src = A.kv + t * A.kv_stride;
  const bool has_key = A.k_idx && slot >= 0 && lane < A.key_units;
  uint4 x[3];
  auto load = [&](int u) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (slot >= 0 && u + 32 * k < A.kv_units) x[k] = src[u + 32 * k];
  };
  load(lane);
  uint4 key = make_uint4(0u, 0u, 0u, 0u);
  if (has_key) key = A.k_idx[t * A.key_units + lane];
  uint4 *const page_keys = A.keys + (static_cast<int64_t>(page) << A.page_shift) * A.key_units;
  auto store = [&]() {
    if (slot < 0) return;
    uint4 *dst = A.cache + page * A.page_stride + r * A.row_stride;
    for (int u = lane; u < A.kv_units; u += 96) {
      if (u != lane) load(u);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (u + 32 * k < A.kv_units) dst[u + 32 * k] = x[k];
    }
    if (has_key) page_keys[static_cast<int64_t>(r) * A.key_units + lane] = key;
  };
  if (A.k_idx) {
    int32_t *const place = places[warp];
    const bool ends = slot >= 0 && r == P - 1;
    bool seek = ends;
    if (!kShort && ends) {
      bool here = true;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 32 * k + lane;
        const int64_t tt = t - (P - 1 - row);
        if (row < P) {
          here = here && tt >= 0 && A.slots[tt] == slot - (P - 1 - row);
          place[row] = static_cast<int>(tt);
        }
      }
      seek = !__all_sync(0xffffffffu, here);
    }
    if (!kShort) store();
    if (seek)
      for (int row = lane; row < P; row += 32) place[row] = -1;
    if (lane == 0) reinterpret_cast<int32_t *>(sought)[warp] = seek ? page : -1;
    if (__syncthreads_or(seek)) {
      const int4 s0 = sought[0], s1 = sought[1];
      const int wants[kAppendWarps] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int w = 0; w < kAppendWarps; ++w) {
        const int want = wants[w];
        if (want < 0) continue;
        auto look = [&](int at, int s) {  // a slot below 0 has a page below 0
          if (s >> A.page_shift == want) places[w][s & (P - 1)] = at;
        };
        auto look4 = [&](int k, const int4 &s) {
          const int at = list.head + 4 * k;
          look(at, s.x);
          look(at + 1, s.y);
          look(at + 2, s.z);
          look(at + 3, s.w);
        };
        if (kShort) {
          look4(tid, held);
          look(list.single_at(tid), held1);
        } else {
          look(list.single_at(tid), list.single(tid));
          constexpr int kBatch = 8;
          for (int k0 = tid; k0 < list.n4; k0 += kBatch * kAppendThreads) {
            int4 s[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) s[k] = list.four(k0 + kAppendThreads * k);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) look4(k0 + kAppendThreads * k, s[k]);
          }
        }
      }
      __syncthreads();
    }
    if (ends) {
      const int half = lane >> 4, u = lane & 15;
      float sum[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = 0.f;
      constexpr int kBatch = 8;
#pragma unroll
      for (int r0 = 0; r0 < 128; r0 += 2 * kBatch) {
        if (r0 >= P) break;
        uint4 y[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int row = r0 + 2 * k + half, at = place[row];
          const uint4 *from = at >= 0 ? A.k_idx + static_cast<int64_t>(at) * A.key_units
                                      : page_keys + static_cast<int64_t>(row) * A.key_units;
          y[k] = u < A.key_units ? from[u] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const uint32_t w[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum[2 * e] += __uint_as_float(w[e] << 16);
            sum[2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
          }
        }
      }
      const float inv = 1.f / static_cast<float>(P);  // a power of two
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = (sum[k] + __shfl_xor_sync(0xffffffffu, sum[k], 16)) * inv;
      if (half == 0 && u < A.key_units)
        A.means[static_cast<int64_t>(page) * A.key_units + u] =
            make_uint4(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]), pack_bf16x2(sum[4], sum[5]),
                       pack_bf16x2(sum[6], sum[7]));
    }
  }
  if (kShort || !A.k_idx) store();
}

}  // namespace

int page_shift(int32_t page_size) {
  for (int s = 4; s <= 7; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_pages_update(int32_t *page_table, int32_t batch, int32_t max_pages, const int32_t *held_lens,
                                       const int32_t *seq_lens, int32_t page_size, int32_t *free_pages,
                                       int32_t num_pages, int32_t *free_count, dsa_stream_t stream) {
  const int shift = page_shift(page_size);
  if (batch < 0 || max_pages < 1 || num_pages < 0 || static_cast<int64_t>(batch) * max_pages > INT32_MAX)
    return DSA_ERR_SHAPE;
  if (shift < 0) return DSA_ERR_UNSUPPORTED;
  if (batch == 0) return DSA_OK;
  if (!page_table || !held_lens || !seq_lens || !free_count || (!free_pages && num_pages > 0)) return DSA_ERR_INVALID_ARG;
  int *err = device_error_word();
  if (!err) return DSA_ERR_CUDA;
  const PagesUpdate P{page_table, free_pages, free_count, held_lens, seq_lens, batch, max_pages, num_pages, shift, err};
  const cudaError_t e =
      launch_overlapped(pages_update_kernel, dim3(1), kUpdateThreads, 0, reinterpret_cast<cudaStream_t>(stream), P);
  return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

extern "C" dsa_status dsa_pages_slots(const int32_t *page_table, int32_t batch, int32_t max_pages,
                                      const int32_t *first_pos, const int32_t *seq_lens, int32_t page_size,
                                      int32_t *slots, int32_t num_slots, dsa_stream_t stream) {
  const int shift = page_shift(page_size);
  if (batch < 0 || max_pages < 1 || num_slots < 0 || static_cast<int64_t>(batch) * max_pages > INT32_MAX)
    return DSA_ERR_SHAPE;
  if (shift < 0) return DSA_ERR_UNSUPPORTED;
  if (num_slots == 0) return DSA_OK;
  if (!slots || (batch > 0 && (!page_table || !seq_lens))) return DSA_ERR_INVALID_ARG;
  int *err = device_error_word();
  if (!err) return DSA_ERR_CUDA;
  // about four slots a thread where the requests are alike, and no more blocks than the SMs hold eight times
  const int64_t even = (static_cast<int64_t>(num_slots) + 4 * kSlotThreads - 1) / (4 * kSlotThreads);
  const int64_t room = 8ll * 8 * num_sms() / (static_cast<int64_t>(batch) + 1);
  const int64_t per = even < room ? even : room;
  const int blocks = static_cast<int>(per > 1 ? per : 1);
  if ((static_cast<int64_t>(batch) + 1) * blocks > INT32_MAX) return DSA_ERR_SHAPE;
  const cudaError_t e = launch_overlapped(
      pages_slots_kernel, dim3(static_cast<unsigned>((batch + 1ll) * blocks)), kSlotThreads, 0,
      reinterpret_cast<cudaStream_t>(stream), page_table, static_cast<int>(batch), static_cast<int>(max_pages), shift,
      first_pos, seq_lens, slots, static_cast<int64_t>(num_slots), blocks, err);
  return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

extern "C" dsa_status dsa_pages_append(const void *kv, int64_t kv_stride, const void *k_idx, const int32_t *slots,
                                       int32_t n, int32_t D, int32_t DI, void *cache, int64_t page_stride,
                                       int64_t row_stride, int32_t num_pages, int32_t page_size, void *key_cache,
                                       void *block_keys, dsa_stream_t stream) {
  const int shift = page_shift(page_size);
  if (n < 0 || num_pages < 0 || D < 8 || D % 8 || D > 65536) return DSA_ERR_SHAPE;
  if (kv_stride < D || kv_stride % 8 || row_stride < D || row_stride % 8 || page_stride % 8 || page_stride < 0)
    return DSA_ERR_SHAPE;
  if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX) return DSA_ERR_SHAPE;
  if (shift < 0 || (k_idx && (DI < 8 || DI % 8 || DI > 8 * kMaxKeyUnits))) return DSA_ERR_UNSUPPORTED;
  if (n == 0) return DSA_OK;
  if (!kv || !slots || !cache || (k_idx && (!key_cache || !block_keys))) return DSA_ERR_INVALID_ARG;
  if (!aligned16(kv) || !aligned16(k_idx) || !aligned16(cache) || !aligned16(key_cache) || !aligned16(block_keys))
    return DSA_ERR_INVALID_ARG;
  int *err = device_error_word();
  if (!err) return DSA_ERR_CUDA;
  PagesAppend A{};
  A.kv = static_cast<const uint4 *>(kv);
  A.k_idx = static_cast<const uint4 *>(k_idx);
  A.slots = slots;
  A.cache = static_cast<uint4 *>(cache);
  A.keys = static_cast<uint4 *>(key_cache);
  A.means = static_cast<uint4 *>(block_keys);
  A.kv_stride = kv_stride / 8;
  A.page_stride = page_stride / 8;
  A.row_stride = row_stride / 8;
  A.n = n;
  A.kv_units = D / 8;
  A.key_units = DI / 8;
  A.page_shift = shift;
  A.num_pages = num_pages;
  A.err = err;
  // held lists: the keys are summed before the rows are stored, with 77 registers (61 rows: 3.5 against 5.0 us); where
  // more than a block's threads hold, 52 registers and the rows' stores first (8,000 rows: 5.7 against 7.8 us)
  const auto kernel = n <= kShortList ? pages_append_kernel<true> : pages_append_kernel<false>;
  const cudaError_t e =
      launch_overlapped(kernel, dim3(static_cast<unsigned>((n + int64_t{kAppendWarps - 1}) / kAppendWarps)), kAppendThreads, 0,
                        reinterpret_cast<cudaStream_t>(stream), A);
  return e == cudaSuccess ? check_launch() : cuda_fail(e);
}
