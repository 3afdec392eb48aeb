// The 4-bit latent-KV cache: rows quantised as they are written into its
// slots, and read back by number (row format: int4_common.cuh).
//
// Quantisation of a row, x its Dv values:
//   A = max |x|;  e = the least integer with A <= 7 * 448 * 2^e
//   s_b = E4M3(max|x_b| / 7 / 2^e)              per block b of 16 columns
//   c   = clamp(rint(x / (s_b * 2^e)), -7, 7)   (s_b = 0: c = 0)
// so the row's power of two gives the range (any bf16 magnitude up to 2^125)
// and the block's E4M3 the precision.  Symmetric integers, not E2M1: at 16
// columns a block their uniform step, max|x_b| / 7, has 18 % less squared error
// than E2M1 scaled to max|x_b| / 6 on normal values, and they decode with one fma a pair.
//
// Decisions are those of the exact quotients, although quotients are products
// with an approximate reciprocal: for x = X 2^i (X of 8 bits) and s = S 2^j (S
// of 4) an exact quotient that is not a half integer is at least 2^-8 of itself
// away from one, the computed one is within 2^-21 of itself; the sum
// 768 + x * (1/s), one fma, rounds it to a multiple of 2^-14, which brings a
// half integer back exactly, and the next sum rounds that to an even integer.  In
// the same way max|x_b| * (1/7) is brought to 16 significant bits before it
// becomes E4M3.  The clamp to -7..7 bites only where s is subnormal or the row's
// e was clamped (E4M3 is within 2^-4 of the quotient elsewhere: at most 7.44
// steps), and is one of x there, to -7 s 2^e..7 s 2^e, a bf16.
//
// Quantising, a warp takes a row and a lane the 16 columns of a block (two or
// four rows a warp: 2.7 and 4.4 us instead of 2.2 for 64 rows, nothing gained
// on many); reading back, a lane holds 8 columns at a time and a warp four rows,
// the loads of all of them in flight (one row a warp: 38 against 28 us for
// 100,003 rows).  HBM-bound: 2^20 rows of 576 (1.66 GB) are quantised in 310 us
// (5.4 TB/s; 364 us into scattered slots) and read back in 240 us (6.9 TB/s;
// 274 us from scattered rows).
#include "int4_common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kWarps = 8;        // per block
constexpr int kReadRows = 4;     // rows a warp reads back
constexpr int kUnits = 2;        // 8-column units a lane reads back at a time

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct Block {
  uint32_t x[8];  // 16 columns
};

// max |x| of a block as its 16-bit magnitude (ordered like the values, NaN above infinity)
__device__ __forceinline__ uint32_t max_mag(const Block &v) {
  const uint32_t m = 0x7fff7fffu;
  uint32_t a = v.x[0] & m;
#pragma unroll
  for (int k = 1; k < 8; ++k) a = __vmaxu2(a, v.x[k] & m);
  return max(a & 0xffffu, a >> 16);
}

// Codes and scale of a block; 2^e is the row's power of two (e >= -100 here).
__device__ __forceinline__ void quantise(const Block &v, int e, uint2 &codes, uint32_t &scale) {
  const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const float want = __uint_as_float(max_mag(v) << 16) * down * (1.f / 7.f);
  const float snapped = __uint_as_float((__float_as_uint(want) + 0x80u) & 0xffffff00u);
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %1;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(scale)
      : "f"(snapped));
  scale &= 0xffu;
  float s, unused;
  unpack_f16x2(e4m3x2_to_f16x2(scale), s, unused);
  Block c = v;
  if (scale < 8u || e == kInt4ExpMax) {
    const float top = 7.f * s * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    const uint32_t hi = pack_bf16x2(top, top), lo = hi ^ 0x80008000u;
#pragma unroll
    for (int k = 0; k < 8; ++k) c.x[k] = min2(max2(c.x[k], lo), hi);
  }
  const float inv = s > 0.f ? rcp_approx(s) * down : 0.f;  // 0: every code is 8
  const uint64_t inv2 = f2_pack(inv, inv), c768 = f2_pack(768.f, 768.f);
  const uint64_t to_int = f2_pack(12582152.f, 12582152.f);  // 1.5 * 2^23 + 8 - 768
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = c.x[4 * h + j];
      float a, b;
      f2_unpack(f2_add(f2_fma(f2_pack(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), inv2, c768), to_int),
                a, b);
      w[h] |= (__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410) & 0x000f000fu) << (4 * j);
    }
  }
  codes = make_uint2(w[0], w[1]);
}

__global__ void __launch_bounds__(kWarps * 32)
    kv_int4_quantize_kernel(const __nv_bfloat16 *__restrict__ kv, int64_t row_stride, int64_t num_rows,
                            const int32_t *__restrict__ slots, uint8_t *__restrict__ cache, int64_t cache_rows,
                            Int4Geom g, int *err) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= num_rows) return;
  const __nv_bfloat16 *src = kv + row * row_stride;
  const int passes = (g.Dv + 32 * kInt4Block - 1) / (32 * kInt4Block);  // a lane's block per pass
  auto load = [&](int pass) {
    const int c = (lane + 32 * pass) * kInt4Block;
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (c < g.Dv) lo = __ldg(reinterpret_cast<const uint4 *>(src + c));
    if (c + 8 < g.Dv) hi = __ldg(reinterpret_cast<const uint4 *>(src + c + 8));
    return Block{{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
  };
  const int64_t slot = slots ? slots[row] : row;
  const Block first = load(0);
  const int rope_units = (g.D - g.Dv) / 8;
  uint4 rope = make_uint4(0u, 0u, 0u, 0u);
  if (lane < rope_units) rope = __ldg(reinterpret_cast<const uint4 *>(src + g.Dv + 8 * lane));
  uint32_t mag = max_mag(first);
  for (int p = 1; p < passes; ++p) mag = max(mag, max_mag(load(p)));
  mag = __reduce_max_sync(0xffffffffu, mag);
  if (slot < 0 || slot >= cache_rows) {  // a negative slot: the row is not written
    if (slot >= 0 && lane == 0) record_error(err, DSA_ERR_DEVICE_BOUNDS, 47, static_cast<int>(row));
    return;
  }
  const bool bad = mag >= 0x7f80u;
  // least e with A <= 3136 * 2^e, 3136 = 1.53125 * 2^11, from A = 1.f * 2^(x - 127)
  int e = static_cast<int>(mag >> 7) - 138 + ((mag & 0x7fu) > 0x44u ? 1 : 0);
  e = min(max(e, kInt4ExpMin), kInt4ExpMax);
  uint8_t *dst = cache + slot * g.row_bytes;
  auto store = [&](int pass, Block x) {
    const int b = lane + 32 * pass;
    uint2 codes;
    uint32_t scale;
    if (bad) {  // stands for NaN throughout
      codes = make_uint2(0x88888888u, 0x88888888u);
      scale = 0;
    } else if (e < -100) {  // 2^-e / s could overflow: the row times 2^64, exact
#pragma unroll
      for (int k = 0; k < 8; ++k) x.x[k] = bf2_mul(x.x[k], 0x5f805f80u);
      quantise(x, e + 64, codes, scale);
    } else {
      quantise(x, e, codes, scale);
    }
    if (b * kInt4Block + 8 < g.Dv) *reinterpret_cast<uint2 *>(dst + 8 * b) = codes;
    else if (b * kInt4Block < g.Dv) *reinterpret_cast<uint32_t *>(dst + 8 * b) = codes.x;
    if (b * kInt4Block < g.Dv) dst[g.scales + b] = static_cast<uint8_t>(scale);
  };
  store(0, first);
  for (int p = 1; p < passes; ++p) store(p, load(p));
  // rope columns as they are, the exponent, and the zero bytes between and behind the sections
  if (lane < rope_units) *reinterpret_cast<uint4 *>(dst + g.rope + 16 * lane) = rope;
  for (int u = 32 + lane; u < rope_units; u += 32)
    *reinterpret_cast<uint4 *>(dst + g.rope + 16 * u) = __ldg(reinterpret_cast<const uint4 *>(src + g.Dv + 8 * u));
  for (int b = g.Dv / 2 + lane; b < g.rope; b += 32) dst[b] = 0;
  if (lane == 0) dst[g.exponent] = static_cast<uint8_t>(bad ? kInt4ExpBad : e + 127);
  for (int b = g.exponent + 1 + lane; b < g.row_bytes; b += 32) dst[b] = 0;
}

__global__ void __launch_bounds__(kWarps * 32)
    kv_int4_dequantize_kernel(const uint8_t *__restrict__ cache, int64_t cache_rows, const int32_t *__restrict__ rows,
                              int64_t num_rows, __nv_bfloat16 *__restrict__ kv, Int4Geom g, int *err) {
  const int lane = threadIdx.x & 31;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kReadRows;
  const int units = g.Dv / 8, rope_units = (g.D - g.Dv) / 8;
  // lanes 0..3 know a row each; a negative number or one out of range is a row of zeros
  int row_l = -1;
  if (lane < kReadRows && i0 + lane < num_rows) {
    const int64_t row = rows ? rows[i0 + lane] : i0 + lane;
    if (row >= cache_rows) record_error(err, DSA_ERR_DEVICE_BOUNDS, 48, static_cast<int>(i0 + lane));
    else row_l = static_cast<int>(row);
  }
  uint32_t factors_l = 0;
  if (row_l >= 0) factors_l = cache[static_cast<int64_t>(row_l) * g.row_bytes + g.exponent];
  int row[kReadRows];
#pragma unroll
  for (int r = 0; r < kReadRows; ++r) row[r] = __shfl_sync(0xffffffffu, row_l, r);
  // the rope columns of the rows together: eight bf16 a lane
  for (int k = lane; k < kReadRows * rope_units; k += 32) {
    const int r = k / rope_units, u = k - r * rope_units;
    if (i0 + r >= num_rows) break;
    int rw = row[0];
#pragma unroll
    for (int q = 1; q < kReadRows; ++q) rw = r == q ? row[q] : rw;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (rw >= 0) x = *reinterpret_cast<const uint4 *>(cache + static_cast<int64_t>(rw) * g.row_bytes + g.rope + 16 * u);
    *reinterpret_cast<uint4 *>(kv + (i0 + r) * g.D + g.Dv + 8 * u) = x;
  }
  factors_l = row_l >= 0 ? int4_row_factors(factors_l) : 0u;
  for (int u0 = 0; u0 < units; u0 += 32 * kUnits) {
    uint32_t w[kReadRows][kUnits], s[kReadRows][kUnits];
#pragma unroll
    for (int r = 0; r < kReadRows; ++r)
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int u = u0 + lane + 32 * i;
        const uint8_t *src = cache + static_cast<int64_t>(row[r]) * g.row_bytes;
        w[r][i] = s[r][i] = 0;
        if (row[r] >= 0 && u < units) {
          w[r][i] = *reinterpret_cast<const uint32_t *>(src + 4 * u);
          s[r][i] = src[g.scales + u / 2];
        }
      }
#pragma unroll
    for (int r = 0; r < kReadRows; ++r) {
      const uint32_t f = __shfl_sync(0xffffffffu, factors_l, r);
      const uint32_t f1 = __byte_perm(f, 0, 0x1010), f2 = __byte_perm(f, 0, 0x3232);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int u = u0 + lane + 32 * i;
        const uint32_t sc = int4_scale(s[r][i] * 0x10001u, f1, f2);
        uint32_t o[4];
        int4_decode8(w[r][i], sc, int4_scale24(sc), o);
        if (i0 + r < num_rows && u < units)
          *reinterpret_cast<uint4 *>(kv + (i0 + r) * g.D + 8 * u) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

unsigned blocks_of(int64_t rows, int per_warp) {
  return static_cast<unsigned>((rows + kWarps * per_warp - 1) / (kWarps * per_warp));
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_kv_int4_row_bytes(int32_t D, int32_t Dv, size_t *bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  Int4Geom g;
  dsa_status st = int4_geom(D, Dv, &g);
  if (st != DSA_OK) return st;
  *bytes = static_cast<size_t>(g.row_bytes);
  return DSA_OK;
}

extern "C" dsa_status dsa_kv_int4_quantize(const void *kv, int64_t row_stride, int32_t num_rows, int32_t D, int32_t Dv,
                                           const int32_t *slots, void *cache, int32_t num_cache_rows,
                                           dsa_stream_t stream) {
  Int4Geom g;
  dsa_status st = int4_geom(D, Dv, &g);
  if (st != DSA_OK) return st;
  if (num_rows < 0 || num_cache_rows < 0 || row_stride < D || row_stride % 8 != 0) return DSA_ERR_SHAPE;
  if (!slots && num_rows > num_cache_rows) return DSA_ERR_SHAPE;
  if (num_rows == 0) return DSA_OK;
  if (!kv || !cache || !aligned16(kv) || !aligned16(cache)) return DSA_ERR_INVALID_ARG;
  int *err = device_error_word();
  if (!err) return DSA_ERR_CUDA;
  kv_int4_quantize_kernel<<<blocks_of(num_rows, 1), kWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const __nv_bfloat16 *>(kv), row_stride, num_rows, slots, static_cast<uint8_t *>(cache),
      num_cache_rows, g, err);
  return check_launch();
}

extern "C" dsa_status dsa_kv_int4_dequantize(const void *cache, int32_t num_cache_rows, int32_t D, int32_t Dv,
                                             const int32_t *rows, int32_t num_rows, void *kv, dsa_stream_t stream) {
  Int4Geom g;
  dsa_status st = int4_geom(D, Dv, &g);
  if (st != DSA_OK) return st;
  if (num_rows < 0 || num_cache_rows < 0) return DSA_ERR_SHAPE;
  if (!rows && num_rows > num_cache_rows) return DSA_ERR_SHAPE;
  if (num_rows == 0) return DSA_OK;
  if (!kv || !cache || !aligned16(kv) || !aligned16(cache)) return DSA_ERR_INVALID_ARG;
  int *err = device_error_word();
  if (!err) return DSA_ERR_CUDA;
  kv_int4_dequantize_kernel<<<blocks_of(num_rows, kReadRows), kWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t *>(cache), num_cache_rows, rows, num_rows, static_cast<__nv_bfloat16 *>(kv), g, err);
  return check_launch();
}
