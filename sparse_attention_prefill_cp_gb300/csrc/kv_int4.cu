// The 4-bit latent-KV cache: rows quantised as they are written into its
// slots, and read back by number (row format: int4_common.cuh).
//
// Quantisation of a row, x its Dv values:
//   A = max |x|;  e = the least integer with A <= 7 * 448 * 2^e
//   s_b = E4M3(max|x_b| / 7 / 2^e)              per block b of 16 columns
//   c   = clamp(rint(x / (s_b * 2^e)), -7, 7)   (s_b = 0: c = 0)
// so the row's power of two gives the range (any bf16 magnitude up to 2^125)
// and the block's E4M3 the precision.  Symmetric integers, not E2M1: at 16
// columns a block their uniform step, max|x_b| / 7, has a third less squared
// error than E2M1's on normal values, and they decode with one fma a pair.
//
// Decisions are those of the exact quotients, although a quotient is taken as
// x * (1 / s): for x = X 2^i (X of 8 bits) and s = S 2^j (S of 4) an exact
// quotient that is not a half integer is at least 2^-8 of itself away from
// one, the computed one is within 2^-22, and rounding it to 16 significant
// bits first brings a half integer back exactly, to be rounded to even.
//
// One warp per row, a lane on 8 columns at a time (16-byte loads, 4-byte code
// stores, both whole lines per warp).  HBM-bound.
#include "int4_common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kRowsPerBlock = 8;
constexpr int kRegGroups = 2;  // 256-column groups of a row kept in registers (Dv <= 512); more are read twice

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// max |x| of eight bf16 values as their 16-bit magnitudes (ordered like the values, NaN above infinity)
__device__ __forceinline__ uint32_t max_mag8(uint4 v) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(a & 0xffffu, a >> 16);
}

// rint(x * inv) + 8 in the low bits, x * inv first to 16 significant bits
__device__ __forceinline__ uint32_t code_of(float xs, float inv) {
  const float y = __uint_as_float((__float_as_uint(xs * inv) + 0x80u) & 0xffffff00u);
  return __float_as_uint(fminf(fmaxf(y, -7.f), 7.f) + 12582920.f) & 15u;  // 1.5 * 2^23 + 8
}

// Codes and scale of the lane's 8 columns; the block's other 8 are the neighbour lane's.
__device__ __forceinline__ void quantise8(uint4 v, uint32_t mag, float down, uint32_t &word, uint32_t &scale) {
  const uint32_t other = __shfl_xor_sync(0xffffffffu, mag, 1);
  const float amax = __uint_as_float(max(mag, other) << 16) * down;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %1;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(scale)
      : "f"(__fdiv_rn(amax, 7.f)));
  scale &= 0xffu;
  float s, unused;
  unpack_f16x2(e4m3x2_to_f16x2(scale), s, unused);
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;  // 0: every code is 8
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  word = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    word |= (code_of(bf16_lo(x[j]) * down, inv) | (code_of(bf16_hi(x[j]) * down, inv) << 16)) << (4 * j);
}

__global__ void __launch_bounds__(kRowsPerBlock * 32)
    kv_int4_quantize_kernel(const __nv_bfloat16 *__restrict__ kv, int64_t row_stride, int64_t num_rows,
                            const int32_t *__restrict__ slots, uint8_t *__restrict__ cache, int64_t cache_rows,
                            Int4Geom g, int *err) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5);
  if (row >= num_rows) return;
  const __nv_bfloat16 *src = kv + row * row_stride;
  const int groups = (g.Dv / 8 + 31) / 32, units = g.Dv / 8;
  const int64_t slot = slots ? slots[row] : row;
  auto load = [&](int i) {
    const int u = lane + 32 * i;
    return u < units ? __ldg(reinterpret_cast<const uint4 *>(src + 8 * u)) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 v[kRegGroups];
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < kRegGroups; ++i) {
    v[i] = load(i);
    mag = max(mag, max_mag8(v[i]));
  }
  for (int i = kRegGroups; i < groups; ++i) mag = max(mag, max_mag8(load(i)));
  mag = __reduce_max_sync(0xffffffffu, mag);
  if (slot < 0 || slot >= cache_rows) {  // a negative slot: the row is not written
    if (slot >= 0 && lane == 0) record_error(err, DSA_ERR_DEVICE_BOUNDS, 47, static_cast<int>(row));
    return;
  }
  const bool bad = mag >= 0x7f80u;
  // least e with A <= 3136 * 2^e, 3136 = 1.53125 * 2^11, from A = 1.f * 2^(x - 127)
  int e = static_cast<int>(mag >> 7) - 138 + ((mag & 0x7fu) > 0x44u ? 1 : 0);
  e = min(max(e, kInt4ExpMin), kInt4ExpMax);
  const float down = bad ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
  uint8_t *dst = cache + slot * g.row_bytes;
  auto store = [&](int i, uint4 x) {
    const int u = lane + 32 * i;
    if (bad) x = make_uint4(0u, 0u, 0u, 0u);
    uint32_t word, scale;
    quantise8(x, max_mag8(x), down, word, scale);
    if (u < units) {
      *reinterpret_cast<uint32_t *>(dst + 4 * u) = word;
      if ((u & 1) == 0) dst[g.scales + u / 2] = static_cast<uint8_t>(scale);
    }
  };
#pragma unroll
  for (int i = 0; i < kRegGroups; ++i)
    if (i < groups) store(i, v[i]);
  for (int i = kRegGroups; i < groups; ++i) store(i, load(i));
  // rope columns as they are, the exponent, and the zero bytes between and behind the sections
  const int rope_units = (g.D - g.Dv) / 8;
  for (int u = lane; u < rope_units; u += 32)
    *reinterpret_cast<uint4 *>(dst + g.rope + 16 * u) = __ldg(reinterpret_cast<const uint4 *>(src + g.Dv + 8 * u));
  for (int b = g.Dv / 2 + lane; b < g.rope; b += 32) dst[b] = 0;
  if (lane == 0) dst[g.exponent] = static_cast<uint8_t>(bad ? kInt4ExpBad : e + 127);
  for (int b = g.exponent + 1 + lane; b < g.row_bytes; b += 32) dst[b] = 0;
}

__global__ void __launch_bounds__(kRowsPerBlock * 32)
    kv_int4_dequantize_kernel(const uint8_t *__restrict__ cache, int64_t cache_rows, const int32_t *__restrict__ rows,
                              int64_t num_rows, __nv_bfloat16 *__restrict__ kv, Int4Geom g, int *err) {
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5);
  if (i >= num_rows) return;
  const int64_t row = rows ? rows[i] : i;
  __nv_bfloat16 *dst = kv + i * g.D;
  if (row < 0 || row >= cache_rows) {  // a negative number: a row of zeros
    if (row >= 0 && lane == 0) record_error(err, DSA_ERR_DEVICE_BOUNDS, 48, static_cast<int>(i));
    for (int u = lane; u < g.D / 8; u += 32) *reinterpret_cast<uint4 *>(dst + 8 * u) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const uint8_t *src = cache + row * g.row_bytes;
  const uint32_t f = int4_row_factors(src[g.exponent]);
  const uint32_t f1 = __byte_perm(f, 0, 0x1010), f2 = __byte_perm(f, 0, 0x3232);
  const int units = g.Dv / 8;
#pragma unroll 2
  for (int u = lane; u < units; u += 32) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(src + 4 * u);
    const uint32_t s = int4_scale(src[g.scales + u / 2] * 0x10001u, f1, f2);
    uint32_t o[4];
    int4_decode8(w, s, int4_scale24(s), o);
    *reinterpret_cast<uint4 *>(dst + 8 * u) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  for (int u = lane; u < (g.D - g.Dv) / 8; u += 32)
    *reinterpret_cast<uint4 *>(dst + g.Dv + 8 * u) = *reinterpret_cast<const uint4 *>(src + g.rope + 16 * u);
}

unsigned blocks_of(int64_t rows) { return static_cast<unsigned>((rows + kRowsPerBlock - 1) / kRowsPerBlock); }

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
  kv_int4_quantize_kernel<<<blocks_of(num_rows), kRowsPerBlock * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
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
  kv_int4_dequantize_kernel<<<blocks_of(num_rows), kRowsPerBlock * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t *>(cache), num_cache_rows, rows, num_rows, static_cast<__nv_bfloat16 *>(kv), g, err);
  return check_launch();
}
