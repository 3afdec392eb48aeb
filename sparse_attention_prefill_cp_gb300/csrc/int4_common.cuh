// The 4-bit latent-KV cache row and its decoding, shared by the cache kernels
// (kv_int4.cu) and the attention that reads it (sparse_attn_int4.cu).
//
// Row of a latent row of D columns, the first Dv of them values:
//   [0, Dv/2)           four-bit integers u = c + 8, c in -7..7: of eight
//                       columns the even ones in nibbles 0-3 and the odd ones
//                       in nibbles 4-7 of a little-endian 32-bit word
//   [rope, ..)          the D - Dv rope columns, bf16 as given
//   [scales, ..)        one E4M3 scale s >= 0 per 16 value columns
//   [exponent]          e + 127 (255: the row holds a NaN or an infinity)
// with every section starting on a 16-byte boundary but the exponent, zero
// bytes between and up to row_bytes (432 at D = 576, Dv = 512).
//
// A value is c * s * 2^e: 3 + 4 significant bits, exact in bf16.  The nibble
// order puts a bf16 pair's two codes 16 bits apart, so that one shift and one
// LOP3 place them in the mantissas of the pair (16 + u, 16 + u'), and one
// packed fma, (16 + u) * s - 24 * s, is the value without any rounding.
#pragma once

#include "dsa_common.cuh"

namespace dsa {

constexpr int kInt4Block = 16;   // value columns per scale
constexpr int kInt4Max = 7;      // largest code
constexpr int kInt4ExpBad = 255; // exponent byte of a row with a NaN or an infinity
// e: the least value is where every nonzero c * s * 2^e is a bf16 (subnormals
// included), the largest where 24 * 448 * 2^e is
constexpr int kInt4ExpMin = -124, kInt4ExpMax = 114;

struct Int4Geom {
  int D, Dv, rope, scales, exponent, row_bytes;
};

__host__ inline dsa_status int4_geom(int32_t D, int32_t Dv, Int4Geom *g) {
  if (D < 1 || Dv < 1 || Dv > D || D > 65536) return DSA_ERR_SHAPE;
  if (Dv % 8 != 0 || (D - Dv) % 8 != 0) return DSA_ERR_SHAPE;
  g->D = D;
  g->Dv = Dv;
  g->rope = (Dv / 2 + 15) / 16 * 16;
  g->scales = g->rope + (2 * (D - Dv) + 15) / 16 * 16;
  g->exponent = g->scales + (Dv + kInt4Block - 1) / kInt4Block;
  g->row_bytes = (g->exponent + 1 + 15) / 16 * 16;
  return DSA_OK;
}

__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// The two bf16 factors, f1 in the low half and f2 in the high one, whose
// product is 2^(120 + e): an E4M3 byte moved into a bf16's exponent and
// mantissa is 2^-120 of its value, and 2^(120 + e) itself need not be a bf16.
// A bad row's second factor is NaN.
__device__ __forceinline__ uint32_t int4_row_factors(uint32_t exponent_byte) {
  const int h = (static_cast<int>(exponent_byte) - 7) >> 1;            // (120 + e) / 2
  const int r = static_cast<int>(exponent_byte) - 7 - h;
  const uint32_t f1 = static_cast<uint32_t>(h + 127) << 7, f2 = static_cast<uint32_t>(r + 127) << 7;
  return f1 | ((exponent_byte == kInt4ExpBad ? 0x7fc0u : f2) << 16);
}

// A block's scale s * 2^e as a bf16 pair (s, s): `two` holds the E4M3 byte in
// bits 0-7 and 16-23; f1, f2 are pairs of the row's factors.  Every step is exact.
__device__ __forceinline__ uint32_t int4_scale(uint32_t two, uint32_t f1, uint32_t f2) {
  return bf2_mul(bf2_mul(two << 4, f1), f2);
}

// Eight codes (one word) -> eight values, columns in order.  s: int4_scale;
// s24 = -24 * s (exact: two bits more than s).
__device__ __forceinline__ void int4_decode8(uint32_t w, uint32_t s, uint32_t s24, uint32_t (&o)[4]) {
  const uint32_t mask = 0x00780078u, base = 0x41804180u;  // mantissa bits 3-6; 16.0
  o[0] = bf2_fma(((w << 3) & mask) | base, s, s24);
  o[1] = bf2_fma(((w >> 1) & mask) | base, s, s24);
  o[2] = bf2_fma(((w >> 5) & mask) | base, s, s24);
  o[3] = bf2_fma(((w >> 9) & mask) | base, s, s24);
}
__device__ __forceinline__ uint32_t int4_scale24(uint32_t s) { return bf2_mul(s, 0xc1c0c1c0u); }  // -24.0

}  // namespace dsa
