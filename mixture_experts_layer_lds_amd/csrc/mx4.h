// MXFP4 (OCP Microscaling, e2m1 elements) device helpers.
//
// 32 consecutive values of a row share one e8m0 scale 2^s (code s + 127);
// an element code holds sign and magnitude 0, 1/2, 1, 3/2, 2, 3, 4 or 6,
// two codes a byte, the lower column in the low nibble.
//
// The product runs on v_mfma_scale_f32_16x16x128_f8f6f4 in its 4-bit mode:
// lane l supplies row / column l % 16, K values 32 (l / 16) .. + 31 (16
// bytes) and that block's scale, one byte of a register chosen by the
// instruction.  A *unit* is the 128 K values of one instruction.  Units come
// in groups of G = 4, 2 or 1, the largest that divides K / 128, so that a
// lane's G scale codes of a group are one 4-, 2- or 1-byte piece:
//
//   block of a group: 16 rows x G units, 1088 G bytes
//     bytes 0 .. 1024 G         unit-major 1 KiB chunks, lane l's 16 bytes at 16 l
//     bytes 1024 G .. 1088 G    lane l's G scale codes (one a unit) at G l
//
// Packed weights and the layer's intermediate rows are stored as such
// blocks: one contiguous stream, codes and scales together.
#pragma once

#include <type_traits>

#include "moe_common.h"

namespace moe {

constexpr int kMx4Unit = 1088;   // bytes of 16 rows x 128 values with their scale codes

// Units per group of a reduction over K values (K % 128 == 0).
__host__ __device__ inline int mx4_group(int K) {
  const int units = K / 128;
  return units % 4 == 0 ? 4 : (units % 2 == 0 ? 2 : 1);
}

// Scale code of a block from the largest magnitude's bits (sign cleared; as
// integers Inf and NaN are the largest): 255 (NaN) if the block holds Inf or
// NaN, else the biased exponent - 2 (2 = the largest e2m1 exponent), at
// least 0.  Zero and subnormal maxima take 0.
__device__ __forceinline__ uint32_t mx4_scale_code(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}

// The float 2^(code - 127) that the conversion instruction divides by (code
// 0: 2^-127, a subnormal).
__device__ __forceinline__ float mx4_scale_value(uint32_t code) {
  return __uint_as_float(code ? code << 23 : 0x00400000u);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Codes of eight values, v[0] in the lowest nibble.  The instruction rounds
// v / scale to nearest even and saturates at 6 (checked against the formula
// over every border of the format and random values).  A block of scale code
// 255 holds zeros: its values are NaN by the scale alone.
__device__ __forceinline__ uint32_t mx4_encode8(const float (&v)[8], uint32_t code) {
  const float sc = mx4_scale_value(code);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], sc, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], sc, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], sc, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], sc, 3);
  return code == 255u ? 0u : r;
}

// Codes of four values in the low 16 bits.
__device__ __forceinline__ uint32_t mx4_encode4(const f32x4& v, uint32_t code) {
  const float sc = mx4_scale_value(code);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], sc, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], sc, 1);
  return code == 255u ? 0u : r;
}

// Two fp32 -> two bf16 in one dword, to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// acc += W * T^T over one unit: w the weights' fragment (rows of the result),
// t the tokens' (columns), SEL the byte of each scale register.
template <int SEL>
__device__ __forceinline__ void mfma_mx4(f32x4& acc, const u32x4& w, const u32x4& t, uint32_t sw, uint32_t st) {
  const i32x8 a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8 b = {(int)t[0], (int)t[1], (int)t[2], (int)t[3], 0, 0, 0, 0};
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, SEL, (int)sw, SEL, (int)st);
}

// The units of a group in turn (the byte selector is part of the instruction).
template <int G, typename F>
__device__ __forceinline__ void mx4_units(F&& f) {
  f(std::integral_constant<int, 0>{});
  if constexpr (G >= 2) f(std::integral_constant<int, 1>{});
  if constexpr (G >= 4) {
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 3>{});
  }
}

}  // namespace moe
