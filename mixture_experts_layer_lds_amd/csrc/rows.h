// Rows of bf16, fp16 or fp32 values: eight at a time to and from fp32.
#pragma once

#include "moe_common.h"

namespace moe {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct RowBf16 {
  typedef uint16_t elem;
  static __device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const u32x4 q = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = bf16_bits_to_f32(q[i] & 0xffffu);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; i++)
      q[i] = (uint32_t)f32_to_bf16_bits(v[2 * i]) | ((uint32_t)f32_to_bf16_bits(v[2 * i + 1]) << 16);
    *reinterpret_cast<u32x4*>(p) = q;
  }
};

struct RowFp16 {
  typedef _Float16 elem;
  static __device__ __forceinline__ void load8(const _Float16* p, float (&v)[8]) {
    const f16x8 q = *reinterpret_cast<const f16x8*>(p);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = (float)q[i];
  }
  static __device__ __forceinline__ void store8(_Float16* p, const float (&v)[8]) {
    f16x8 q;
#pragma unroll
    for (int i = 0; i < 8; i++) q[i] = (_Float16)v[i];   // to nearest even
    *reinterpret_cast<f16x8*>(p) = q;
  }
};

struct RowFp32 {
  typedef float elem;
  static __device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
  static __device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
};

// f(RowBf16{} / RowFp16{} / RowFp32{}) by moe_row_type_t.
template <typename F>
static hipError_t with_row_type(int row_type, F&& f) {
  switch (row_type) {
    case MOE_ROW_BF16: return f(RowBf16{});
    case MOE_ROW_FP16: return f(RowFp16{});
    case MOE_ROW_FP32: return f(RowFp32{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe
