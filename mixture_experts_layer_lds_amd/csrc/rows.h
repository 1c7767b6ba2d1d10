// Rows of bf16, fp16 or fp32 values, 16 bytes at a time to and from fp32.
#pragma once

#include "mx4.h"

namespace moe {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// kVec values are 16 bytes; unpack and pack go between those and fp32 (to
// nearest even).
struct RowBf16 {
  typedef uint16_t elem;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void unpack(const u32x4& q, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&v)[8]) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; i++) q[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    return q;
  }
};

struct RowFp16 {
  typedef _Float16 elem;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void unpack(const u32x4& q, float (&v)[8]) {
    const f16x8 h = __builtin_bit_cast(f16x8, q);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = (float)h[i];
  }
  static __device__ __forceinline__ u32x4 pack(const float (&v)[8]) {
    f16x8 h;
#pragma unroll
    for (int i = 0; i < 8; i++) h[i] = (_Float16)v[i];
    return __builtin_bit_cast(u32x4, h);
  }
};

struct RowFp32 {
  typedef float elem;
  static constexpr int kVec = 4;
  static __device__ __forceinline__ void unpack(const u32x4& q, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = __uint_as_float(q[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float (&v)[4]) {
    return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  }
};

// 16 bytes of a row as fp32, and back.
template <typename R>
__device__ __forceinline__ void row_load(const typename R::elem* p, float (&v)[R::kVec]) {
  R::unpack(*reinterpret_cast<const u32x4*>(p), v);
}
template <typename R>
__device__ __forceinline__ void row_store(typename R::elem* p, const float (&v)[R::kVec]) {
  *reinterpret_cast<u32x4*>(p) = R::pack(v);
}

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
