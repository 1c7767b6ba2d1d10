// Gate-up epilogue of the MXFP4 GEMMs: SiLU(gate) * up of one token row as
// MXFP4 codes in the blocks that the down GEMM reads (mx4.h).
#pragma once

#include "mx4.h"

namespace moe {

// g / (1 + e^-g).  e^-g = 2^(t + r) with t = -g log2(e) rounded and r the rest
// of the product: 2^t (1 + r ln 2) from the hardware's 2^x, and its reciprocal
// (each within a step of fp32).  About a quarter of the instructions of the
// library exponential and the division, which took 6 us a tile of 192 rows.
__device__ __forceinline__ float mx4_silu(float g) {
  constexpr float kLog2e = 1.44269504088896340736f, kLog2eLo = 1.92596299112661746887e-8f, kLn2 = 0.69314718055994530942f;
  const float t = -g * kLog2e;
  const float r = __builtin_fmaf(-g, kLog2e, -t) - g * kLog2eLo;
  const float p = __builtin_fminf(__builtin_amdgcn_exp2f(t), 3.4028234664e38f);   // no inf times r
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(p * kLn2, r, p));
}

// Where the 32 columns `c32` of 16-row block `slot` go, for rows of `units`
// units in groups of G.
struct Mx4Out {
  char* codes;     // 16 bytes a row
  char* scale;     // one byte a row, G apart
  int G;
};

__device__ __forceinline__ Mx4Out mx4_out(void* c, size_t slot, int c32, int units, int G) {
  const int unit = c32 >> 2, kb = c32 & 3, u = unit & (G - 1);   // G is 1, 2 or 4
  char* base = static_cast<char*>(c) + (slot * units + (unit - u)) * kMx4Unit;
  return Mx4Out{base + u * 1024 + 256 * kb, base + G * 1024 + 16 * kb * G + u, G};
}

}  // namespace moe
