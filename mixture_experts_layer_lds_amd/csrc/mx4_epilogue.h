// Gate-up epilogue of the MXFP4 GEMMs: SiLU(gate) * up of one token row as
// MXFP4 codes in the blocks that the down GEMM reads (mx4.h).
#pragma once

#include "mx4.h"

namespace moe {

// g / (1 + e^-g) to a few steps of fp32 for every g whose e^-g fp32 holds (g >
// -88.7; below, -0).  e^-g = 2^t (1 + r ln 2) with t = -g log2(e) rounded and r
// the rest of the product, without which it is off by up to 1.2 |g| 2^-24 of
// itself.  A quarter of both sides of the division keeps the
// hardware's reciprocal, which returns no subnormals, in range up to e^-g =
// 2^128.  The clamp keeps r finite; past it e^-g is 0 or infinite already.  The
// hardware's 2^x and reciprocal are within a step of fp32 each and take sixteen
// cycles a wave, the nine others four; the library exponential and a division
// take several times that, of an epilogue that the whole CU waits for.
__device__ __forceinline__ float mx4_silu(float g) {
  constexpr float kLog2e = 1.44269504088896340736f, kLog2eLo = 1.92596299112661746887e-8f, kLn2 = 0.69314718055994530942f;
  const float c = __builtin_amdgcn_fmed3f(g, -128.0f, 128.0f);
  const float t = -kLog2e * c;
  const float r = __builtin_fmaf(-kLog2eLo, c, __builtin_fmaf(-kLog2e, c, -t));
  const float e = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(r, kLn2, 1.0f);
  return 0.25f * g * __builtin_amdgcn_rcpf(__builtin_fmaf(0.25f, e, 0.25f));
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
