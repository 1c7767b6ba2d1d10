// Gate-up epilogue of the MXFP4 GEMMs: SiLU(gate) * up of one token row as
// MXFP4 codes in the blocks that the down GEMM reads (mx4.h).
#pragma once

#include "mx4.h"

namespace moe {

// g / (1 + e^-g) by the hardware's 2^x and reciprocal (each within a step of
// fp32).  Rounding g log2(e) leaves e^-g off by |g| 2^-23 of itself, a share of
// the sum's own rounding error; an infinite e^-g gives a zero.  Two
// transcendental instructions of sixteen cycles a wave and three others of
// four: the library exponential and a division take several times that, and
// keeping the rest of the product in a second term twice that, of an epilogue
// that the whole CU waits for.
__device__ __forceinline__ float mx4_silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * g));
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
