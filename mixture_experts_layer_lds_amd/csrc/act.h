// Activations of the linear layers and their derivatives, in fp32.
#pragma once

#include "rows.h"

namespace moe {

// sigma(z) and 1 - sigma(z) by t = e^-|z|, which does not overflow: the smaller
// of the two is t / (1 + t) and keeps its relative precision (a few 2^-24 times
// 1 + |z|, from the rounded argument of 2^x) as far as fp32 holds e^-|z|.  The
// results are rounded to eleven bits or fewer, so the hardware's 2^x and 1/x
// (one step of fp32 each) are enough.
struct Sigmoid {
  float s, c;
};
__device__ __forceinline__ Sigmoid sigmoid(float z) {
  const float t = __builtin_amdgcn_exp2f(-1.44269504088896341f * __builtin_fabsf(z));
  const float big = __builtin_amdgcn_rcpf(1.0f + t), small = t * big;
  return z >= 0.0f ? Sigmoid{big, small} : Sigmoid{small, big};
}

__device__ __forceinline__ float silu(float z) { return z * sigmoid(z).s; }

// d/dz z sigma(z) = sigma (1 + z (1 - sigma))
__device__ __forceinline__ float silu_slope(float z) {
  const Sigmoid q = sigmoid(z);
  return q.s * (1.0f + z * q.c);
}

// Phi(z) = erfc(-z / sqrt 2) / 2, the form that keeps its precision at negative z.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.707106781186547524f * z); }

__device__ __forceinline__ float gelu(float z) { return z * normal_cdf(z); }

// d/dz z Phi(z) = Phi(z) + z phi(z)
__device__ __forceinline__ float gelu_slope(float z) {
  const float pdf = 0.398942280401432678f * __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
  return normal_cdf(z) + z * pdf;
}

// act(z) and act'(z) of the activations without a gate; `act` is uniform.
__device__ __forceinline__ float activate(float z, int act) {
  return act == MOE_ACT_SILU ? silu(z) : act == MOE_ACT_GELU ? gelu(z) : z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  return act == MOE_ACT_SILU ? silu_slope(z) : act == MOE_ACT_GELU ? gelu_slope(z) : 1.0f;
}

}  // namespace moe
