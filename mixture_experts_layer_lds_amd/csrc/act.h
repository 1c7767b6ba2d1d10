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

// Phi(z), the normal distribution function, and e^(-z^2 / 2).  For x = |z|:
// 1 - Phi(x) = t e^(-x^2 / 2) Q(t) / 2 with t = 1 / (1 + 0.35 x) and Q the polynomial of
// degree 8 with the least largest relative error on [0, 40], fitted to e^(x^2 / 2)
// erfc(x / sqrt 2) / t by linear programming: 1.9e-7 with coefficients rounded to fp32,
// 4.7e-7 evaluated in it.
// The tail at negative z keeps that precision, times 1 + z^2 for the rounded
// argument of 2^x, as far as fp32 holds it.  (The library's erfcf takes both sides
// of its branches in most waves, and five times the instructions.)
struct Normal {
  float cdf, bell;
};
__device__ __forceinline__ Normal normal(float z) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.35f * __builtin_fabsf(z));
  const float bell = __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
  float q = -0.049991507083177567f;
  q = q * t + 0.2517763376235962f;
  q = q * t - 0.44557279348373413f;
  q = q * t + 0.25329554080963135f;
  q = q * t - 0.008356956765055656f;
  q = q * t + 0.19782276451587677f;
  q = q * t + 0.24233156442642212f;
  q = q * t + 0.27944034337997437f;
  q = q * t + 0.27925488352775574f;
  const float tail = 0.5f * t * bell * q;
  return {z >= 0.0f ? 1.0f - tail : tail, bell};
}

__device__ __forceinline__ float gelu(float z) { return z * normal(z).cdf; }

// d/dz z Phi(z) = Phi(z) + z phi(z)
__device__ __forceinline__ float gelu_slope(float z) {
  const Normal n = normal(z);
  return n.cdf + z * (0.398942280401432678f * n.bell);
}

// act(z) and act'(z) of the activations without a gate; `act` is uniform.
__device__ __forceinline__ float activate(float z, int act) {
  return act == MOE_ACT_SILU ? silu(z) : act == MOE_ACT_GELU ? gelu(z) : z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  return act == MOE_ACT_SILU ? silu_slope(z) : act == MOE_ACT_GELU ? gelu_slope(z) : 1.0f;
}

}  // namespace moe
