// The gated activations of the dense block in fp32, with their derivatives.  Unlike
// fminf / fmaxf the comparisons let a NaN through.
#pragma once

#include "common.cuh"

namespace moe {

// One activation's parameters as the kernels see them.
struct GluAct {
  int act;            // MOE_ACT_*
  float limit, alpha;
};

__device__ __forceinline__ float sigmoid_f32(float v) { return 1.f / (1.f + __expf(-v)); }

__device__ __forceinline__ float glu_value(const GluAct& a, float g, float u) {
  if (a.act == MOE_ACT_SWIGLU) return g * sigmoid_f32(g) * u;
  g = g > a.limit ? a.limit : g;
  u = u > a.limit ? a.limit : (u < -a.limit ? -a.limit : u);
  return (u + 1.f) * g * sigmoid_f32(a.alpha * g);
}

// dg = dh dh/dg, du = dh dh/du; a clamp passes the gradient up to its border, inclusive.
__device__ __forceinline__ void glu_grad(const GluAct& a, float g, float u, float dh, float& dg, float& du) {
  if (a.act == MOE_ACT_SWIGLU) {
    const float s = sigmoid_f32(g);
    du = dh * g * s;
    dg = dh * u * (s + g * s * (1.f - s));
    return;
  }
  const float gc = g > a.limit ? a.limit : g;
  const float uc = u > a.limit ? a.limit : (u < -a.limit ? -a.limit : u);
  const float s = sigmoid_f32(a.alpha * gc);
  du = (u > a.limit || u < -a.limit) ? 0.f : dh * gc * s;
  dg = g > a.limit ? 0.f : dh * (uc + 1.f) * (s + a.alpha * gc * s * (1.f - s));
}

}  // namespace moe
