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

// exp and the quotient by their fast forms (a few 2^-23 off, far below the bf16 rounding
// that follows); an infinite exp gives 0.
__device__ __forceinline__ float sigmoid_f32(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

template <bool CLAMPED>
__device__ __forceinline__ float glu_value(const GluAct& a, float g, float u) {
  if (!CLAMPED) return g * sigmoid_f32(g) * u;
  g = g > a.limit ? a.limit : g;
  u = u > a.limit ? a.limit : (u < -a.limit ? -a.limit : u);
  return (u + 1.f) * g * sigmoid_f32(a.alpha * g);
}

__device__ __forceinline__ float glu_value(const GluAct& a, float g, float u) {
  return a.act == MOE_ACT_SWIGLU ? glu_value<false>(a, g, u) : glu_value<true>(a, g, u);
}

// dg = dh dh/dg, du = dh dh/du; a clamp passes the gradient up to its border, inclusive.
template <bool CLAMPED>
__device__ __forceinline__ void glu_grad(const GluAct& a, float g, float u, float dh, float& dg, float& du) {
  if (!CLAMPED) {
    const float s = sigmoid_f32(g), gs = g * s;
    du = dh * gs;
    dg = dh * u * (s + gs * (1.f - s));
    return;
  }
  const float gc = g > a.limit ? a.limit : g;
  const float uc = u > a.limit ? a.limit : (u < -a.limit ? -a.limit : u);
  const float s = sigmoid_f32(a.alpha * gc), gs = gc * s;
  du = (u > a.limit || u < -a.limit) ? 0.f : dh * gs;
  dg = g > a.limit ? 0.f : dh * (uc + 1.f) * (s + a.alpha * gs * (1.f - s));
}

}  // namespace moe
