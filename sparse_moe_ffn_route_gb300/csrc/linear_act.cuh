// The linear layer's epilogue: what becomes of a sum on its way to y.
#pragma once

#include "../../include/moe_linear.h"
#include "glu_act.cuh"

namespace moe {

// v = sum (x_scale w_scale) + bias; y = act(v) + residual.  glu: two sums make one y.
struct LinearEpi {
  int act;                        // MOE_LINEAR_*; with glu, see gated
  int glu;
  GluAct gated;
  const uint16_t *bias, *residual;   // bf16 [rows], [T, n_out], or null
  uint16_t* pre;                  // v in bf16 [T, n_out], or null
  const float *x_scale, *w_scale;    // e4m3: [T], [rows]; else null
};

// sqrt(8 / pi): tanh(u) of the approximate GELU is 2 sigmoid(2 u) - 1, and
// v (1 + tanh u) / 2 = v sigmoid(2 u), which does not cancel for negative v.
constexpr float kTanhSlope = 1.5957691216057308f, kTanhCube = 0.044715f;

// v (1 + erf(v / sqrt 2)) / 2 with erfc, which keeps its relative accuracy for negative v.
__device__ __forceinline__ float normal_cdf(float v) { return 0.5f * erfcf(v * -0.70710678118654752f); }

template <int ACT>
__device__ __forceinline__ float linear_value(float v) {
  if (ACT == MOE_LINEAR_SILU) return v * sigmoid_f32(v);
  if (ACT == MOE_LINEAR_GELU) return v * normal_cdf(v);
  if (ACT == MOE_LINEAR_GELU_TANH) return v * sigmoid_f32(kTanhSlope * fmaf(kTanhCube * v * v, v, v));
  return v;
}

// act'(v); 1 - sigmoid(v) is taken as sigmoid(-v).
template <int ACT>
__device__ __forceinline__ float linear_slope(float v) {
  if (ACT == MOE_LINEAR_SILU) return sigmoid_f32(v) * fmaf(v, sigmoid_f32(-v), 1.f);
  if (ACT == MOE_LINEAR_GELU) return fmaf(v * 0.39894228040143268f, __expf(-0.5f * v * v), normal_cdf(v));
  if (ACT == MOE_LINEAR_GELU_TANH) {
    const float u = kTanhSlope * fmaf(kTanhCube * v * v, v, v);
    return sigmoid_f32(u) * fmaf(v * sigmoid_f32(-u), kTanhSlope * fmaf(3.f * kTanhCube, v * v, 1.f), 1.f);
  }
  return 1.f;
}

// N values of one row through the activation.
template <int N>
__device__ __forceinline__ void linear_values(int act, float (&v)[N]) {
  if (act == MOE_LINEAR_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = linear_value<MOE_LINEAR_SILU>(v[i]);
  } else if (act == MOE_LINEAR_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = linear_value<MOE_LINEAR_GELU>(v[i]);
  } else if (act == MOE_LINEAR_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = linear_value<MOE_LINEAR_GELU_TANH>(v[i]);
  }
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& q, float (&f)[8]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(u[i]);
    f[2 * i + 1] = bf16_hi(u[i]);
  }
}

// Sums of 8 neighbouring weight rows o, o + 1, ... of one token row to v: v scale + bias.
// xs: the token's scale (EIGHT).
template <bool EIGHT>
__device__ __forceinline__ void linear_affine8(const LinearEpi& e, float xs, int o, float* v) {
  if (EIGHT) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(e.w_scale + o));
    const float4 b = __ldg(reinterpret_cast<const float4*>(e.w_scale + o) + 1);
    const float s[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * xs * s[i];   // in this order: no product of scales that could underflow
  }
  if (e.bias) {
    float b[8];
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(e.bias + o)), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
}

__device__ __forceinline__ void add_bf16x8(float* v, const uint4& q) {
  float f[8];
  unpack_bf16x8(q, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += f[i];
}

}  // namespace moe
