// The linear layer's epilogue: what becomes of a sum on its way to y.
#pragma once

#include "block.h"
#include "f32x2.cuh"
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

// An epilogue that nothing hides takes as long as its arithmetic, so the activations work on pairs
// and take two special instructions a value (2^x and 1 / x, both 2 2^-23 off at most).
__device__ __forceinline__ F2 exp2_pair(F2 x) {
  float lo, hi;
  split(x, lo, hi);
  asm("ex2.approx.f32 %0, %0;" : "+f"(lo));
  asm("ex2.approx.f32 %0, %0;" : "+f"(hi));
  return f2(lo, hi);
}
__device__ __forceinline__ F2 recip_pair(F2 x) {
  float lo, hi;
  split(x, lo, hi);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(lo));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(hi));
  return f2(lo, hi);
}

constexpr float kLog2E = 1.44269504088896341f;
// sqrt(8 / pi): tanh(u) of the approximate GELU is 2 sigmoid(2 u) - 1, and
// v (1 + tanh u) / 2 = v sigmoid(2 u), which does not cancel for negative v.
constexpr float kTanhSlope = 1.5957691216057308f, kTanhCube = 0.044715f;

// sigmoid(-x / log2 e)
__device__ __forceinline__ F2 logistic(F2 x) { return recip_pair(add2(f2(1.f), exp2_pair(x))); }

// e = exp(-v^2 / 2) and the upper tail q = erfc(a / sqrt 2) / 2 of the normal distribution, a =
// |v|: q e^(a^2 / 2) as a polynomial of 1 / (1 + 0.26 a), fitted to the smallest relative error
// (Lawson's iteration) for a up to 15, where q underflows: 7 2^-23 off in fp32.  So the GELU keeps
// its relative accuracy for negative v, as with erfc itself, which took 12 us more of a
// 4096 x 2048 x 2048 product.
__device__ __forceinline__ void normal_tail(F2 v, F2 a, F2& e, F2& q) {
  e = exp2_pair(mul2(mul2(v, v), f2(-0.5f * kLog2E)));
  const F2 t = recip_pair(fma2(a, f2(0.26f), f2(1.f)));
  F2 p = f2(-0.07727190107107162f);
  p = fma2(p, t, f2(0.2464762032032013f));
  p = fma2(p, t, f2(-0.13571906089782715f));
  p = fma2(p, t, f2(0.19245390594005585f));
  p = fma2(p, t, f2(0.06007691100239754f));
  p = fma2(p, t, f2(0.11101660132408142f));
  p = fma2(p, t, f2(0.10293087363243103f));
  p = fma2(p, t, f2(3.630387072917074e-05f));
  q = mul2(e, p);
}

template <int ACT>
__device__ __forceinline__ F2 linear_value(F2 v) {
  if (ACT == MOE_LINEAR_SILU) return mul2(v, logistic(mul2(v, f2(-kLog2E))));
  if (ACT == MOE_LINEAR_GELU) {
    // max(v, 0) - |v| q; the comparisons let a NaN through, and 20 stands for all above it
    float lo, hi;
    split(v, lo, hi);
    const F2 a = f2(lo > 20.f ? 20.f : fabsf(lo), hi > 20.f ? 20.f : fabsf(hi));
    F2 e, q;
    normal_tail(v, a, e, q);
    return fma2(mul2(a, f2(-1.f)), q, f2(lo < 0.f ? 0.f : lo, hi < 0.f ? 0.f : hi));
  }
  if (ACT == MOE_LINEAR_GELU_TANH) {
    constexpr float a = -kTanhSlope * kLog2E;
    return mul2(v, logistic(mul2(v, fma2(mul2(v, v), f2(a * kTanhCube), f2(a)))));
  }
  return v;
}

// act'(v); 1 - sigmoid(v) is taken as sigmoid(-v).
template <int ACT>
__device__ __forceinline__ F2 linear_slope(F2 v) {
  if (ACT == MOE_LINEAR_SILU) {
    const F2 x = mul2(v, f2(kLog2E));
    return mul2(logistic(mul2(x, f2(-1.f))), fma2(v, logistic(x), f2(1.f)));
  }
  if (ACT == MOE_LINEAR_GELU) {   // Phi(v) + v phi(v)
    float lo, hi;
    split(v, lo, hi);
    F2 e, q;
    normal_tail(v, f2(fabsf(lo), fabsf(hi)), e, q);
    float ql, qh;
    split(q, ql, qh);
    return fma2(mul2(v, f2(0.39894228040143268f)), e, f2(lo < 0.f ? ql : 1.f - ql, hi < 0.f ? qh : 1.f - qh));
  }
  if (ACT == MOE_LINEAR_GELU_TANH) {
    // s(2u) + v s(2u) s(-2u) 2u'.  Past 16 one of the logistics s is 0, and v^2 held at 256 keeps the
    // rest finite: v^3 leaves fp32's range from 1e13 on.
    constexpr float a = kTanhSlope * kLog2E;
    float lo, hi;
    split(mul2(v, v), lo, hi);
    const F2 sq = f2(fminf(lo, 256.f), fminf(hi, 256.f)), x = mul2(v, fma2(sq, f2(a * kTanhCube), f2(a)));
    const F2 up = logistic(mul2(x, f2(-1.f))), down = logistic(x);
    return fma2(mul2(mul2(up, down), v), fma2(sq, f2(3.f * kTanhCube * kTanhSlope), f2(kTanhSlope)), up);
  }
  return f2(1.f);
}

// N pairs through the activation.
template <int N>
__device__ __forceinline__ void linear_values(int act, F2 (&v)[N]) {
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

template <bool B>
struct Bool {
  static constexpr bool value = B;
};

// 2 N sums of a gate's and an up's rows to N pairs of values.
template <int N>
__device__ __forceinline__ void gated_values(const GluAct& a, F2 (&g)[N], const F2 (&u)[N]) {
  auto each = [&](auto clamped) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float gl, gh, ul, uh;
      split(g[i], gl, gh);
      split(u[i], ul, uh);
      g[i] = f2(glu_value<decltype(clamped)::value>(a, gl, ul), glu_value<decltype(clamped)::value>(a, gh, uh));
    }
  };
  if (a.act == MOE_ACT_CLAMPED_GLU) each(Bool<true>{});
  else each(Bool<false>{});
}

// Sums of 8 neighbouring weight rows o, o + 1, ... of one token row to v: v scale + bias.
// xs: the token's scale (EIGHT).
template <bool EIGHT>
__device__ __forceinline__ void linear_affine8(const LinearEpi& e, float xs, int o, F2 (&v)[4]) {
  if (EIGHT) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(e.w_scale + o));
    const float4 b = __ldg(reinterpret_cast<const float4*>(e.w_scale + o) + 1);
    const F2 s[4] = {f2(a.x, a.y), f2(a.z, a.w), f2(b.x, b.y), f2(b.z, b.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(mul2(v[i], f2(xs)), s[i]);   // in this order: the scales' product could underflow
  }
  if (e.bias) {
    F2 b[4];
    unpack8(__ldg(reinterpret_cast<const uint4*>(e.bias + o)), b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], b[i]);
  }
}

// Columns first, first + step, ... of a bias's gradient: a warp to a column, its lanes in turn
// down the rows of partial sums, in one order wherever this runs.
__device__ __forceinline__ void bias_sums(const BiasParts& b, int first, int step, int lane) {
  for (int c = first; c < b.n; c += step) {
    float s = 0.f;
    for (int r = lane; r < b.rows; r += 32) s += b.parts[(size_t)r * b.n + c];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) b.out[c] = f32_to_bf16(s);
  }
}

}  // namespace moe
