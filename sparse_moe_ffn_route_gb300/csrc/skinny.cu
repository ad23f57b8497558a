// Linear layers for the few tokens of a decode step: y[t, o] = sum_k x[t, k] W[o, k], with
// bf16 weights or 4-bit codes with group scales, optionally both halves of a gated layer
// with the activation fused (h = act(x Wg^T, x Wu^T)).
//
// The weights dominate: every weight is read once per 16 tokens, so the work is a stream
// of weights past operands that stay close.  A warp multiplies 16 weight rows (the A
// operand of the m16n8k16 warp MMA, loaded straight into registers, 16 bytes per lane)
// with 8 tokens at a time (the B operand); the 8 warps of a CTA take alternate pieces of
// k and add their partial sums through shared memory in a fixed order.  The order of k
// within an MMA is free as long as A and B agree: lane c of a quad takes 8 consecutive k
// (bf16), so both operands load as whole 16-byte vectors.
//
// 4-bit codes: 8 codes of a 32-bit word become four bf16 pairs by masking them onto the
// bits of 128.0 (128 + q is exact in bf16), from which 128 + zero is subtracted exactly;
// the scale multiplies each group's fp32 partial sum, so no product is rounded early.
#include "block.h"
#include "common.cuh"
#include "glu_act.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;   // weight rows per tile

// The CTA's partial sums [warp][matrix][row][token] added in warp order, activation, y.
template <bool GLU, int NC>
__device__ __forceinline__ void finish_tile(float* red, const float (&acc)[GLU ? 2 : 1][NC][4], int rb, int n_out,
                                            int t0, int T, const GluAct& act, uint16_t* y) {
  constexpr int NM = GLU ? 2 : 1, TOK = 8 * NC;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
  float* w = red + warp * NM * kRows * TOK;
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int col = 8 * n + 2 * c;
      float* p = w + m * kRows * TOK;
      *reinterpret_cast<float2*>(p + gq * TOK + col) = make_float2(acc[m][n][0], acc[m][n][1]);
      *reinterpret_cast<float2*>(p + (gq + 8) * TOK + col) = make_float2(acc[m][n][2], acc[m][n][3]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * TOK; i += kWarps * 32) {
    const int r = i & (kRows - 1), t = i / kRows;
    float s[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      s[m] = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) s[m] += red[(v * NM + m) * kRows * TOK + r * TOK + t];
    }
    const int o = rb * kRows + r;
    if (o < n_out && t0 + t < T)
      y[(size_t)(t0 + t) * n_out + o] = f32_to_bf16(GLU ? glu_value(act, s[0], s[NM - 1]) : s[0]);
  }
  __syncthreads();
}

template <bool GLU, int NC>
__global__ void __launch_bounds__(kWarps * 32) skinny_bf16_kernel(const uint16_t* __restrict__ w0,
                                                                  const uint16_t* __restrict__ w1, int n_out, int K,
                                                                  const uint16_t* x, int T, GluAct act,
                                                                  uint16_t* __restrict__ y, uint32_t* clear_status) {
  constexpr int NM = GLU ? 2 : 1;
  __shared__ float red[kWarps * NM * kRows * 8 * NC];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
  pdl_wait();
  if (clear_status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *clear_status = 0u;
  const int t0 = blockIdx.y * 8 * NC;
  const int n_rb = (n_out + kRows - 1) / kRows;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int rb = blockIdx.x; rb < n_rb; rb += gridDim.x) {
    const size_t ra = (size_t)min(rb * kRows + gq, n_out - 1) * K, rc = (size_t)min(rb * kRows + gq + 8, n_out - 1) * K;
    float acc[NM][NC][4] = {};
    constexpr int U = 4;   // 32-k steps in flight
    for (int kb = warp * 32 * U; kb < K; kb += kWarps * 32 * U) {
      uint4 a[U][NM][2], b[U][NC];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int k = kb + 32 * i + 8 * c;
        const bool in = k < K;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          const uint16_t* w = m ? w1 : w0;
          a[i][m][0] = in ? ldg_stream_v4(w + ra + k) : zero;
          a[i][m][1] = in ? ldg_stream_v4(w + rc + k) : zero;
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const int t = t0 + 8 * n + gq;
          b[i][n] = in && t < T ? *reinterpret_cast<const uint4*>(x + (size_t)t * K + k) : zero;
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            mma_bf16_16816(acc[m][n], a[i][m][0].x, a[i][m][1].x, a[i][m][0].y, a[i][m][1].y, b[i][n].x, b[i][n].y);
            mma_bf16_16816(acc[m][n], a[i][m][0].z, a[i][m][1].z, a[i][m][0].w, a[i][m][1].w, b[i][n].z, b[i][n].w);
          }
    }
    finish_tile<GLU, NC>(red, acc, rb, n_out, t0, T, act, y);
  }
  pdl_trigger();
}

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// 4 x 4 words across the lanes of a quad: word j of lane c becomes word c of lane j.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int c) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool hi = c & bit;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & bit) continue;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? w[j] : w[j + bit], bit);
      if (hi) w[j] = got;
      else w[j + bit] = got;
    }
  }
}

// The 8 codes of one word (code i in bits 4i..4i+3) as bf16 pairs (0,4) (1,5) (2,6) (3,7),
// minus the zero point; zp = (128 + zero) as a bf16 pair.
__device__ __forceinline__ void w4_pairs(uint32_t w, uint32_t zp, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = bf16x2_sub(((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, zp);
}

// (128 + z) twice, as bf16: 128 + z for z in 0..15 is 0x4300 + z.
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) { return (0x4300u + z) * 0x00010001u; }

template <int GROUP, bool GLU, int NC>
__global__ void __launch_bounds__(kWarps * 32) skinny_w4_kernel(const uint8_t* __restrict__ codes,
                                                                const uint16_t* __restrict__ scales,
                                                                const uint8_t* __restrict__ zeros, int n_out, int K,
                                                                const uint16_t* x, int T, GluAct act,
                                                                uint16_t* __restrict__ y) {
  constexpr int NM = GLU ? 2 : 1;
  __shared__ float red[kWarps * NM * kRows * 8 * NC];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
  pdl_wait();
  const int t0 = blockIdx.y * 8 * NC;
  const int n_rb = (n_out + kRows - 1) / kRows, ng = K / GROUP;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int rb = blockIdx.x; rb < n_rb; rb += gridDim.x) {
    size_t row[NM][2];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) row[m][h] = (size_t)m * n_out + min(rb * kRows + gq + 8 * h, n_out - 1);
    float acc[NM][NC][4] = {};
    for (int kb = warp * 128; kb < K; kb += kWarps * 128) {
      // lane c holds the 32 codes of inputs kb + 32 c .. + 31 of its rows
      const bool in = kb + 32 * c < K;
      uint32_t w[NM][2][4];
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 v = in ? ldg_stream_v4(codes + row[m][h] * (size_t)(K / 2) + kb / 2 + 16 * c) : zero;
          w[m][h][0] = v.x;
          w[m][h][1] = v.y;
          w[m][h][2] = v.z;
          w[m][h][3] = v.w;
        }
      // word j: GROUP 128, inputs kb + 32 c + 8 j .. + 7; else the quad's words are
      // exchanged so that word j of all four lanes lies in inputs kb + 32 j .. + 31
      uint4 xv[4][NC];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = GROUP == 128 ? kb + 32 * c + 8 * j : kb + 32 * j + 8 * c;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const int t = t0 + 8 * n + gq;
          xv[j][n] = k < K && t < T ? *reinterpret_cast<const uint4*>(x + (size_t)t * K + k) : zero;
        }
      }
      if (GROUP != 128) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) quad_transpose(w[m][h], c);
      }
      constexpr int kWords = GROUP / 32;   // words (of all lanes) per group
#pragma unroll
      for (int j0 = 0; j0 < 4; j0 += kWords) {
        const int kg = kb + 32 * j0;
        if (kg >= K) break;   // K is a multiple of GROUP, not of 128
        const int gi = kg / GROUP;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          float part[NC][4] = {};
          const size_t ga = row[m][0] * ng + gi, gc = row[m][1] * ng + gi;
          const uint32_t za = zero_pair(zeros ? zeros[ga] & 15u : 8u), zc = zero_pair(zeros ? zeros[gc] & 15u : 8u);
#pragma unroll
          for (int j = j0; j < j0 + kWords; ++j) {
            uint32_t pa[4], pc[4];
            w4_pairs(w[m][0][j], za, pa);
            w4_pairs(w[m][1][j], zc, pc);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              const uint4 v = xv[j][n];
              mma_bf16_16816(part[n], pa[0], pc[0], pa[1], pc[1], prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u));
              mma_bf16_16816(part[n], pa[2], pc[2], pa[3], pc[3], prmt(v.y, v.w, 0x5410u), prmt(v.y, v.w, 0x7632u));
            }
          }
          const float sa = bf16_to_f32(scales[ga]), sc = bf16_to_f32(scales[gc]);
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            acc[m][n][0] += sa * part[n][0];
            acc[m][n][1] += sa * part[n][1];
            acc[m][n][2] += sc * part[n][2];
            acc[m][n][3] += sc * part[n][3];
          }
        }
      }
    }
    finish_tile<GLU, NC>(red, acc, rb, n_out, t0, T, act, y);
  }
  pdl_trigger();
}

dim3 grid_for(int n_out, int T, int nc) {
  const int rb = (n_out + kRows - 1) / kRows, most = 4 * sm_count();
  return dim3(rb < most ? rb : most, (T + 8 * nc - 1) / (8 * nc));
}

template <int GROUP>
cudaError_t launch_w4(const moe_w4_cfg_t& c, const moe_w4_weights_t& w, const uint16_t* x, int T, uint16_t* y,
                      cudaStream_t s) {
  const uint8_t* codes = static_cast<const uint8_t*>(w.codes);
  const uint16_t* sc = static_cast<const uint16_t*>(w.scales);
  const uint8_t* z = static_cast<const uint8_t*>(w.zeros);
  const GluAct act{c.act, c.glu_limit, c.glu_alpha};
  const dim3 b(kWarps * 32);
  const int nc = T <= 8 ? 1 : 2;
  const dim3 g = grid_for(c.n_out, T, nc);
  if (c.glu)
    return nc == 1 ? launch_pdl(skinny_w4_kernel<GROUP, true, 1>, g, b, 0, s, codes, sc, z, c.n_out, c.n_in, x, T, act, y)
                   : launch_pdl(skinny_w4_kernel<GROUP, true, 2>, g, b, 0, s, codes, sc, z, c.n_out, c.n_in, x, T, act, y);
  return nc == 1 ? launch_pdl(skinny_w4_kernel<GROUP, false, 1>, g, b, 0, s, codes, sc, z, c.n_out, c.n_in, x, T, act, y)
                 : launch_pdl(skinny_w4_kernel<GROUP, false, 2>, g, b, 0, s, codes, sc, z, c.n_out, c.n_in, x, T, act, y);
}

}  // namespace

cudaError_t launch_skinny_bf16(const uint16_t* w0, const uint16_t* w1, int n_out, int n_in, const uint16_t* x, int T,
                               const GluParams* p, uint16_t* y, uint32_t* clear_status, cudaStream_t s) {
  const GluAct act = p ? GluAct{p->act, p->limit, p->alpha} : GluAct{0, 0.f, 0.f};
  const dim3 b(kWarps * 32);
  const int nc = T <= 8 ? 1 : 2;
  const dim3 g = grid_for(n_out, T, nc);
  if (p)
    return nc == 1 ? launch_pdl(skinny_bf16_kernel<true, 1>, g, b, 0, s, w0, w1, n_out, n_in, x, T, act, y, clear_status)
                   : launch_pdl(skinny_bf16_kernel<true, 2>, g, b, 0, s, w0, w1, n_out, n_in, x, T, act, y, clear_status);
  return nc == 1 ? launch_pdl(skinny_bf16_kernel<false, 1>, g, b, 0, s, w0, w1, n_out, n_in, x, T, act, y, clear_status)
                 : launch_pdl(skinny_bf16_kernel<false, 2>, g, b, 0, s, w0, w1, n_out, n_in, x, T, act, y, clear_status);
}

cudaError_t launch_skinny_w4(const moe_w4_cfg_t& c, const moe_w4_weights_t& w, const uint16_t* x, int T, uint16_t* y,
                             cudaStream_t s) {
  switch (c.group) {
    case 32: return launch_w4<32>(c, w, x, T, y, s);
    case 64: return launch_w4<64>(c, w, x, T, y, s);
    default: return launch_w4<128>(c, w, x, T, y, s);
  }
}

}  // namespace moe
