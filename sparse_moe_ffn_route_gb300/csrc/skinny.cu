// Linear layers for the few tokens of a decode step: y[t, o] = sum_k x[t, k] W[o, k], with
// bf16 weights or 4-bit codes with group scales, optionally both halves of a gated layer
// with the activation fused (h = act(x Wg^T, x Wu^T)).
//
// The weights dominate: every weight is read once per 16 tokens, so the work is a stream
// of weights past operands that stay close.  One persistent CTA of 16 warps per SM takes
// units of 32 weight rows (gated: 16 gate rows and the 16 up rows of the same features).
// Its warps take alternate steps of k, keep the loads of two steps in flight in registers
// (64 to 128 KiB per SM, and the next unit's first steps while a unit is summed up), and
// add their partial sums through shared memory in a fixed order.  x lies in shared memory
// as the fragments that the warp MMA wants, one conflict-free 16-byte read per 8 tokens
// and 32 k, which serves two tiles of 16 rows: read from L2 instead, x of 16 tokens was
// four times the traffic of 4-bit weights.  Longer x than 128 KiB is taken in phases: all
// of the CTA's units over the first piece of k, then over the next (the loads in flight
// need the rest of the SM's 256 KiB as L1: with 215 KiB of shared memory in use a
// 4096 x 12288 product took 41 us instead of 25).
//
// The weights are the A operand (16 rows) of the m16n8k16 MMA, loaded straight into
// registers, 16 bytes per lane; the tokens are its 8 columns.  The order of k within an
// MMA is free as long as A and B agree: lane c of a quad takes 8 consecutive k (bf16).
//
// 4-bit codes: 8 codes of a 32-bit word become four bf16 pairs by masking them onto the
// bits of 128.0 (128 + q is exact in bf16), from which 128 + zero is subtracted exactly;
// the scale multiplies each group's fp32 partial sum, so no product is rounded early.
#include "block.h"
#include "common.cuh"
#include "glu_act.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kUnitRows = 32;
constexpr int kPitch = kUnitRows + 4;   // floats per token of a warp's partial sums
constexpr int kPhaseBytes = 128 * 1024;   // x in shared memory
constexpr int kPartBytes = 16 * 1024;     // units' sums kept between phases

// x (and, gated FFN, the low halves of a two-part x: token columns 8..15) as the caller has it
struct Tokens {
  const uint16_t *x, *lo;
  int T, K;
};

// Where the 8 values of token column n (0 .. 8 NC - 1) of this pass from input k on lie;
// null past the last token or input.
__device__ __forceinline__ const uint16_t* token_at(const Tokens& tk, int t0, int n, int k) {
  const uint16_t* p = tk.x;
  int t = t0 + n;
  if (tk.lo && n >= 8) {
    p = tk.lo;
    t = n - 8;
  }
  return t < tk.T && k < tk.K ? p + (size_t)t * tk.K + k : nullptr;
}

// Starts the copy of those 8 values to shared memory (zeros where there are none).
__device__ __forceinline__ void stage8(uint4* dst, const Tokens& tk, int t0, int n, int k) {
  const uint16_t* p = token_at(tk, t0, n, k);
  tc::cp_async16(tc::smem_u32(dst), p ? p : tk.x, p ? 16u : 0u);
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Inputs (0,4) (1,5) (2,6) (3,7) of 8: the pairs that masking a word of codes gives.
__device__ __forceinline__ uint4 code_pairs(const uint4& v) {
  return make_uint4(prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u), prmt(v.y, v.w, 0x5410u), prmt(v.y, v.w, 0x7632u));
}

// The 16 warps' partial sums of a unit, added in warp order: thread (row, token).
// acc[b][n][i]: rows 16 b + g (+ 8 for i >= 2), token columns 8 n + 2 c + (i & 1).
// With several phases of k the sums so far of the CTA's i-th unit wait in part[i].
template <bool GLU, int NC>
__device__ __forceinline__ void finish_unit(float* red, float* part, bool first, bool last, float (&acc)[2][NC][4],
                                            int unit, int n_out, int t0, const Tokens& tk, const GluAct& act,
                                            uint16_t* y, uint16_t* y_lo) {
  constexpr int TOK = 8 * NC;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
  float* w = red + warp * TOK * kPitch;
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[(8 * n + 2 * c + (i & 1)) * kPitch + 16 * b + gq + 8 * (i >> 1)] = acc[b][n][i];
        acc[b][n][i] = 0.f;
      }
  __syncthreads();
  const int row = lane, t = warp;
  if (t < TOK && !(tk.lo && t >= 8)) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) s += red[(v * TOK + t) * kPitch + row];
    if (NC == 2 && tk.lo) {
      float l = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) l += red[(v * TOK + t + 8 * (NC - 1)) * kPitch + row];
      s += l;
    }
    if (!first) s += part[t * kUnitRows + row];
    if (!last) part[t * kUnitRows + row] = s;
    int o = unit * kUnitRows + row;
    if (GLU) {
      const float u = __shfl_down_sync(0xffffffffu, s, 16);
      s = glu_value(act, s, u);
      o = row < 16 ? unit * 16 + row : n_out;
    }
    if (last && o < n_out && t0 + t < tk.T) {
      const size_t at = (size_t)(t0 + t) * n_out + o;
      const uint16_t hi = f32_to_bf16(s);
      y[at] = hi;
      if (y_lo) {   // what the rounding lost (nothing where hi is not finite)
        const float d = s - bf16_to_f32(hi);
        y_lo[at] = fabsf(d) < 3.0e38f ? f32_to_bf16(d) : (uint16_t)0;
      }
    }
  }
  __syncthreads();
}

// Row h (0, 1: +8) of tile b of a unit, as seen by lane group gq; clamped to the last row
// (whose sums are then not stored).
template <bool GLU>
__device__ __forceinline__ size_t unit_row(int unit, int b, int h, int gq, int n_out) {
  const int r = (GLU ? unit * 16 : unit * kUnitRows + 16 * b) + gq + 8 * h;
  return (size_t)(GLU ? b * n_out : 0) + (r < n_out ? r : n_out - 1);
}

// The steps of a warp in order: phase by phase, in a phase unit by unit, in a unit its
// steps st = warp + 16 j of the phase's.
struct Walk {
  int phase, unit, j;
  __device__ __forceinline__ void next(int per, int units) {
    if (++j < per) return;
    j = 0;
    unit += gridDim.x;
    if (unit < units) return;
    unit = blockIdx.x;
    ++phase;
  }
};

// How a product is cut: steps of k in all and per phase, steps of a warp per unit and phase.
struct Cut {
  int steps, phase_steps, phases, per, units;
  __device__ __forceinline__ int step(const Walk& w, int warp) const {   // -1: none
    const int in = warp + kWarps * w.j, st = w.phase * phase_steps + in;
    return w.phase < phases && in < phase_steps && st < steps ? st : -1;
  }
};

// ---------------------------------------------------------------- bf16 weights
// A step is 64 k: two vectors per row.
struct StepBf16 {
  uint4 v[2][2][2];   // tile, row half, 32 k
};

// early: what precedes on the stream is this file's gate/up kernel, which lets the next
// start only after everything before it is done; so the weights may be read before the
// wait for it.
template <bool GLU, int NC>
__global__ void __launch_bounds__(kWarps * 32, 1) skinny_bf16_kernel(const uint16_t* w0, const uint16_t* w1, int n_out,
                                                                     Tokens tk, Cut cut, GluAct act, uint16_t* y,
                                                                     uint16_t* y_lo, uint32_t* clear_status, bool early) {
  extern __shared__ uint4 smem[];
  float* red = reinterpret_cast<float*>(smem);
  uint4* xs = smem + kWarps * 8 * NC * kPitch / 4;
  float* part = reinterpret_cast<float*>(xs + 2 * cut.phase_steps * NC * 32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
  const int K = tk.K, t0 = blockIdx.y * 8 * NC;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if (!early) pdl_wait();

  auto load = [&](StepBf16& s, const Walk& w) {
    const int st = cut.step(w, warp);
    if (st < 0) return;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint16_t* m = GLU && b ? w1 : w0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint16_t* p = m + (unit_row<GLU>(w.unit, b, h, gq, n_out) - (GLU && b ? n_out : 0)) * K;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int k = 64 * st + 32 * q + 8 * c;
          s.v[b][h][q] = k < K ? ldg_stream_v4(p + k) : zero;
        }
      }
    }
  };
  float acc[2][NC][4] = {};
  Walk at{0, (int)blockIdx.x, 0}, ld = at;   // the step being multiplied, the step being loaded
  auto multiply = [&](const StepBf16& s) {
    const int st = cut.step(at, warp) - at.phase * cut.phase_steps;
    if (st < 0) return;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const uint4 x = xs[((2 * st + q) * NC + n) * 32 + lane];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint4 &a = s.v[b][0][q], &d = s.v[b][1][q];
          mma_bf16_16816(acc[b][n], a.x, d.x, a.y, d.y, x.x, x.y);
          mma_bf16_16816(acc[b][n], a.z, d.z, a.w, d.w, x.z, x.w);
        }
      }
  };
  StepBf16 s0, s1;
  load(s0, ld);
  ld.next(cut.per, cut.units);
  load(s1, ld);
  ld.next(cut.per, cut.units);
  if (early) pdl_wait();
  pdl_trigger();
  if (clear_status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *clear_status = 0u;
  auto stage = [&](int phase) {   // x of a phase; what the last phase read is done with
    for (int i = threadIdx.x; i < 2 * cut.phase_steps * NC * 32; i += kWarps * 32) {
      const int l = i & 31, n = (i >> 5) % NC, q = (i >> 5) / NC + 2 * cut.phase_steps * phase;
      stage8(xs + i, tk, t0, 8 * n + (l >> 2), 32 * q + 8 * (l & 3));
    }
    tc::cp_async_wait_all();
    __syncthreads();
  };
  stage(0);
  auto turn = [&](StepBf16& s) {
    multiply(s);
    load(s, ld);
    ld.next(cut.per, cut.units);
    if (at.j == cut.per - 1)
      finish_unit<GLU, NC>(red, part + (at.unit / gridDim.x) * 8 * NC * kUnitRows, at.phase == 0,
                           at.phase == cut.phases - 1, acc, at.unit, n_out, t0, tk, act, y, y_lo);
    const int phase = at.phase;
    at.next(cut.per, cut.units);
    if (at.phase != phase && at.phase < cut.phases) stage(at.phase);
  };
  while (at.phase < cut.phases) {
    turn(s0);
    if (at.phase >= cut.phases) break;
    turn(s1);
  }
}

// ---------------------------------------------------------------- 4-bit codes
__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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

// A step is 128 k: lane c holds the 32 codes of inputs 128 st + 32 c .. + 31 of its rows,
// and one group's scale (upper half) and zero (lower half) per row: the group of those
// inputs.
struct StepW4 {
  uint32_t w[2][2][4];
  uint32_t sz[2][2];
};

template <int GROUP, bool GLU, int NC>
__global__ void __launch_bounds__(kWarps * 32, 1) skinny_w4_kernel(const uint8_t* codes, const uint16_t* scales,
                                                                   const uint8_t* zeros, int n_out, Tokens tk, Cut cut,
                                                                   GluAct act, uint16_t* y) {
  extern __shared__ uint4 smem[];
  float* red = reinterpret_cast<float*>(smem);
  uint4* xs = smem + kWarps * 8 * NC * kPitch / 4;
  float* part = reinterpret_cast<float*>(xs + 4 * cut.phase_steps * NC * 32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
  const int K = tk.K, ng = K / GROUP, t0 = blockIdx.y * 8 * NC;
  pdl_wait();
  pdl_trigger();

  auto load = [&](StepW4& s, const Walk& wk) {
    const int st = cut.step(wk, warp);
    if (st < 0) return;
    const int k = 128 * st + 32 * c;
    const bool in = k < K;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const size_t r = unit_row<GLU>(wk.unit, b, h, gq, n_out);
        const uint4 v = in ? ldg_stream_v4(codes + r * (size_t)(K / 2) + k / 2) : make_uint4(0u, 0u, 0u, 0u);
        s.w[b][h][0] = v.x;
        s.w[b][h][1] = v.y;
        s.w[b][h][2] = v.z;
        s.w[b][h][3] = v.w;
        const size_t at = r * ng + k / GROUP;
        const uint32_t sc = in ? scales[at] : 0u, z = in && zeros ? zeros[at] & 15u : 8u;
        s.sz[b][h] = (sc << 16) | z;
      }
  };
  float acc[2][NC][4] = {};
  Walk at{0, (int)blockIdx.x, 0}, ld = at;
  auto multiply = [&](StepW4& s) {
    const int st = cut.step(at, warp) - at.phase * cut.phase_steps;
    if (st < 0) return;
    // word j: GROUP 128, inputs 128 st + 32 c + 8 j .. + 7; else the quad's words are
    // exchanged so that word j of all four lanes lies in inputs 128 st + 32 j .. + 31
    if (GROUP != 128) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) quad_transpose(s.w[b][h], c);
    }
    constexpr int kWords = GROUP / 32;   // words (of all lanes) per group
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += kWords) {
      float part[2][NC][4] = {};
      uint32_t sz[2][2], zp[2][2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // lane j0 of the quad loaded this group's scale
          sz[b][h] = GROUP == 128 ? s.sz[b][h] : __shfl_sync(0xffffffffu, s.sz[b][h], (lane & ~3) | j0);
          zp[b][h] = (0x4300u + (sz[b][h] & 15u)) * 0x00010001u;   // 128 + zero, twice
        }
#pragma unroll
      for (int i = j0; i < j0 + kWords; ++i) {
        uint4 x[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n)
          x[n] = xs[((4 * st + i) * NC + n) * 32 + lane];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t pa[4], pc[4];
          w4_pairs(s.w[b][0][i], zp[b][0], pa);
          w4_pairs(s.w[b][1][i], zp[b][1], pc);
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            mma_bf16_16816(part[b][n], pa[0], pc[0], pa[1], pc[1], x[n].x, x[n].y);
            mma_bf16_16816(part[b][n], pa[2], pc[2], pa[3], pc[3], x[n].z, x[n].w);
          }
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float sa = __uint_as_float(sz[b][0] & 0xffff0000u), sc = __uint_as_float(sz[b][1] & 0xffff0000u);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          acc[b][n][0] += sa * part[b][n][0];
          acc[b][n][1] += sa * part[b][n][1];
          acc[b][n][2] += sc * part[b][n][2];
          acc[b][n][3] += sc * part[b][n][3];
        }
      }
    }
  };
  StepW4 s0, s1;
  load(s0, ld);
  ld.next(cut.per, cut.units);
  load(s1, ld);
  ld.next(cut.per, cut.units);
  auto stage = [&](int phase) {
    const int n = 4 * cut.phase_steps * NC * 32;
    for (int i = threadIdx.x; i < n; i += kWarps * 32) {
      const int l = i & 31, col = (i >> 5) % NC, q = (i >> 5) / NC + 4 * cut.phase_steps * phase;   // 4 step + word
      const int k = 128 * (q >> 2) + (GROUP == 128 ? 32 * (l & 3) + 8 * (q & 3) : 32 * (q & 3) + 8 * (l & 3));
      stage8(xs + i, tk, t0, 8 * col + (l >> 2), k);
    }
    tc::cp_async_wait_all();
    // each thread turns the vectors that it copied into the codes' order
    for (int i = threadIdx.x; i < n; i += kWarps * 32) xs[i] = code_pairs(xs[i]);
    __syncthreads();
  };
  stage(0);
  auto turn = [&](StepW4& s) {
    multiply(s);
    load(s, ld);
    ld.next(cut.per, cut.units);
    if (at.j == cut.per - 1)
      finish_unit<GLU, NC>(red, part + (at.unit / gridDim.x) * 8 * NC * kUnitRows, at.phase == 0,
                           at.phase == cut.phases - 1, acc, at.unit, n_out, t0, tk, act, y, nullptr);
    const int phase = at.phase;
    at.next(cut.per, cut.units);
    if (at.phase != phase && at.phase < cut.phases) stage(at.phase);
  };
  while (at.phase < cut.phases) {
    turn(s0);
    if (at.phase >= cut.phases) break;
    turn(s1);
  }
}

// ---------------------------------------------------------------- host
// Everything but the kernel: token columns of a pass (16 when more than 8 are there), the
// cut of k, shared memory and the grid.
struct Plan {
  int nc, passes, ctas, smem;
  Cut cut;
};

Plan plan_for(int T, int K, int step, int units, bool two_part) {
  Plan p;
  p.nc = T > 8 || two_part ? 2 : 1;
  p.passes = two_part ? 1 : (T + 8 * p.nc - 1) / (8 * p.nc);
  Cut& c = p.cut;
  c.units = units;
  c.steps = (K + step - 1) / step;
  const int most = kPhaseBytes / (16 * p.nc * step);   // steps of x that fit
  c.phases = (c.steps + most - 1) / most;
  c.phase_steps = c.phases == 1 ? c.steps : most;
  c.per = (c.phase_steps + kWarps - 1) / kWarps;
  p.smem = kWarps * 8 * p.nc * kPitch * 4 + c.phase_steps * step * p.nc * 16 + (c.phases > 1 ? kPartBytes : 0);
  // the passes over 8 or 16 tokens run side by side, so that the later ones find the
  // weights in L2
  p.ctas = sm_count() / p.passes;
  if (p.ctas < 1) p.ctas = 1;
  if (p.ctas > units) p.ctas = units;
  if (c.phases > 1) {
    const int each = kPartBytes / (8 * p.nc * kUnitRows * 4);   // units whose sums a CTA can keep
    const int least = (units + each - 1) / each;
    if (p.ctas < least) p.ctas = least;
  }
  return p;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_skinny(void (*kernel)(KArgs...), const Plan& p, cudaStream_t s, Args&&... args) {
  if (p.smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(p.ctas, p.passes), dim3(kWarps * 32), p.smem, s, static_cast<Args&&>(args)...);
}

template <int GROUP, bool GLU>
cudaError_t launch_w4(const moe_w4_cfg_t& c, const moe_w4_weights_t& w, const uint16_t* x, int T, uint16_t* y,
                      cudaStream_t s) {
  const uint8_t* codes = static_cast<const uint8_t*>(w.codes);
  const uint16_t* sc = static_cast<const uint16_t*>(w.scales);
  const uint8_t* z = static_cast<const uint8_t*>(w.zeros);
  const GluAct act{c.act, c.glu_limit, c.glu_alpha};
  const Tokens tk{x, nullptr, T, c.n_in};
  const Plan p = plan_for(T, c.n_in, 128, GLU ? (c.n_out + 15) / 16 : (c.n_out + kUnitRows - 1) / kUnitRows, false);
  auto* k = p.nc == 2 ? skinny_w4_kernel<GROUP, GLU, 2> : skinny_w4_kernel<GROUP, GLU, 1>;
  return launch_skinny(k, p, s, codes, sc, z, c.n_out, tk, p.cut, act, y);
}

}  // namespace

cudaError_t launch_skinny_bf16(const uint16_t* w0, const uint16_t* w1, int n_out, int n_in, const uint16_t* x,
                               const uint16_t* x_lo, int T, const GluParams* g, uint16_t* y, uint16_t* y_lo,
                               uint32_t* clear_status, bool early, cudaStream_t s) {
  const GluAct act = g ? GluAct{g->act, g->limit, g->alpha} : GluAct{0, 0.f, 0.f};
  const Tokens tk{x, x_lo, T, n_in};
  const Plan p = plan_for(T, n_in, 64, g ? (n_out + 15) / 16 : (n_out + kUnitRows - 1) / kUnitRows, x_lo != nullptr);
  auto* k = g ? (p.nc == 2 ? skinny_bf16_kernel<true, 2> : skinny_bf16_kernel<true, 1>)
              : (p.nc == 2 ? skinny_bf16_kernel<false, 2> : skinny_bf16_kernel<false, 1>);
  return launch_skinny(k, p, s, w0, w1, n_out, tk, p.cut, act, y, y_lo, clear_status, early);
}

cudaError_t launch_skinny_w4(const moe_w4_cfg_t& c, const moe_w4_weights_t& w, const uint16_t* x, int T, uint16_t* y,
                             cudaStream_t s) {
  constexpr int kMost = 1 << 18;   // tokens of a launch: at most 65535 passes of 8
  for (; T > kMost; T -= kMost, x += (size_t)kMost * c.n_in, y += (size_t)kMost * c.n_out) {
    const cudaError_t e = launch_skinny_w4(c, w, x, kMost, y, s);
    if (e != cudaSuccess) return e;
  }
  switch (c.group) {
    case 32: return c.glu ? launch_w4<32, true>(c, w, x, T, y, s) : launch_w4<32, false>(c, w, x, T, y, s);
    case 64: return c.glu ? launch_w4<64, true>(c, w, x, T, y, s) : launch_w4<64, false>(c, w, x, T, y, s);
    default: return c.glu ? launch_w4<128, true>(c, w, x, T, y, s) : launch_w4<128, false>(c, w, x, T, y, s);
  }
}

}  // namespace moe
