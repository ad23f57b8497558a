// Linear layers for the few tokens of a decode step: y[t, o] = sum_k x[t, k] W[o, k], with
// bf16 weights or 4-bit codes with group scales, optionally both halves of a gated layer
// with the activation fused (h = act(x Wg^T, x Wu^T)).
//
// The weights dominate: every weight is read once per 16 tokens, so the work is a stream
// of weights past operands that stay close.  One CTA of 16 warps per SM takes its share of
// the units of 32 weight rows (gated: 16 gate rows and the 16 up rows of the same
// features) at one time, 16, 8, 4, 2 or 1 warps to a unit.  The warps of a unit divide k
// among them and meet only at the end, to add their partial sums through shared memory in
// a fixed order.  A step is 64 bytes of each of the 32 rows; every warp has a ring of its
// own of 3 or 4 steps in shared memory that it fills with asynchronous copies (64 to 128
// KiB in flight per SM without a register or a barrier between warps).
//
// x lies in shared memory, its rows padded so that the MMA's fragments are conflict-free
// 16-byte reads, each of which serves two tiles of 16 rows: read from L2 instead, x of 16
// tokens was four times the traffic of 4-bit weights.  It is copied row by row (512
// contiguous bytes per warp and instruction; gathered in the fragments' order, 16 bytes at
// a time, 128 KiB of it took 12 us).  Longer x than fits is taken in phases of k.
//
// The weights are the A operand (16 rows) of the m16n8k16 MMA, the tokens its 8 columns.
// The order of k within an MMA is free as long as A and B agree: lane c of a quad takes 8
// consecutive k (bf16).
//
// 4-bit codes: 8 codes of a 32-bit word become four bf16 pairs by masking them onto the
// bits of 128.0 (128 + q is exact in bf16), from which 128 + zero is subtracted exactly;
// the scale multiplies each group's fp32 partial sum, so no product is rounded early.
//
// Measured: bf16, 8 tokens, 4096 x 12288 forward 53.3 us for 302 MB (5.67 TB/s, 83% of a
// copy's rate).  4 bits, 16 tokens, 4096 x 32768: 30.4 us for 74 MB (2.4 TB/s), bound by
// issue, integer and MMA work of about 8 us each that overlap poorly (23 us without the
// MMAs); 1 token, 2048 x 512 gated: 3.7 us, the host's launch.
#include "block.h"
#include "common.cuh"
#include "glu_act.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kUnitRows = 32;
constexpr int kPitch = kUnitRows + 4;       // floats per token of a warp's partial sums
constexpr int kSlotBytes = kUnitRows * 64;  // one step of a warp

// Steps ahead of a warp, and the bytes of x that leaves: 16 rings and x fill 227 KiB.
template <int NC>
struct Mem {
  static constexpr int kDepth = NC == 1 ? 4 : 3;
  static constexpr int kRingBytes = kWarps * kDepth * kSlotBytes;
  static constexpr int kPhaseBytes = 227 * 1024 - kRingBytes;
};

// x (and, gated FFN, the low halves of a two-part x: token columns 8..15) as the caller has it
struct Tokens {
  const uint16_t *x, *lo;
  int T, K;
};

// How a product is cut: units of 32 rows, warps to a unit, steps of k in all and per phase.
struct Cut {
  int units, ws, steps, phase_steps;
};

// 16 bytes of weights to shared memory; L2 fetches the 256 bytes around them, which the
// next steps of the row read.
__device__ __forceinline__ void copy_weights16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The same, of which only `bytes` (0 or 16) are read and the rest is zero.
__device__ __forceinline__ void copy_weights16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The row of tile b of a unit that this lane takes first (gq), clamped to the last row, and
// how many rows on its second one lies (8, clamped alike; a clamped row's sums are not
// stored).
template <bool GLU>
__device__ __forceinline__ void unit_rows(int unit, int b, int gq, int n_out, size_t& row, int& down) {
  const int first = GLU ? unit * 16 : unit * kUnitRows + 16 * b;
  const int r0 = min(first + gq, n_out - 1);
  row = (size_t)(GLU ? b * n_out : 0) + r0;
  down = min(first + gq + 8, n_out - 1) - r0;
}

// A slot holds rows [tile][8 + 8 rows][64 bytes]; the four 16-byte pieces of a row lie at
// piece ^ twist(row), so that the quads' reads of 16, 8 or 4 bytes per lane, at the same
// place of 8 rows, meet no bank twice.
__device__ __forceinline__ int twist(int row) { return (row & 2) | ((row >> 2) & 1); }

// ---------------------------------------------------------------- bf16 weights
// A step is 32 k: lane c's piece of a row is k 8 c .. + 7.
struct Bf16 {
  static constexpr int kStep = 32, kScaleSteps = 1 << 20;
  static constexpr int kPad = 64;       // bytes between x's rows beyond a multiple of 128
  static constexpr bool kPairs = false;
  static constexpr bool kZeroEnd = true;   // past the end of a row: zeros, since x's zeros times infinity are NaN
  const uint16_t *w0, *w1;   // gated: gate, up
  struct Scales {};
  struct ScaleRows {};

  static __device__ __forceinline__ uint4 staged(const uint4& v) { return v; }
  template <bool GLU>
  __device__ __forceinline__ const char* row(int b, size_t r, int n_out, int K) const {
    return reinterpret_cast<const char*>(GLU && b ? w1 + (r - n_out) * K : w0 + r * K);
  }
  static __device__ __forceinline__ size_t row_bytes(int K) { return (size_t)K * 2; }
  template <bool GLU>
  __device__ __forceinline__ void scale_rows(ScaleRows&, int, int, int, int) const {}
  __device__ __forceinline__ void load_scales(Scales&, const ScaleRows&, int, int, int) const {}

  // xs: row gq of x at the step's first k; pitch: bytes between x's rows
  template <int NC>
  __device__ __forceinline__ void multiply(const uint8_t* slot, const Scales&, int, const uint8_t* xs, int pitch,
                                           float (&acc)[2][NC][4], int lane) const {
    const int gq = lane >> 2, piece = ((lane & 3) ^ twist(gq)) * 16;
    uint4 w[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i >> 1][i & 1] = *reinterpret_cast<const uint4*>(slot + (8 * i + gq) * 64 + piece);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const uint4 x = *reinterpret_cast<const uint4*>(xs + 8 * n * pitch + 16 * (lane & 3));
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        mma_bf16_16816(acc[b][n], w[b][0].x, w[b][1].x, w[b][0].y, w[b][1].y, x.x, x.y);
        mma_bf16_16816(acc[b][n], w[b][0].z, w[b][1].z, w[b][0].w, w[b][1].w, x.z, x.w);
      }
    }
  }
};

// ---------------------------------------------------------------- 4-bit codes
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The warp MMA with nothing to add to.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// (a & b) | c in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// A step is 128 k, 32 codes per lane and row: words of 8 codes that, word by word, lie in
// one group for all four lanes of a quad (the MMA sums over them before the scale).
template <int GROUP>
struct W4 {
  static constexpr int kStep = 128;
  static constexpr int kPad = GROUP == 32 ? 64 : 16;   // bytes between x's rows beyond a multiple of 128
  static constexpr bool kPairs = true;
  static constexpr bool kZeroEnd = false;  // past the end of a row: any codes, which are finite
  static constexpr int kGroups = 128 / GROUP, kWords = 4 / kGroups;   // groups of a step; words of a group
  static constexpr int kScaleSteps = 4 / kGroups;   // steps whose groups the four lanes of a quad hold
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;

  struct Scales {
    uint32_t sz[2][2];       // this lane's group: scale (upper half) and 128 + zero, both bf16
  };
  struct ScaleRows {
    size_t at[2];            // tile: index of the row's first scale
    unsigned down[2];        // scales to the lane's second row
  };
  // word j of lane c: inputs input(c, j) .. + 7 of the step
  static __device__ __forceinline__ int input(int c, int j) {
    return GROUP == 32 ? 32 * j + 8 * c : 64 * (j >> 1) + 16 * c + 8 * (j & 1);
  }
  // inputs (0,4) (1,5) (2,6) (3,7) of 8: the pairs that masking a word of codes gives
  static __device__ __forceinline__ uint4 staged(const uint4& v) {
    return make_uint4(prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u), prmt(v.y, v.w, 0x5410u),
                      prmt(v.y, v.w, 0x7632u));
  }
  template <bool GLU>
  __device__ __forceinline__ const char* row(int, size_t r, int, int K) const {
    return reinterpret_cast<const char*>(codes) + r * (size_t)(K / 2);
  }
  static __device__ __forceinline__ size_t row_bytes(int K) { return (size_t)(K / 2); }
  template <bool GLU>
  __device__ __forceinline__ void scale_rows(ScaleRows& r, int unit, int gq, int n_out, int K) const {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      size_t row;
      int down;
      unit_rows<GLU>(unit, b, gq, n_out, row, down);
      r.at[b] = row * (size_t)(K / GROUP);
      r.down[b] = (unsigned)down * (unsigned)(K / GROUP);
    }
  }
  // Lane c: group kGroups st + c of its rows; past the end a scale of 0, since the sum of x's
  // zeros there times an infinite one would be NaN.
  __device__ __forceinline__ void load_scales(Scales& s, const ScaleRows& r, int st, int c, int K) const {
    const int end = K / GROUP - 1, gi = min(kGroups * st + c, end);
    const uint32_t keep = GROUP == 128 || kGroups * st + c <= end ? 0xffffu : 0u;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const size_t at = r.at[b] + (unsigned)gi + (h ? r.down[b] : 0u);
        s.sz[b][h] = ((scales[at] & keep) << 16) | (0x4300u + (zeros ? zeros[at] & 15u : 8u));
      }
  }

  // The lane's words of group g of the step in the row at `row` (a multiple of 8 rows from
  // the slot's start, plus gq).
  static __device__ __forceinline__ void words(const uint8_t* row, int c, int tw, int g, uint32_t (&w)[kWords]) {
    if constexpr (GROUP == 32) {
      w[0] = *reinterpret_cast<const uint32_t*>(row + ((g ^ tw) << 4) + 4 * c);
    } else {
#pragma unroll
      for (int q = 0; q < kWords / 2; ++q) {
        const uint2 v = *reinterpret_cast<const uint2*>(row + (((2 * (g + q) + (c >> 1)) ^ tw) << 4) + 8 * (c & 1));
        w[2 * q] = v.x;
        w[2 * q + 1] = v.y;
      }
    }
  }

  template <int NC>
  __device__ __forceinline__ void multiply(const uint8_t* slot, const Scales& scale, int j, const uint8_t* xs, int pitch,
                                           float (&acc)[2][NC][4], int lane) const {
    const int gq = lane >> 2, c = lane & 3, tw = twist(gq);
    const int from = (lane & ~3) | (j % kScaleSteps * kGroups);   // the lane with the step's first group
    uint32_t mask, one;   // kept in registers, so that masking is one instruction
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x43004300;" : "=r"(one));
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float part[2][NC][4];
      uint32_t sz[2][2], zp[2][2], w[2][2][kWords];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        words(slot + (8 * i + gq) * 64, c, tw, g, w[i >> 1][i & 1]);
        sz[i >> 1][i & 1] = __shfl_sync(0xffffffffu, scale.sz[i >> 1][i & 1], from + g);
        zp[i >> 1][i & 1] = prmt(sz[i >> 1][i & 1], 0u, 0x1010u);   // 128 + zero, twice
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint4 x[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n)
          x[n] = *reinterpret_cast<const uint4*>(xs + 8 * n * pitch + 2 * input(c, g * kWords + i));
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t p[2][4];   // row half: pairs (0,4) (1,5) (2,6) (3,7) minus the zero
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[h][e] = bf16x2_sub(and_or(w[b][h][i] >> (4 * e), mask, one), zp[b][h]);
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            if (i == 0) mma_bf16_first(part[b][n], p[0][0], p[1][0], p[0][1], p[1][1], x[n].x, x[n].y);
            else mma_bf16_16816(part[b][n], p[0][0], p[1][0], p[0][1], p[1][1], x[n].x, x[n].y);
            mma_bf16_16816(part[b][n], p[0][2], p[1][2], p[0][3], p[1][3], x[n].z, x[n].w);
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
  }
};

// ---------------------------------------------------------------- the kernel
// early: what precedes on the stream is this file's gate/up kernel, which lets the next
// start only after everything before it is done; so the weights may be read before the
// wait for it.
template <class F, bool GLU, int NC>
__global__ void __launch_bounds__(kWarps * 32, 1) skinny_kernel(const F f, int n_out, const Tokens tk, const Cut cut,
                                                                const GluAct act, uint16_t* y, uint16_t* y_lo,
                                                                uint32_t* clear_status, bool early) {
  constexpr int TOK = 8 * NC, DEPTH = Mem<NC>::kDepth;
  extern __shared__ __align__(16) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem);        // over the rings, once their steps are done with
  uint8_t* xs = smem + Mem<NC>::kRingBytes;           // [token column][k of the phase | pad]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
  const uint8_t* ring = smem + warp * DEPTH * kSlotBytes;
  const uint32_t mine_at = tc::smem_u32(ring) + gq * 64 + ((c ^ twist(gq)) << 4);   // this lane's piece of slot 0
  const int K = tk.K, t0 = blockIdx.y * TOK;
  const int ws = cut.ws, slots = kWarps / ws, mine = warp / ws, part = warp - mine * ws;
  // a warp's steps: a run of per_phase in each phase, from phase_steps phase + first on
  const int per_phase = cut.phase_steps / ws, first = part * per_phase;
  const int phases = (cut.steps + cut.phase_steps - 1) / cut.phase_steps;
  if (!early) pdl_wait();

  const int pitch = cut.phase_steps * F::kStep * 2 / 128 * 128 + 128 + F::kPad;   // bytes between x's rows
  int staged = -1;   // the phase of k whose x is in shared memory
  // Columns without a token keep what is there: they meet no other column in an MMA and are
  // not stored.  Past the last k a token's x is zero.
  auto stage = [&](int phase) {
    if (phase == staged) return;
    if (staged >= 0) __syncthreads();   // the last phase's x is done with
    staged = phase;
    const int k0 = phase * cut.phase_steps * F::kStep, nv = cut.phase_steps * F::kStep / 8;   // vectors of a row
    const int live = min((K - k0) / 8, nv);
    for (int col = warp >> 1; col < TOK; col += kWarps / 2) {
      const bool low = tk.lo && col >= 8;
      const int t = low ? col - 8 : t0 + col;
      if (t >= tk.T) continue;
      const uint16_t* src = (low ? tk.lo : tk.x) + (size_t)t * K + k0;
      uint8_t* dst = xs + col * pitch;
      for (int v = (warp & 1) * 32 + lane; v < nv; v += 64)
        tc::cp_async16(tc::smem_u32(dst + 16 * v), src + (v < live ? 8 * v : 0), v < live ? 16u : 0u);
    }
    tc::cp_async_wait_all();   // and the steps ahead, which were asked for before
    if (F::kPairs)             // each thread turns the vectors that it copied into the order of the codes
      for (int col = warp >> 1; col < TOK; col += kWarps / 2)
        for (int v = (warp & 1) * 32 + lane; v < nv; v += 64) {
          uint4* q = reinterpret_cast<uint4*>(xs + col * pitch + 16 * v);
          *q = F::staged(*q);
        }
    __syncthreads();
  };

  float acc[2][NC][4] = {};
  typename F::Scales scale, scale_next;
  typename F::ScaleRows scale_rows;
  bool begun = false;
  for (int base = blockIdx.x; base < cut.units; base += slots * gridDim.x) {
    const int unit = base + mine * gridDim.x;
    const bool busy = unit < cut.units;
    const char* p[2][2];   // this lane's piece of the first step of its rows
    const int last = (int)F::row_bytes(K) - 16 - 16 * c;
    if (busy) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        size_t row;
        int down;
        unit_rows<GLU>(unit, b, gq, n_out, row, down);
        p[b][0] = f.template row<GLU>(b, row, n_out, K) + 16 * c;
        p[b][1] = p[b][0] + down * F::row_bytes(K);
      }
      f.template scale_rows<GLU>(scale_rows, unit, gq, n_out, K);
    }
    for (int phase = 0; phase < phases; ++phase) {
      const int st0 = phase * cut.phase_steps + first;
      const int run = busy ? min(per_phase, cut.steps - st0) : 0;   // may be negative
      int off = 64 * st0;
      // the copies: DEPTH steps ahead of the multiplications; past the end of a row zeros, or
      // its last piece again (x is zero there)
      auto copy = [&](uint32_t dst) {
        const int o = min(off, last);
        const uint32_t bytes = off <= last ? 16u : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (F::kZeroEnd) copy_weights16(dst + 512 * e, p[e >> 1][e & 1] + o, bytes);
          else copy_weights16(dst + 512 * e, p[e >> 1][e & 1] + o);
        }
        off += 64;
      };
      if (run > 0) f.load_scales(scale_next, scale_rows, st0, c, K);
#pragma unroll
      for (int s = 0; s < DEPTH; ++s) {
        if (s < run) copy(mine_at + s * kSlotBytes);
        tc::cp_async_commit();
      }
      if (!begun) {
        begun = true;
        if (early) pdl_wait();
        pdl_trigger();
        if (clear_status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *clear_status = 0u;
      }
      stage(phase);
      int at = 0;                 // the slot, in bytes
      const uint8_t* x = xs + gq * pitch + first * (F::kStep * 2);
      for (int i = 0; i < run; ++i) {
        if (i % F::kScaleSteps == 0) {
          scale = scale_next;
          if (i + F::kScaleSteps < run) f.load_scales(scale_next, scale_rows, st0 + i + F::kScaleSteps, c, K);
        }
        tc::cp_async_wait<DEPTH - 1>();
        __syncwarp();
        f.template multiply<NC>(ring + at, scale, i, x, pitch, acc, lane);
        x += F::kStep * 2;
        __syncwarp();   // the slot is read
        if (i + DEPTH < run) copy(mine_at + at);
        tc::cp_async_commit();
        at = at == (DEPTH - 1) * kSlotBytes ? 0 : at + kSlotBytes;
      }
    }
    __syncthreads();   // every ring is done with
    // partial sums of the warps: rows 16 b + g (+ 8 for i >= 2), columns 8 n + 2 c + (i & 1)
    float* w = red + warp * TOK * kPitch;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[(8 * n + 2 * c + (e & 1)) * kPitch + 16 * b + gq + 8 * (e >> 1)] = acc[b][n][e];
          acc[b][n][e] = 0.f;
        }
    __syncthreads();
    // a warp takes token columns warp, warp + 16, ... of the slots' units: lane = row
    const int lg = NC == 1 || tk.lo ? 3 : 4;   // 8 or 16 columns
    for (int e = warp; e < slots << lg; e += kWarps) {
      const int sl = e >> lg, t = e & ((1 << lg) - 1), u = base + sl * gridDim.x;
      if (u >= cut.units) break;
      const float* q = red + ((size_t)sl * ws * TOK + t) * kPitch + lane;
      float s = 0.f;
      for (int v = 0; v < ws; ++v) s += q[v * TOK * kPitch];
      if (NC == 2 && tk.lo) {
        float l = 0.f;
        for (int v = 0; v < ws; ++v) l += q[(v * TOK + 8) * kPitch];
        // the low halves only refine: where a weight is infinite they, or their zeros, would
        // turn it into NaN
        if (isfinite(s)) s += l;
      }
      int o = u * kUnitRows + lane;
      if (GLU) {
        const float up = __shfl_down_sync(0xffffffffu, s, 16);
        s = glu_value(act, s, up);
        o = lane < 16 ? u * 16 + lane : n_out;
      }
      if (o < n_out && t0 + t < tk.T) {
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
}

// ---------------------------------------------------------------- host
template <class F, bool GLU, int NC>
cudaError_t launch_one(const F& f, int n_out, const Tokens& tk, const GluAct& act, uint16_t* y, uint16_t* y_lo,
                       uint32_t* clear_status, bool early, cudaStream_t s) {
  Cut c;
  c.units = GLU ? (n_out + 15) / 16 : (n_out + kUnitRows - 1) / kUnitRows;
  c.steps = (tk.K + F::kStep - 1) / F::kStep;
  // the passes over 8 or 16 tokens run side by side, so that the later ones find the
  // weights in L2
  const int passes = tk.lo ? 1 : (tk.T + 8 * NC - 1) / (8 * NC);
  int ctas = sm_count() / passes;
  if (ctas < 1) ctas = 1;
  if (ctas > c.units) ctas = c.units;
  // as many warps to a unit as let a CTA take all of its units at one time
  const int each = (c.units + ctas - 1) / ctas;
  c.ws = kWarps;
  while (c.ws > 1 && kWarps / c.ws < each) c.ws >>= 1;
  // steps of x that fit
  const int most = (Mem<NC>::kPhaseBytes / (8 * NC) - 256) / (F::kStep * 2) / kWarps * kWarps;
  c.phase_steps = c.steps <= most ? (c.steps + c.ws - 1) / c.ws * c.ws : most;
  const int smem = Mem<NC>::kRingBytes + 8 * NC * (c.phase_steps * F::kStep * 2 / 128 * 128 + 128 + F::kPad);
  const cudaError_t e = allow_smem<skinny_kernel<F, GLU, NC>>(227 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(skinny_kernel<F, GLU, NC>, dim3(ctas, passes), dim3(kWarps * 32), smem, s, f, n_out, tk, c, act, y, y_lo, clear_status,
                    early);
}

template <class F>
cudaError_t launch_format(const F& f, bool glu, int n_out, const Tokens& tk, const GluAct& act, uint16_t* y,
                          uint16_t* y_lo, uint32_t* clear_status, bool early, cudaStream_t s) {
  if (tk.T > 8 || tk.lo)
    return glu ? launch_one<F, true, 2>(f, n_out, tk, act, y, y_lo, clear_status, early, s)
               : launch_one<F, false, 2>(f, n_out, tk, act, y, y_lo, clear_status, early, s);
  return glu ? launch_one<F, true, 1>(f, n_out, tk, act, y, y_lo, clear_status, early, s)
             : launch_one<F, false, 1>(f, n_out, tk, act, y, y_lo, clear_status, early, s);
}

}  // namespace

cudaError_t launch_skinny_bf16(const uint16_t* w0, const uint16_t* w1, int n_out, int n_in, const uint16_t* x,
                               const uint16_t* x_lo, int T, const GluParams* g, uint16_t* y, uint16_t* y_lo,
                               uint32_t* clear_status, bool early, cudaStream_t s) {
  const GluAct act = g ? GluAct{g->act, g->limit, g->alpha} : GluAct{0, 0.f, 0.f};
  return launch_format(Bf16{w0, w1}, g != nullptr, n_out, Tokens{x, x_lo, T, n_in}, act, y, y_lo, clear_status, early, s);
}

cudaError_t launch_skinny_w4(const moe_w4_cfg_t& c, const moe_w4_weights_t& w, const uint16_t* x, int T, uint16_t* y,
                             cudaStream_t s) {
  constexpr int kMost = 1 << 18;   // tokens of a launch: at most 65535 passes of 8
  for (; T > kMost; T -= kMost, x += (size_t)kMost * c.n_in, y += (size_t)kMost * c.n_out) {
    const cudaError_t e = launch_skinny_w4(c, w, x, kMost, y, s);
    if (e != cudaSuccess) return e;
  }
  const uint8_t* codes = static_cast<const uint8_t*>(w.codes);
  const uint16_t* sc = static_cast<const uint16_t*>(w.scales);
  const uint8_t* z = static_cast<const uint8_t*>(w.zeros);
  const GluAct act{c.act, c.glu_limit, c.glu_alpha};
  const Tokens tk{x, nullptr, T, c.n_in};
  if (c.group == 32) return launch_format(W4<32>{codes, sc, z}, c.glu, c.n_out, tk, act, y, nullptr, nullptr, false, s);
  if (c.group == 64) return launch_format(W4<64>{codes, sc, z}, c.glu, c.n_out, tk, act, y, nullptr, nullptr, false, s);
  return launch_format(W4<128>{codes, sc, z}, c.glu, c.n_out, tk, act, y, nullptr, nullptr, false, s);
}

}  // namespace moe
