// The linear layer for the few tokens (at most 16) of a decode step: the weights stream past x,
// bf16 or e4m3, as in skinny.cu through warp MMAs fed by rings of asynchronous copies.
//
// Bound by the weights' bytes: each CTA (one per SM) takes an even share of the features, to the
// row, in tiles of 16 weight rows (gated: 8 gate rows and the 8 up rows of the same features),
// all tiles at one time where they are 16 or fewer, 16 / tiles warps to a tile that divide k among
// them.  Rows past a CTA's share are not read.  (Units of 32 rows, of which some SMs get one
// more than others, take 25.7 us for 16 tokens and 4096 x 12288 gated in 8 bits, these shares
// 23.9; units of two tiles for the smaller products gained nothing.)
//
// A step is 128 bytes of each of the 16 rows; a warp's ring holds as many steps as fit beside x.
// The weights are the A operand of m16n8k16 MMAs, the tokens its columns; the order of k
// within an MMA is free as long as A and B agree, so lane c of a quad takes pieces c and c + 4
// of 16 bytes.  e4m3 values become f16, which holds all of them, so that products are exact and
// sums fp32 (the warp MMA on e4m3 itself was slower: 26.7 us instead of 25.7).
//
// Measured: 1 token, 4096 x 12288 gated, bf16 35.7 us for 201 MB (5.6 TB/s, 83% of a copy's
// rate), 8 bits 20.5 us for 101 MB: about 4 us of a launch go by before the stream is up to
// speed and after it, the rest runs at 6.4 TB/s.  16 tokens take 3 us more: x is copied to every
// SM, and the MMAs' columns are all in use.
#include <algorithm>

#include "block.h"
#include "common.cuh"
#include "linear_act.cuh"
#include "stream_cut.h"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kWarps = kStreamWarps, kSpace = kStreamSpace;

struct StreamArgs {
  const uint8_t *w, *x;        // rows of `row` bytes
  int n, T, row;
  Cut cut;
  LinearEpi epi;
  uint16_t* y;
  uint32_t* status;
};

// All but the last n (at most 12) groups of this thread's copies are there.
__device__ __forceinline__ void copies_wait(int n) {
  if (n >= 8) {
    if (n >= 12) tc::cp_async_wait<12>();
    else if (n == 11) tc::cp_async_wait<11>();
    else if (n == 10) tc::cp_async_wait<10>();
    else if (n == 9) tc::cp_async_wait<9>();
    else tc::cp_async_wait<8>();
  } else if (n >= 4) {
    if (n == 7) tc::cp_async_wait<7>();
    else if (n == 6) tc::cp_async_wait<6>();
    else if (n == 5) tc::cp_async_wait<5>();
    else tc::cp_async_wait<4>();
  } else {
    if (n == 3) tc::cp_async_wait<3>();
    else if (n == 2) tc::cp_async_wait<2>();
    else if (n == 1) tc::cp_async_wait<1>();
    else tc::cp_async_wait<0>();
  }
}

__device__ __forceinline__ void copy_weights16(uint32_t dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16u : 0u) : "memory");
}

__device__ __forceinline__ void halves(uint32_t q, uint32_t& a, uint32_t& b) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(a), "=r"(b)
      : "r"(q));
}

// 16 bytes of k of rows g and g + 8 by those of NC x 8 tokens.
template <bool EIGHT, int NC>
__device__ __forceinline__ void multiply(const uint4& w0, const uint4& w1, const uint4 (&x)[NC], float (&acc)[NC][4]) {
  const uint32_t a[4] = {w0.x, w0.y, w0.z, w0.w}, b[4] = {w1.x, w1.y, w1.z, w1.w};
  if (EIGHT) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a0, a1, a2, a3;
      halves(a[i], a0, a2);
      halves(b[i], a1, a3);
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        uint32_t b0, b1;
        halves(i == 0 ? x[n].x : i == 1 ? x[n].y : i == 2 ? x[n].z : x[n].w, b0, b1);
        mma_f16_16816(acc[n], a0, a1, a2, a3, b0, b1);
      }
    }
  } else {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      mma_bf16_16816(acc[n], a[0], b[0], a[1], b[1], x[n].x, x[n].y);
      mma_bf16_16816(acc[n], a[2], b[2], a[3], b[3], x[n].z, x[n].w);
    }
  }
}

template <bool EIGHT, bool GLU, int NC>
__global__ void __launch_bounds__(kWarps * 32, 1) linear_stream_kernel(const __grid_constant__ StreamArgs a) {
  constexpr int TOK = 8 * NC, FEATURES = GLU ? 8 : 16;   // of a tile
  extern __shared__ __align__(16) uint8_t smem[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
  const Cut& cut = a.cut;
  float* red = reinterpret_cast<float*>(smem);                   // over the rings, once they are done with
  uint8_t* xs = smem + warps * cut.depth * kSlotBytes;           // [token][k of the phase | pad]
  const uint32_t ring = tc::smem_u32(smem) + warp * cut.depth * kSlotBytes;
  const int f0 = (int)((long long)a.n * blockIdx.x / gridDim.x), f1 = (int)((long long)a.n * (blockIdx.x + 1) / gridDim.x);
  const int tiles = (f1 - f0 + FEATURES - 1) / FEATURES;
  const int slot = warp / cut.ws, part = warp - slot * cut.ws;
  const int per_phase = cut.phase_steps / cut.ws, phases = (cut.steps + cut.phase_steps - 1) / cut.phase_steps;
  const int pitch = cut.phase_steps * kStepBytes + kXPad;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0u;

  int staged = -1;
  // Asks for a phase's x, ahead of the weights; whether it was not there.
  auto stage = [&](int phase) {
    if (phase == staged) return false;
    if (staged >= 0) __syncthreads();   // the last phase's x is done with
    staged = phase;
    const int k0 = phase * cut.phase_steps * kStepBytes, vecs = cut.phase_steps * kStepBytes / 16, live = (a.row - k0) / 16;
    const int each = max(1, warps / a.T), rows = warps / each;   // warps to a row; rows at one time
    for (int t = warp / each; t < a.T && warp < rows * each; t += rows)
      for (int v = (warp % each) * 32 + lane; v < vecs; v += 32 * each)
        tc::cp_async16(tc::smem_u32(xs + t * pitch + 16 * v), a.x + (size_t)t * a.row + k0 + (v < live ? 16 * v : 0), v < live ? 16u : 0u);
    tc::cp_async_commit();
    return true;
  };

  // this lane copies piece lane % 8 of rows lane / 8, + 4, + 8, + 12 of a step; they lie at piece
  // ^ 4 (row & 1), so that the reads of 8 lanes, of two rows, meet no bank twice
  const int crow = lane >> 3, piece = lane & 7;
  const uint32_t to = ring + crow * kStepBytes + ((piece ^ ((crow & 1) << 2)) << 4);
  const uint32_t odd = (gq & 1) << 2;
  const uint8_t* mine = smem + warp * cut.depth * kSlotBytes + gq * kStepBytes;

  for (int base = 0; base < tiles; base += cut.slots) {
    const int first = f0 + (base + slot) * FEATURES;
    const bool busy = slot < cut.slots && first < f1;
    const uint8_t* from[4];
    bool live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = crow + 4 * i, f = first + (GLU ? r & 7 : r);
      live[i] = busy && f < f1;
      from[i] = a.w + (live[i] ? ((size_t)f + (GLU && (r & 8) ? a.n : 0)) * a.row : 0) + 16 * piece;
    }
    float acc[NC][4] = {};
    for (int phase = 0; phase < phases; ++phase) {
      const int st0 = phase * cut.phase_steps + part * per_phase;
      const int run = busy ? min(per_phase, cut.steps - st0) : 0;   // may be negative
      int off = st0 * kStepBytes, in = 0, out = 0;
      auto copy = [&]() {
        const bool there = off + 16 * piece < a.row;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          copy_weights16(to + in + i * 4 * kStepBytes, from[i] + (there && live[i] ? off : 0), there && live[i]);
        off += kStepBytes;
        if ((in += kSlotBytes) == cut.depth * kSlotBytes) in = 0;
      };
      const bool fresh = stage(phase);
      for (int s = 0; s < cut.depth; ++s) {
        if (s < run) copy();
        tc::cp_async_commit();
      }
      if (fresh) {
        copies_wait(cut.depth);
        __syncthreads();
      }
      // columns without a token take the last one's: they are not stored
      const uint8_t* x[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) x[n] = xs + min(8 * n + gq, a.T - 1) * pitch + part * per_phase * kStepBytes + 16 * c;
      for (int i = 0; i < run; ++i) {
        copies_wait(cut.depth - 1);
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 q[NC];
#pragma unroll
          for (int n = 0; n < NC; ++n) q[n] = *reinterpret_cast<const uint4*>(x[n] + 64 * h);
          const uint8_t* at = mine + out + (((c + 4 * h) ^ odd) << 4);
          const uint4 w0 = *reinterpret_cast<const uint4*>(at), w1 = *reinterpret_cast<const uint4*>(at + 8 * kStepBytes);
          multiply<EIGHT, NC>(w0, w1, q, acc);
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) x[n] += kStepBytes;
        if ((out += kSlotBytes) == cut.depth * kSlotBytes) out = 0;
        __syncwarp();   // the slot is read
        if (i + cut.depth < run) copy();
        tc::cp_async_commit();
      }
    }
    tc::cp_async_wait_all();
    __syncthreads();   // every ring is done with
    // partial sums: rows gq and gq + 8, columns 8 n + 2 c and + 1
    float* p = red + warp * TOK * kRedPitch;
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) p[(8 * n + 2 * c + (e & 1)) * kRedPitch + gq + 8 * (e >> 1)] = acc[n][e];
    __syncthreads();
    for (int e = threadIdx.x; e < cut.slots * a.T * FEATURES; e += blockDim.x) {
      const int r = e & (FEATURES - 1), st = e / FEATURES, s = st / a.T, t = st - s * a.T;
      const int f = f0 + (base + s) * FEATURES + r;
      if (f >= f1) continue;
      const float* q = red + (s * cut.ws * TOK + t) * kRedPitch + r;
      float v = 0.f, u = 0.f;
      for (int i = 0; i < cut.ws; ++i) {
        v += q[i * TOK * kRedPitch];
        if (GLU) u += q[i * TOK * kRedPitch + 8];
      }
      if (EIGHT) {
        const float by = a.epi.x_scale[t];
        v = v * by * a.epi.w_scale[f];
        if (GLU) u = u * by * a.epi.w_scale[a.n + f];
      }
      if (a.epi.bias) {
        v += bf16_to_f32(a.epi.bias[f]);
        if (GLU) u += bf16_to_f32(a.epi.bias[a.n + f]);
      }
      const size_t at = (size_t)t * a.n + f;
      if (GLU) {
        v = glu_value(a.epi.gated, v, u);
      } else {
        if (a.epi.pre) a.epi.pre[at] = f32_to_bf16(v);
        F2 one[1] = {f2(v)};
        linear_values(a.epi.act, one);
        split(one[0], v, u);
      }
      if (a.epi.residual) v += bf16_to_f32(a.epi.residual[at]);
      a.y[at] = f32_to_bf16(v);
    }
    __syncthreads();
  }
  pdl_trigger();
}

// ---------------------------------------------------------------- host
template <bool EIGHT, bool GLU, int NC>
cudaError_t launch(StreamArgs& a, cudaStream_t s) {
  constexpr int TOK = 8 * NC, FEATURES = GLU ? 8 : 16;
  const int ctas = std::min(sm_count(), (a.n + 3) / 4), share = (a.n + ctas - 1) / ctas;   // four features at least
  int smem;
  a.cut = stream_cut(a.T, a.row, share, FEATURES, TOK, smem);
  const cudaError_t e = allow_smem<linear_stream_kernel<EIGHT, GLU, NC>>(kSpace);
  if (e != cudaSuccess) return e;
  return launch_pdl(linear_stream_kernel<EIGHT, GLU, NC>, dim3(ctas), dim3(a.cut.slots * a.cut.ws * 32), smem, s, a);
}

template <bool EIGHT>
cudaError_t launch_format(StreamArgs& a, cudaStream_t s) {
  if (a.T > 8) return a.epi.glu ? launch<EIGHT, true, 2>(a, s) : launch<EIGHT, false, 2>(a, s);
  return a.epi.glu ? launch<EIGHT, true, 1>(a, s) : launch<EIGHT, false, 1>(a, s);
}

}  // namespace

// Up to 8 tokens always.  Up to 16, where the MMAs' second half of columns and x cost more,
// unless the weights are many or x has to come in phases (16 tokens here, and 17 in tiles: 4096 x
// 12288 gated, 8 bits 23.6 us and 20.0, bf16 37.4 and 34.1; 8192 x 1024 bf16 11.6 and 8.6; 4096 x
// 4096 bf16 9.0 and 12.5; 2880 x 2880 7.2 and 8.5).
bool linear_streams(const LinearShape& l, int T, bool glu) {
  const long long row = l.eight ? l.n_in : 2LL * l.n_in;
  if (T <= 8) return true;
  return T <= 16 && row * l.n_out * (glu ? 2 : 1) < (64LL << 20) && T * (row + kXPad) + 2 * kWarps * kSlotBytes <= kSpace;
}

cudaError_t launch_linear_stream(const LinearShape& l, const void* x, int T, const void* w, uint16_t* y, const LinearEpi& epi,
                                 uint32_t* status, cudaStream_t s) {
  StreamArgs a{};
  a.w = static_cast<const uint8_t*>(w);
  a.x = static_cast<const uint8_t*>(x);
  a.n = l.n_out;
  a.T = T;
  a.row = l.eight ? l.n_in : 2 * l.n_in;
  a.epi = epi;
  a.y = y;
  a.status = status;
  return l.eight ? launch_format<true>(a, s) : launch_format<false>(a, s);
}

}  // namespace moe
