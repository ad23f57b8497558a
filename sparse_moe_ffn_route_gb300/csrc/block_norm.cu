// The norms either side of a block with its gate and residual scale, in one pass over the
// rows: y = residual_scale x + c n(z) post_w, a = n(y) pre_w (see moe_block.h), and the
// gradients of the same.
//
// Bound by memory: forward reads x, z and writes y, a (8 bytes per element), backward
// reads x, z, dy, da and writes dx, dz (12 bytes).  One CTA holds one row at a time in
// registers, 8 elements (one 16-byte vector) per thread and step, so every tensor passes
// memory once; the row sums cross the CTA through shared memory (forward: sum z^2, then
// sum y^2; backward: sum z^2, then sum y^2 and sum da pre_w y together, then
// sum D post_w z, from which both dgate and dz follow).
//
// Backward: with rz = 1 / sqrt(mean z^2 + eps), ry alike for y, c the branch's factor,
//   D  = dy + ry (da pre_w - y ry^2 mean(da pre_w y))        (gradient of y)
//   dx = residual_scale D;   W = D post_w;   S = sum W z
//   dgate = branch_scale s (1 - s) rz S;   dz = c rz (W - z rz^2 S / d)
//   dpost_w += c D z rz;   dpre_w += da y ry
// A CTA keeps its columns' weight gradients in registers over all its rows and writes one
// row of partial sums; a second kernel adds the partial rows in order.
#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 16;

// Sum of N values over the CTA, in every thread, in a fixed order.  `buf` holds
// N * kMaxWarps floats; consecutive calls alternate between two buffers.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * kMaxWarps + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < nw; ++w) v[i] += buf[i * kMaxWarps + w];
  }
}

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(u[i]);
    v[2 * i + 1] = bf16_hi(u[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

struct NormArgs {
  const uint16_t *x, *z, *post_w, *pre_w;
  const float* gate;
  int T, d;
  float eps, rs, bs;
  // forward
  uint16_t *y, *a;
  // backward
  const uint16_t *dy, *da;
  uint16_t *dx, *dz;
  float *dgate, *part;   // part: [gridDim.x][2][d] (dpost_w, dpre_w), or null
};

__device__ __forceinline__ uint4 ld8(const uint16_t* p, size_t at) { return *reinterpret_cast<const uint4*>(p + at); }

// V vectors of 8 elements per thread: element 8 (threadIdx.x + i blockDim.x).
template <int V>
__global__ void __launch_bounds__(kMaxWarps * 32) block_norm_fwd_kernel(const NormArgs g) {
  __shared__ float buf[2][kMaxWarps];
  pdl_wait();
  const float inv_d = 1.f / (float)g.d;
  for (int t = blockIdx.x; t < g.T; t += gridDim.x) {
    const size_t base = (size_t)t * g.d;
    float y[V][8];
    if (g.z) {
      float z[V][8], ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = 8 * (threadIdx.x + i * blockDim.x);
        uint4 xq = make_uint4(0u, 0u, 0u, 0u), zq = xq;
        if (e < g.d) {
          xq = ld8(g.x, base + e);
          zq = ld8(g.z, base + e);
        }
        unpack8(xq, y[i]);
        unpack8(zq, z[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] += z[i][j] * z[i][j];
      }
      float c = g.bs;
      if (g.gate) c *= 1.f / (1.f + expf(-g.gate[t]));
      if (g.post_w) {
        cta_sum(ss, buf[0]);
        c *= 1.f / sqrtf(ss[0] * inv_d + g.eps);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = 8 * (threadIdx.x + i * blockDim.x);
        if (e < g.d) {
          float w[8];
          if (g.post_w) unpack8(ld8(g.post_w, e), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[i][j] = g.rs * y[i][j] + c * (g.post_w ? z[i][j] * w[j] : z[i][j]);
          *reinterpret_cast<uint4*>(g.y + base + e) = pack8(y[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = 8 * (threadIdx.x + i * blockDim.x);
        unpack8(e < g.d ? ld8(g.x, base + e) : make_uint4(0u, 0u, 0u, 0u), y[i]);
      }
    }
    if (g.pre_w) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] += y[i][j] * y[i][j];
      cta_sum(ss, buf[1]);
      const float r = 1.f / sqrtf(ss[0] * inv_d + g.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = 8 * (threadIdx.x + i * blockDim.x);
        if (e < g.d) {
          float w[8];
          unpack8(ld8(g.pre_w, e), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[i][j] *= r * w[j];
          *reinterpret_cast<uint4*>(g.a + base + e) = pack8(y[i]);
        }
      }
    }
    // the buffers of this row's sums are not rewritten before every thread has read them:
    // each sum's own barrier lies between (with one sum a row, this one)
    if (!(g.z && g.post_w && g.pre_w)) __syncthreads();
  }
  pdl_trigger();
}

template <int V>
__global__ void __launch_bounds__(kMaxWarps * 32) block_norm_bwd_kernel(const NormArgs g) {
  __shared__ float buf[3][2 * kMaxWarps];
  pdl_wait();
  const float inv_d = 1.f / (float)g.d;
  float dpost[V][8] = {}, dpre[V][8] = {};
  for (int t = blockIdx.x; t < g.T; t += gridDim.x) {
    const size_t base = (size_t)t * g.d;
    float y[V][8], z[V][8], D[V][8], da[V][8];
    float sz[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (threadIdx.x + i * blockDim.x);
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      const bool in = e < g.d;
      const uint4 xq = in ? ld8(g.x, base + e) : zero;
      const uint4 zq = in && g.z ? ld8(g.z, base + e) : zero;
      const uint4 dq = in && g.dy ? ld8(g.dy, base + e) : zero;
      const uint4 aq = in && g.da ? ld8(g.da, base + e) : zero;
      unpack8(xq, y[i]);
      unpack8(zq, z[i]);
      unpack8(dq, D[i]);
      unpack8(aq, da[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sz[0] += z[i][j] * z[i][j];
    }
    float c = g.bs, s = 1.f, rz = 1.f;
    if (g.gate) {
      s = 1.f / (1.f + expf(-g.gate[t]));
      c *= s;
    }
    if (g.post_w) {
      cta_sum(sz, buf[0]);
      rz = 1.f / sqrtf(sz[0] * inv_d + g.eps);
    }
    float sy[2] = {0.f, 0.f};   // sum y^2, sum da pre_w y
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (threadIdx.x + i * blockDim.x);
      if (e < g.d) {
        float w[8];
        if (g.z) {
          if (g.post_w) unpack8(ld8(g.post_w, e), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[i][j] = g.rs * y[i][j] + c * rz * (g.post_w ? z[i][j] * w[j] : z[i][j]);
        }
        if (g.da) {
          unpack8(ld8(g.pre_w, e), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sy[0] += y[i][j] * y[i][j];
            sy[1] += da[i][j] * w[j] * y[i][j];
          }
        }
      }
    }
    float ry = 0.f, k = 0.f;
    if (g.da) {
      cta_sum(sy, buf[1]);
      ry = 1.f / sqrtf(sy[0] * inv_d + g.eps);
      k = ry * ry * sy[1] * inv_d;
    }
    float sw[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (threadIdx.x + i * blockDim.x);
      if (e < g.d) {
        float w[8];
        if (g.da) {
          unpack8(ld8(g.pre_w, e), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            D[i][j] += ry * (da[i][j] * w[j] - y[i][j] * k);
            dpre[i][j] += da[i][j] * y[i][j] * ry;
          }
        }
        if (g.dx) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = (g.z ? g.rs : 1.f) * D[i][j];
          *reinterpret_cast<uint4*>(g.dx + base + e) = pack8(o);
        }
        if (g.z) {
          if (g.post_w) unpack8(ld8(g.post_w, e), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (g.post_w) {
              dpost[i][j] += c * D[i][j] * z[i][j] * rz;
              D[i][j] *= w[j];
            }
            sw[0] += D[i][j] * z[i][j];
          }
        }
      }
    }
    if (g.z && (g.dz || g.dgate)) {
      float kz = 0.f;
      if (g.post_w || g.dgate) {
        cta_sum(sw, buf[2]);
        if (g.post_w) kz = rz * rz * sw[0] * inv_d;
        if (g.dgate && threadIdx.x == 0) g.dgate[t] = g.bs * s * (1.f - s) * rz * sw[0];
      }
      if (g.dz) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = 8 * (threadIdx.x + i * blockDim.x);
          if (e < g.d) {
#pragma unroll
            for (int j = 0; j < 8; ++j) D[i][j] = c * rz * (D[i][j] - z[i][j] * kz);
            *reinterpret_cast<uint4*>(g.dz + base + e) = pack8(D[i]);
          }
        }
      }
    }
    __syncthreads();   // the sums' buffers are free again
  }
  if (g.part) {
    float* p = g.part + (size_t)blockIdx.x * 2 * g.d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (threadIdx.x + i * blockDim.x);
      if (e < g.d) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float(&v)[8] = h ? dpre[i] : dpost[i];
          float4* o = reinterpret_cast<float4*>(p + (size_t)h * g.d + e);
          o[0] = make_float4(v[0], v[1], v[2], v[3]);
          o[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
  }
  pdl_trigger();
}

// Column sums of the partial rows: 32 columns per CTA, 8 rows of threads that take every
// eighth partial row, added in order.
__global__ void __launch_bounds__(256) block_norm_reduce_kernel(const float* part, int parts, int d, float* dpost,
                                                                float* dpre) {
  __shared__ float s[8][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, col = blockIdx.x * 32 + lane, h = blockIdx.y;
  float* out = h ? dpre : dpost;
  if (!out) return;
  float v = 0.f;
  if (col < d)
    for (int i = r; i < parts; i += 8) v += part[((size_t)i * 2 + h) * d + col];
  s[r][lane] = v;
  __syncthreads();
  if (r == 0 && col < d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    out[col] = v;
  }
}

// Threads and vectors per thread of a row of d: up to 512 threads, V 1, 2 or 4.
int pick_v(int d, int* threads) {
  const int vecs = d / 8;
  int v = 1;
  while (v < 4 && vecs > v * 256) v <<= 1;
  *threads = ((vecs + v - 1) / v + 31) / 32 * 32;
  return v;
}

NormArgs make_args(const moe_norm_cfg_t& c, const moe_norm_inputs_t& in, int T) {
  NormArgs g{};
  g.x = static_cast<const uint16_t*>(in.x);
  g.z = static_cast<const uint16_t*>(in.branch);
  g.post_w = static_cast<const uint16_t*>(in.post_w);
  g.pre_w = static_cast<const uint16_t*>(in.pre_w);
  g.gate = in.gate;
  g.T = T;
  g.d = c.d_model;
  g.eps = c.eps;
  g.rs = c.residual_scale;
  g.bs = c.branch_scale;
  return g;
}

}  // namespace

cudaError_t launch_block_norm_fwd(const moe_norm_cfg_t& c, const moe_norm_inputs_t& in, int T, uint16_t* y,
                                  uint16_t* a, cudaStream_t s) {
  NormArgs g = make_args(c, in, T);
  g.y = y;
  g.a = a;
  int threads;
  const int v = pick_v(g.d, &threads);
  const int most = sm_count() * (2048 / threads);
  const dim3 grid(T < most ? T : most), block(threads);
  if (v == 1) return launch_pdl(block_norm_fwd_kernel<1>, grid, block, 0, s, g);
  if (v == 2) return launch_pdl(block_norm_fwd_kernel<2>, grid, block, 0, s, g);
  return launch_pdl(block_norm_fwd_kernel<4>, grid, block, 0, s, g);
}

int block_norm_parts(int d, int T) {
  int threads;
  pick_v(d, &threads);
  const int most = sm_count() * (1024 / threads > 1 ? 1024 / threads : 1);
  return T < most ? T : most;
}

cudaError_t launch_block_norm_bwd(const moe_norm_cfg_t& c, const moe_norm_inputs_t& in, int T, const uint16_t* dy,
                                  const uint16_t* da, const moe_norm_grads_t& o, float* parts, cudaStream_t s) {
  NormArgs g = make_args(c, in, T);
  g.dy = dy;
  g.da = da;
  g.dx = static_cast<uint16_t*>(o.dx);
  g.dz = static_cast<uint16_t*>(o.dbranch);
  g.dgate = o.dgate;
  g.part = o.dpost_w || o.dpre_w ? parts : nullptr;
  int threads;
  const int v = pick_v(g.d, &threads);
  const int n = block_norm_parts(g.d, T);
  const dim3 grid(n), block(threads);
  cudaError_t e = v == 1   ? launch_pdl(block_norm_bwd_kernel<1>, grid, block, 0, s, g)
                  : v == 2 ? launch_pdl(block_norm_bwd_kernel<2>, grid, block, 0, s, g)
                           : launch_pdl(block_norm_bwd_kernel<4>, grid, block, 0, s, g);
  if (e != cudaSuccess || !g.part) return e;
  return launch_pdl(block_norm_reduce_kernel, dim3((g.d + 31) / 32, 2), dim3(256), 0, s, static_cast<const float*>(parts),
                    n, g.d, o.dpost_w, o.dpre_w);
}

}  // namespace moe
