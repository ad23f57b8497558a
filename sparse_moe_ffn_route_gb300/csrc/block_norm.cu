// The norms either side of a block with its gate and residual scale, in one pass over the
// rows: y = residual_scale x + c n(z) post_w, a = n(y) pre_w (see moe_block.h), and the
// gradients of the same.
//
// Bound by memory: forward reads x, z and writes y, a (8 bytes per element), backward
// reads x, z, dy, da and writes dx, dz (12 bytes).  One CTA works on one row at a time, 8
// elements (one 16-byte vector) per thread and step, so every tensor passes memory once.
// Each thread copies its own vectors of the next rows into shared memory ahead of time
// (cp.async: the rows' latency stays off the chain of sums, and needs no registers and no
// barrier, since a thread reads only what it copied).  The row sums cross the CTA through
// shared memory (forward: sum z^2, then sum y^2; backward: sum z^2, then sum y^2 and
// sum da pre_w y together, then sum D post_w z, from which both dgate and dz follow).
// The sums of y are taken from y itself and not expanded into sums of x and z, which
// would cost one exchange less but cancel where the branch takes back the residual.
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
// N * kMaxWarps floats; a row's sums use buffers of their own, and rows alternate between
// two sets (a warp a row ahead waits at that row's first barrier for the last reader).
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
    float s = 0.f;
    for (int w = 0; w < nw; w += 4) {   // slots past the last warp hold zeros
      const float4 q = *reinterpret_cast<const float4*>(buf + i * kMaxWarps + w);
      s += (q.x + q.y) + (q.z + q.w);
    }
    v[i] = s;
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

__device__ __forceinline__ uint4 ld8(const uint16_t* p, int at) { return *reinterpret_cast<const uint4*>(p + at); }

// This thread's vectors of a row, and the copies of the rows ahead: DEPTH slots of NA arrays.
// Vector i holds elements 8 (threadIdx.x + i blockDim.x) .. + 7 of the row.
template <int NA, int V, int DEPTH>
struct Ahead {
  uint32_t base;            // shared address of this thread's first vector
  const uint4* mine;
  int n;                    // threads
  __device__ __forceinline__ Ahead(uint4* smem)
      : base((uint32_t)__cvta_generic_to_shared(smem + threadIdx.x)), mine(smem + threadIdx.x), n((int)blockDim.x) {}
  __device__ __forceinline__ int elem(int i) const { return 8 * ((int)threadIdx.x + i * n); }
  // starts the copies of row t (none past the last row or for a missing array)
  __device__ __forceinline__ void start(int slot, const uint16_t* const (&p)[NA], int t, int T, int d) const {
    if (t < T) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (elem(i) < d) {
          const size_t off = (size_t)t * d + elem(i);
#pragma unroll
          for (int a = 0; a < NA; ++a)
            if (p[a])
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + 16u * (uint32_t)(((slot * NA + a) * V + i) * n)),
                           "l"(p[a] + off)
                           : "memory");
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
  __device__ __forceinline__ uint4 get(int slot, int a, int i) const { return mine[((slot * NA + a) * V + i) * n]; }
};

// Z: there is a branch; POST: with a norm; PRE: with the next block's norm (a).
template <int V, int DEPTH, bool Z, bool POST, bool PRE>
__global__ void __launch_bounds__(kMaxWarps * 32) block_norm_fwd_kernel(const __grid_constant__ NormArgs g) {
  extern __shared__ uint4 rows[];
  __shared__ __align__(16) float buf[2][2][kMaxWarps];
  for (int i = threadIdx.x; i < 4 * kMaxWarps; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
  pdl_wait();
  __syncthreads();
  const int d = g.d, T = g.T;
  const float inv_d = 1.f / (float)d, eps = g.eps, rs = g.rs;
  const Ahead<2, V, DEPTH> ahead(rows);
  const uint16_t* const src[2] = {g.x, Z ? g.z : nullptr};
#pragma unroll
  for (int s = 0; s < DEPTH; ++s) ahead.start(s, src, blockIdx.x + s * gridDim.x, T, d);
  int slot = 0, par = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x, par ^= 1) {
    const size_t base = (size_t)t * d;
    float y[V][8];
    ahead.wait();
    if (Z) {
      float c = g.bs;
      if (g.gate) c *= 1.f / (1.f + expf(-g.gate[t]));
      if (POST) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (ahead.elem(i) < d) {
            float z[8];
            unpack8(ahead.get(slot, 1, i), z);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss[0] += z[j] * z[j];
          }
        cta_sum(ss, buf[par][0]);
        c *= 1.f / sqrtf(ss[0] * inv_d + eps);
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d) {
          float z[8];
          unpack8(ahead.get(slot, 0, i), y[i]);
          unpack8(ahead.get(slot, 1, i), z);
          if (POST) {
            float w[8];
            unpack8(ld8(g.post_w, ahead.elem(i)), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] *= w[j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) y[i][j] = rs * y[i][j] + c * z[j];
          *reinterpret_cast<uint4*>(g.y + base + ahead.elem(i)) = pack8(y[i]);
        }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d) unpack8(ahead.get(slot, 0, i), y[i]);
    }
    ahead.start(slot, src, t + DEPTH * (int)gridDim.x, T, d);
    if (++slot == DEPTH) slot = 0;
    if (PRE) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d)
#pragma unroll
          for (int j = 0; j < 8; ++j) ss[0] += y[i][j] * y[i][j];
      cta_sum(ss, buf[par][1]);
      const float r = 1.f / sqrtf(ss[0] * inv_d + eps);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d) {
          float w[8];
          unpack8(ld8(g.pre_w, ahead.elem(i)), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[i][j] *= r * w[j];
          *reinterpret_cast<uint4*>(g.a + base + ahead.elem(i)) = pack8(y[i]);
        }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  pdl_trigger();
}

// Z, POST: as above; DA: da is given (else a's gradient is zero).
template <int V, int DEPTH, bool Z, bool POST, bool DA>
__global__ void __launch_bounds__(kMaxWarps * 32) block_norm_bwd_kernel(const __grid_constant__ NormArgs g) {
  extern __shared__ uint4 rows[];
  __shared__ __align__(16) float buf[2][4][kMaxWarps];
  for (int i = threadIdx.x; i < 8 * kMaxWarps; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
  pdl_wait();
  __syncthreads();
  const int d = g.d, T = g.T;
  const float inv_d = 1.f / (float)d, eps = g.eps, rs = Z ? g.rs : 1.f;
  const bool has_dy = g.dy != nullptr;
  float dpost[V][8] = {}, dpre[V][8] = {};
  const Ahead<4, V, DEPTH> ahead(rows);
  const uint16_t* const src[4] = {DA ? g.x : nullptr, Z ? g.z : nullptr, g.dy, DA ? g.da : nullptr};
#pragma unroll
  for (int s = 0; s < DEPTH; ++s) ahead.start(s, src, blockIdx.x + s * gridDim.x, T, d);
  int slot = 0, par = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x, par ^= 1) {
    const size_t base = (size_t)t * d;
    float y[V][8], D[V][8];
    float c = g.bs, s = 1.f, rz = 1.f;
    if (g.gate) {
      s = 1.f / (1.f + expf(-g.gate[t]));
      c *= s;
    }
    ahead.wait();
    if (POST) {
      float sz[1] = {0.f};
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d) {
          float z[8];
          unpack8(ahead.get(slot, 1, i), z);
#pragma unroll
          for (int j = 0; j < 8; ++j) sz[0] += z[j] * z[j];
        }
      cta_sum(sz, buf[par][0]);
      rz = 1.f / sqrtf(sz[0] * inv_d + eps);
    }
    const float cr = c * rz;
    float ry = 0.f, k = 0.f;
    if (DA) {
      float sy[2] = {0.f, 0.f};   // sum y^2, sum da pre_w y
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d) {
          float w[8], v[8];
          unpack8(ahead.get(slot, 0, i), y[i]);
          if (Z) {
            unpack8(ahead.get(slot, 1, i), v);
            if (POST) {
              unpack8(ld8(g.post_w, ahead.elem(i)), w);
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) y[i][j] = rs * y[i][j] + cr * v[j];
          }
          unpack8(ahead.get(slot, 3, i), v);
          unpack8(ld8(g.pre_w, ahead.elem(i)), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            D[i][j] = v[j] * w[j];   // the gradient through a, before its row terms
            sy[0] += y[i][j] * y[i][j];
            sy[1] += D[i][j] * y[i][j];
          }
        }
      cta_sum(sy, buf[par][1]);
      ry = 1.f / sqrtf(sy[0] * inv_d + eps);
      k = ry * ry * sy[1] * inv_d;
    }
    float sw[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ahead.elem(i) < d) {
        float v[8];
        if (DA) {
          unpack8(ahead.get(slot, 3, i), v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            D[i][j] = ry * (D[i][j] - y[i][j] * k);
            dpre[i][j] += v[j] * (y[i][j] * ry);
          }
          if (has_dy) {
            unpack8(ahead.get(slot, 2, i), v);
#pragma unroll
            for (int j = 0; j < 8; ++j) D[i][j] += v[j];
          }
        } else {
          unpack8(ahead.get(slot, 2, i), D[i]);
        }
        if (g.dx) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = rs * D[i][j];
          *reinterpret_cast<uint4*>(g.dx + base + ahead.elem(i)) = pack8(v);
        }
        if (Z) {
          unpack8(ahead.get(slot, 1, i), v);
          if (POST) {
            float w[8];
            unpack8(ld8(g.post_w, ahead.elem(i)), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              dpost[i][j] += cr * (D[i][j] * v[j]);
              D[i][j] *= w[j];
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) sw[0] += D[i][j] * v[j];
        }
      }
    if (Z && (g.dz || g.dgate)) {
      float kz = 0.f;
      if (POST || g.dgate) {
        cta_sum(sw, buf[par][3]);
        if (POST) kz = rz * rz * sw[0] * inv_d;
        if (g.dgate && threadIdx.x == 0) g.dgate[t] = g.bs * s * (1.f - s) * rz * sw[0];
      }
      if (g.dz) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (ahead.elem(i) < d) {
            if (POST) {
              float v[8];
              unpack8(ahead.get(slot, 1, i), v);
#pragma unroll
              for (int j = 0; j < 8; ++j) D[i][j] = D[i][j] - v[j] * kz;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) D[i][j] *= cr;
            *reinterpret_cast<uint4*>(g.dz + base + ahead.elem(i)) = pack8(D[i]);
          }
      }
    }
    ahead.start(slot, src, t + DEPTH * (int)gridDim.x, T, d);
    if (++slot == DEPTH) slot = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (g.part) {
    float* p = g.part + (size_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ahead.elem(i) < d) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float(&v)[8] = h ? dpre[i] : dpost[i];
          float4* o = reinterpret_cast<float4*>(p + (size_t)h * d + ahead.elem(i));
          o[0] = make_float4(v[0], v[1], v[2], v[3]);
          o[1] = make_float4(v[4], v[5], v[6], v[7]);
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

// The launch shape of a row of d: threads, vectors per thread (1 up to 2048 elements, 2 up
// to 8192, else 4), rows ahead, CTAs.  Rows ahead as deep as leaves an SM several CTAs.
struct Shape {
  int v, threads, smem, ctas;
};

template <int NA, int V, int DEPTH, typename K>
Shape shape_of(K kernel, int d, int T) {
  Shape h;
  h.v = V;
  h.threads = ((d / 8 + V - 1) / V + 31) / 32 * 32;
  h.smem = DEPTH * NA * V * h.threads * 16;
  if (h.smem > 46 * 1024)   // with the static shared memory, past the default 48 KiB
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, h.smem);
  const int sms = sm_count();
  int per_sm = 1;
  if (T > sms &&
      (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, h.threads, h.smem) != cudaSuccess || per_sm < 1))
    per_sm = 1;
  const int most = sms * per_sm;
  h.ctas = T < most ? T : most;
  return h;
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

template <int V, int DEPTH, bool Z, bool POST, bool PRE>
cudaError_t run_fwd(const NormArgs& g, cudaStream_t s) {
  auto* kernel = block_norm_fwd_kernel<V, DEPTH, Z, POST, PRE>;
  const Shape h = shape_of<2, V, DEPTH>(kernel, g.d, g.T);
  return launch_pdl(kernel, dim3(h.ctas), dim3(h.threads), h.smem, s, g);
}

template <int V, int DEPTH>
cudaError_t pick_fwd(const NormArgs& g, cudaStream_t s) {
  if (!g.z) return run_fwd<V, DEPTH, false, false, true>(g, s);
  if (g.post_w) return g.pre_w ? run_fwd<V, DEPTH, true, true, true>(g, s) : run_fwd<V, DEPTH, true, true, false>(g, s);
  return g.pre_w ? run_fwd<V, DEPTH, true, false, true>(g, s) : run_fwd<V, DEPTH, true, false, false>(g, s);
}

// The backward kernel's partial sums are one row per CTA; their number must not depend on
// more than d and T, since the caller sized the workspace by it.
constexpr int kBwdPerSm = 4;

template <int V, int DEPTH, bool Z, bool POST, bool DA>
cudaError_t run_bwd(const NormArgs& g, int* ctas, cudaStream_t s) {
  auto* kernel = block_norm_bwd_kernel<V, DEPTH, Z, POST, DA>;
  const Shape h = shape_of<4, V, DEPTH>(kernel, g.d, g.T);
  *ctas = h.ctas < *ctas ? h.ctas : *ctas;
  return launch_pdl(kernel, dim3(*ctas), dim3(h.threads), h.smem, s, g);
}

template <int V, int DEPTH>
cudaError_t pick_bwd(const NormArgs& g, int* ctas, cudaStream_t s) {
  if (!g.z) return run_bwd<V, DEPTH, false, false, true>(g, ctas, s);
  if (g.post_w)
    return g.da ? run_bwd<V, DEPTH, true, true, true>(g, ctas, s) : run_bwd<V, DEPTH, true, true, false>(g, ctas, s);
  return g.da ? run_bwd<V, DEPTH, true, false, true>(g, ctas, s) : run_bwd<V, DEPTH, true, false, false>(g, ctas, s);
}

}  // namespace

cudaError_t launch_block_norm_fwd(const moe_norm_cfg_t& c, const moe_norm_inputs_t& in, int T, uint16_t* y,
                                  uint16_t* a, cudaStream_t s) {
  NormArgs g = make_args(c, in, T);
  g.y = y;
  g.a = a;
  if (g.d <= 2048) return pick_fwd<1, 3>(g, s);
  if (g.d <= 8192) return pick_fwd<2, 2>(g, s);
  return pick_fwd<4, 1>(g, s);
}

int block_norm_parts(int d, int T) {
  (void)d;
  const int most = kBwdPerSm * sm_count();
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
  int n = block_norm_parts(g.d, T);
  const cudaError_t e = g.d <= 2048   ? pick_bwd<1, 3>(g, &n, s)
                        : g.d <= 8192 ? pick_bwd<2, 2>(g, &n, s)
                                      : pick_bwd<4, 1>(g, &n, s);
  if (e != cudaSuccess || !g.part) return e;
  return launch_pdl(block_norm_reduce_kernel, dim3((g.d + 31) / 32, 2), dim3(256), 0, s, static_cast<const float*>(parts),
                    n, g.d, o.dpost_w, o.dpre_w);
}

}  // namespace moe
