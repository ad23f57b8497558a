// The norms either side of a block with its gate and residual scale, in one pass over the
// rows: y = residual_scale x + c n(z) post_w, a = n(y) pre_w (see moe_block.h), and the
// gradients of the same.
//
// Bound by memory: forward reads x, z and writes y, a (8 bytes per element), backward
// reads x, z, dy, da and writes dx, dz (12 bytes).  A group of threads (forward: a CTA)
// works on one row at a time, held in registers, so every tensor passes memory once.
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
//   dgate = branch_scale s (1 - s) rz S, s = sigmoid(gate);   dz = c rz (W - z rz^2 S / d)
//   dpost_w += c D z rz;   dpre_w += da y ry
// One CTA per SM holds several groups of threads, each on rows of its own (named barriers),
// with 16 elements per thread and row: the fixed work of a row (exchanges, roots) is paid
// by fewer warps than at 8 elements (4400 instructions per row of 2048 then, of which half
// were that).  The next row's sum z^2 shares the exchange of this row's S.  A thread keeps
// its columns' weight gradients in registers over all its rows; the groups add theirs up
// and the CTA writes one row of partial sums, which a second kernel adds in order.
//
// Measured: forward 8192 x 2880 29.7 us in the kernel, 33.3 a call (189 MB, 83% of a copy's
// rate); backward 8192 x 2048 47.7 us (201 MB, 4.2 TB/s), bound by issue: about 3500
// instructions a row.
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

// rsqrtf is 2 units in the last place off at most, sigmoid a few: far below what the sums
// that go in have lost, and what the rounding to bf16 of all that they scale loses after.
__device__ __forceinline__ float inv_rms(float sum, float inv_d, float eps) { return rsqrtf(sum * inv_d + eps); }
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }
// sigmoid(v) sigmoid(-v) = e / (1 + e)^2 with e = exp(-|v|): dgate is fp32, and 1 - sigmoid(v)
// would cancel for open gates (a thousandth off at 10, 0 from 17 on).
__device__ __forceinline__ float sigmoid_slope(float v) {
  const float e = expf(-fabsf(v)), r = __fdividef(1.f, 1.f + e);
  return e * r * r;
}

// Two fp32 values that one instruction works on (fma.rn.f32x2 and its kin): the kernels
// are near the issue rate, and this halves their arithmetic.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float both(F2 a) {
  float lo, hi;
  split(a, lo, hi);
  return lo + hi;
}

__device__ __forceinline__ void unpack8(const uint4& q, F2 (&v)[4]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2(bf16_lo(u[i]), bf16_hi(u[i]));
}

__device__ __forceinline__ uint4 pack8(const F2 (&v)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    split(v[i], lo, hi);
    u[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
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

// A thread's vectors of a row (vector i of thread tid of n: elements 8 (tid + i n) .. + 7) and
// the copies of the rows ahead: DEPTH slots of NA arrays.
template <int NA, int V, int DEPTH>
struct Ahead {
  uint32_t base;            // shared address of this thread's first vector
  const uint4* mine;
  int tid, n;
  __device__ __forceinline__ Ahead(uint4* smem, int tid_, int n_)
      : base((uint32_t)__cvta_generic_to_shared(smem + tid_)), mine(smem + tid_), tid(tid_), n(n_) {}
  __device__ __forceinline__ int elem(int i) const { return 8 * (tid + i * n); }
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
  // all but the last LEFT rows asked for are there
  template <int LEFT>
  __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
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
  const float inv_d = 1.f / (float)d, eps = g.eps;
  const F2 rs = f2(g.rs);
  const Ahead<2, V, DEPTH> ahead(rows, threadIdx.x, blockDim.x);
  const uint16_t* const src[2] = {g.x, Z ? g.z : nullptr};
#pragma unroll
  for (int s = 0; s < DEPTH; ++s) ahead.start(s, src, blockIdx.x + s * gridDim.x, T, d);
  int slot = 0, par = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x, par ^= 1) {
    const size_t base = (size_t)t * d;
    F2 y[V][4];
    ahead.template wait<DEPTH - 1>();
    if (Z) {
      float c = g.bs;
      if (g.gate) c *= sigmoid(g.gate[t]);
      if (POST) {
        F2 sum = f2(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (ahead.elem(i) < d) {
            F2 z[4];
            unpack8(ahead.get(slot, 1, i), z);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum = fma2(z[j], z[j], sum);
          }
        float ss[1] = {both(sum)};
        cta_sum(ss, buf[par][0]);
        c *= inv_rms(ss[0], inv_d, eps);
      }
      const F2 c2 = f2(c);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d) {
          F2 z[4];
          unpack8(ahead.get(slot, 0, i), y[i]);
          unpack8(ahead.get(slot, 1, i), z);
          if (POST) {
            F2 w[4];
            unpack8(ld8(g.post_w, ahead.elem(i)), w);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = mul2(z[j], w[j]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i][j] = fma2(c2, z[j], mul2(rs, y[i][j]));
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
      F2 sum = f2(0.f);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum = fma2(y[i][j], y[i][j], sum);
      float ss[1] = {both(sum)};
      cta_sum(ss, buf[par][1]);
      const F2 r = f2(inv_rms(ss[0], inv_d, eps));
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d) {
          F2 w[4];
          unpack8(ld8(g.pre_w, ahead.elem(i)), w);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i][j] = mul2(y[i][j], mul2(r, w[j]));
          *reinterpret_cast<uint4*>(g.a + base + ahead.elem(i)) = pack8(y[i]);
        }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  pdl_trigger();
}

// Sum of N values over a group of n threads (whole warps) in every thread, in a fixed order;
// `buf` and its turns as in cta_sum.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* buf, int tid, int n, int barrier) {
  const int warp = tid >> 5, lane = tid & 31, nw = n >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (nw == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * kMaxWarps + warp] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(n) : "memory");
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

// Threads of a CTA of the backward kernel, at most (768 with 80 registers each: 81 us instead
// of 53 at 8192 x 2048; rows ahead 3 instead of 2: 57 us).
constexpr int kBwdThreads = 512;

// The two weights in fp32 in shared memory: the halves of a vector of 8 apart, so that a
// warp's reads of 16 bytes per thread meet no bank twice.
struct Weights {
  float4* w;
  int n;      // vectors of 8
  __device__ __forceinline__ void fill(int which, const uint16_t* src) const {
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      F2 v[4];
      unpack8(ld8(src, 8 * i), v);
      F2* lo = reinterpret_cast<F2*>(w + (2 * which) * n + i);
      F2* hi = reinterpret_cast<F2*>(w + (2 * which + 1) * n + i);
      lo[0] = v[0];
      lo[1] = v[1];
      hi[0] = v[2];
      hi[1] = v[3];
    }
  }
  __device__ __forceinline__ void get(int which, int vec, F2 (&v)[4]) const {
    const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(w + (2 * which) * n + vec);
    const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(w + (2 * which + 1) * n + vec);
    v[0].v = lo.x;
    v[1].v = lo.y;
    v[2].v = hi.x;
    v[3].v = hi.y;
  }
};

// Z, POST: as above; DA: da is given (else a's gradient is zero).  gt: threads of a group.
template <int V, int DEPTH, bool Z, bool POST, bool DA>
__global__ void __launch_bounds__(kBwdThreads, 1)
block_norm_bwd_kernel(const __grid_constant__ NormArgs g, const int gt) {
  extern __shared__ uint4 rows[];
  // group, row parity, exchange: two values per warp of the group
  __shared__ __align__(16) float sums[kBwdThreads / 32][2][2][2 * kMaxWarps];
  constexpr bool kShared = V <= 2;   // the weights in shared memory, after the rows
  const Weights weights{reinterpret_cast<float4*>(rows + (size_t)blockDim.x * DEPTH * 4 * V), g.d / 8};
  const int group = threadIdx.x / gt, groups = blockDim.x / gt, tid = threadIdx.x - group * gt;
  for (int i = threadIdx.x; i < groups * 8 * kMaxWarps; i += blockDim.x) (&sums[0][0][0][0])[i] = 0.f;
  pdl_wait();
  if (kShared) {
    if (POST) weights.fill(0, g.post_w);
    if (DA) weights.fill(1, g.pre_w);
  }
  __syncthreads();
  const int d = g.d, T = g.T, stride = gridDim.x * groups;
  const float inv_d = 1.f / (float)d, eps = g.eps;
  const F2 rs = f2(Z ? g.rs : 1.f);
  const bool has_dy = g.dy != nullptr;
  F2 dpost[V][4], dpre[V][4];
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) dpost[i >> 2][i & 3] = dpre[i >> 2][i & 3] = f2(0.f);
  const Ahead<4, V, DEPTH> ahead(rows + (size_t)group * DEPTH * 4 * V * gt, tid, gt);
  const uint16_t* const src[4] = {DA ? g.x : nullptr, Z ? g.z : nullptr, g.dy, DA ? g.da : nullptr};
  int t = blockIdx.x + gridDim.x * group;
#pragma unroll
  for (int s = 0; s < DEPTH; ++s) ahead.start(s, src, t + s * stride, T, d);
  auto weight = [&](int which, int i, F2 (&w)[4]) {
    if (kShared) weights.get(which, ahead.elem(i) >> 3, w);
    else unpack8(ld8(which ? g.pre_w : g.post_w, ahead.elem(i)), w);
  };
  // sum z^2 of the row in `slot`
  auto sum_z = [&](int slot) {
    F2 sum = f2(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ahead.elem(i) < d) {
        F2 z[4];
        unpack8(ahead.get(slot, 1, i), z);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = fma2(z[j], z[j], sum);
      }
    return both(sum);
  };
  int slot = 0, par = 0;
  float gate = g.gate && t < T ? g.gate[t] : 0.f;
  float sz = 0.f;   // sum z^2 of the row
  if (t < T && Z) {
    ahead.template wait<DEPTH - 1>();
    if (POST) {
      float first[1] = {sum_z(0)};
      group_sum(first, sums[group][1][1], tid, gt, 1 + group);
      sz = first[0];
    }
  }
  for (; t < T; t += stride, par ^= 1) {
    const size_t base = (size_t)t * d;
    F2 y[V][4], D[V][4];
    float c = g.bs;
    const float own = gate;   // this row's
    if (g.gate) {
      c *= sigmoid(own);
      if (t + stride < T) gate = g.gate[t + stride];   // the next row's, ahead of its use
    }
    const float rz = POST ? inv_rms(sz, inv_d, eps) : 1.f;
    const F2 cr = f2(c * rz);
    if (!Z) ahead.template wait<DEPTH - 1>();
    F2 ry = f2(0.f), k = ry;   // 1 / rms(y), and -ry times the mean term of D
    if (DA) {
      F2 yy = f2(0.f), qy = yy;   // sum y^2, sum da pre_w y
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d) {
          F2 w[4], v[4];
          unpack8(ahead.get(slot, 0, i), y[i]);
          if (Z) {
            unpack8(ahead.get(slot, 1, i), v);
            if (POST) weight(0, i, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[i][j] = fma2(cr, POST ? mul2(v[j], w[j]) : v[j], mul2(rs, y[i][j]));
          }
          unpack8(ahead.get(slot, 3, i), v);
          weight(1, i, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            D[i][j] = mul2(v[j], w[j]);   // the gradient through a, before its row terms
            yy = fma2(y[i][j], y[i][j], yy);
            qy = fma2(D[i][j], y[i][j], qy);
          }
        }
      float sy[2] = {both(yy), both(qy)};
      group_sum(sy, sums[group][par][0], tid, gt, 1 + group);
      const float r = inv_rms(sy[0], inv_d, eps);
      ry = f2(r);
      k = f2(-(r * r * sy[1] * inv_d));
    }
    F2 dot = f2(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ahead.elem(i) < d) {
        F2 v[4];
        if (DA) {
          unpack8(ahead.get(slot, 3, i), v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dpre[i][j] = fma2(v[j], mul2(y[i][j], ry), dpre[i][j]);
            D[i][j] = fma2(k, y[i][j], D[i][j]);
          }
          if (has_dy) {
            unpack8(ahead.get(slot, 2, i), v);
#pragma unroll
            for (int j = 0; j < 4; ++j) D[i][j] = fma2(ry, D[i][j], v[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) D[i][j] = mul2(ry, D[i][j]);
          }
        } else {
          unpack8(ahead.get(slot, 2, i), D[i]);
        }
        if (g.dx) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = mul2(rs, D[i][j]);
          *reinterpret_cast<uint4*>(g.dx + base + ahead.elem(i)) = pack8(v);
        }
        if (Z) {
          F2 z[4];
          unpack8(ahead.get(slot, 1, i), z);
          if (POST) {
            F2 w[4];
            weight(0, i, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              dpost[i][j] = fma2(cr, mul2(D[i][j], z[j]), dpost[i][j]);
              D[i][j] = mul2(D[i][j], w[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dot = fma2(D[i][j], z[j], dot);
            if (POST) y[i][j] = z[j];   // z waits in y's place until S is known
          }
        }
      }
    // this row's copies are read; z of the next row is there with all but the DEPTH - 1
    // rows asked for last
    ahead.start(slot, src, t + DEPTH * stride, T, d);
    if (++slot == DEPTH) slot = 0;
    if (Z) {
      ahead.template wait<DEPTH - 1>();
      float sw[2] = {both(dot), 0.f};     // S, sum z^2 of the next row
      if (POST && t + stride < T) sw[1] = sum_z(slot);
      if (POST || g.dgate) group_sum(sw, sums[group][par][1], tid, gt, 1 + group);
      sz = sw[1];
      const F2 kz = f2(POST ? -(rz * rz * sw[0] * inv_d) : 0.f);
      if (g.dgate && tid == 0) g.dgate[t] = g.bs * sigmoid_slope(own) * rz * sw[0];
      if (g.dz) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (ahead.elem(i) < d) {
#pragma unroll
            for (int j = 0; j < 4; ++j) D[i][j] = mul2(cr, POST ? fma2(kz, y[i][j], D[i][j]) : D[i][j]);
            *reinterpret_cast<uint4*>(g.dz + base + ahead.elem(i)) = pack8(D[i]);
          }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (g.part) {
    // the groups' sums, added in order by the first group
    __syncthreads();
    float* acc = reinterpret_cast<float*>(rows);   // [group][2][d]
    if (group) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            F2* o = reinterpret_cast<F2*>(acc + ((size_t)group * 2 + h) * d + ahead.elem(i));
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = h ? dpre[i][j] : dpost[i][j];
          }
    }
    __syncthreads();
    if (!group) {
      float* p = g.part + (size_t)blockIdx.x * 2 * d;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ahead.elem(i) < d)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            F2(&v)[4] = h ? dpre[i] : dpost[i];
            for (int q = 1; q < groups; ++q) {
              const F2* a = reinterpret_cast<const F2*>(acc + ((size_t)q * 2 + h) * d + ahead.elem(i));
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = add2(v[j], a[j]);
            }
            F2* o = reinterpret_cast<F2*>(p + (size_t)h * d + ahead.elem(i));
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = v[j];
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
  constexpr auto* kernel = block_norm_fwd_kernel<V, DEPTH, Z, POST, PRE>;
  const int threads = ((g.d / 8 + V - 1) / V + 31) / 32 * 32, smem = DEPTH * 2 * V * threads * 16;
  cudaError_t e = allow_smem<kernel>(DEPTH * 2 * V * kMaxWarps * 32 * 16);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  int per_sm = 1;
  if (g.T > sms) {   // as many CTAs as the GPU holds
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    if (e != cudaSuccess) return e;
  }
  const int most = sms * (per_sm > 0 ? per_sm : 1);
  return launch_pdl(kernel, dim3(g.T < most ? g.T : most), dim3(threads), smem, s, g);
}

template <int V, int DEPTH>
cudaError_t pick_fwd(const NormArgs& g, cudaStream_t s) {
  if (!g.z) return run_fwd<V, DEPTH, false, false, true>(g, s);
  if (g.post_w) return g.pre_w ? run_fwd<V, DEPTH, true, true, true>(g, s) : run_fwd<V, DEPTH, true, true, false>(g, s);
  return g.pre_w ? run_fwd<V, DEPTH, true, false, true>(g, s) : run_fwd<V, DEPTH, true, false, false>(g, s);
}

template <int V, int DEPTH, bool Z, bool POST, bool DA>
cudaError_t run_bwd(const NormArgs& g, int ctas, cudaStream_t s) {
  auto* kernel = block_norm_bwd_kernel<V, DEPTH, Z, POST, DA>;
  const int gt = ((g.d / 8 + V - 1) / V + 31) / 32 * 32, threads = kBwdThreads / gt * gt;
  constexpr int kWeightBytes = V <= 2 ? 8192 * 2 * 4 : 0;   // of the longest row
  const int smem = DEPTH * 4 * V * threads * 16 + (V <= 2 ? g.d * 2 * 4 : 0);
  const cudaError_t e = allow_smem<block_norm_bwd_kernel<V, DEPTH, Z, POST, DA>>(DEPTH * 4 * V * kBwdThreads * 16 +
                                                                                         kWeightBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(ctas), dim3(threads), smem, s, g, gt);
}

template <int V, int DEPTH>
cudaError_t pick_bwd(const NormArgs& g, int n, cudaStream_t s) {
  if (!g.z) return run_bwd<V, DEPTH, false, false, true>(g, n, s);
  if (g.post_w)
    return g.da ? run_bwd<V, DEPTH, true, true, true>(g, n, s) : run_bwd<V, DEPTH, true, true, false>(g, n, s);
  return g.da ? run_bwd<V, DEPTH, true, false, true>(g, n, s) : run_bwd<V, DEPTH, true, false, false>(g, n, s);
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

int block_norm_parts(int T) {
  const int most = sm_count();
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
  const int n = block_norm_parts(T);
  const cudaError_t e = g.d <= 8192 ? pick_bwd<2, 2>(g, n, s) : pick_bwd<4, 1>(g, n, s);
  if (e != cudaSuccess || !g.part) return e;
  return launch_pdl(block_norm_reduce_kernel, dim3((g.d + 31) / 32, 2), dim3(256), 0, s, static_cast<const float*>(parts),
                    n, g.d, o.dpost_w, o.dpre_w);
}

}  // namespace moe
