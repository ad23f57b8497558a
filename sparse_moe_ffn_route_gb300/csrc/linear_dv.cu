// Backward pass of the linear layer before its products: dv = dy act'(pre) in bf16, and the
// bias's gradient, the sum of dv's rows.
//
// Bound by memory: reads dy and pre, writes dv (6 bytes per element; without an activation
// dy alone, for the bias).  A CTA takes 256 columns, 8 to a lane, and a run of rows, one per
// warp at a time (pieces of 512 bytes; of 128 bytes, with the sums meeting in a cluster, a step of
// 4096 x 2048 x 2048 took 65 us instead of 57); each lane adds its columns up in registers, the
// warps add theirs in order, and the launch of the products, or where there is none a second
// kernel, adds the CTAs' partial sums in order.  4096 x 2048: 13 us (50 MB, 3.9 TB/s; half of the
// issue slots), dv then lies in L2 for the products.
#include "block.h"
#include "common.cuh"
#include "linear_act.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kCols = 256, kAhead = 4;

int cdiv(int a, int b) { return (a + b - 1) / b; }

template <int ACT>
__global__ void __launch_bounds__(kWarps * 32) linear_dv_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ pre,
                                                                int T, int n, uint16_t* dv, float* parts, uint32_t* status,
                                                                uint32_t* clear, int zeros) {
  __shared__ float sums[kWarps][kCols];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = blockIdx.x * kCols + 8 * lane;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0u;
  const long long first = blockIdx.y * gridDim.x + blockIdx.x;
  for (long long i = first * blockDim.x + threadIdx.x; i < zeros; i += (long long)gridDim.x * gridDim.y * blockDim.x) clear[i] = 0u;
  const int r0 = (int)((long long)T * blockIdx.y / gridDim.y), r1 = (int)((long long)T * (blockIdx.y + 1) / gridDim.y);
  F2 sum[4] = {};
  if (col < n)
    for (int r = r0 + warp; r < r1; r += kWarps * kAhead) {
      uint4 a[kAhead], z[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (r + i * kWarps < r1) {
          const size_t at = (size_t)(r + i * kWarps) * n + col;
          a[i] = __ldg(reinterpret_cast<const uint4*>(dy + at));
          if (ACT != MOE_LINEAR_NONE) z[i] = __ldg(reinterpret_cast<const uint4*>(pre + at));
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (r + i * kWarps < r1) {
          F2 v[4];
          unpack8(a[i], v);
          if (ACT != MOE_LINEAR_NONE) {
            F2 p[4];
            unpack8(z[i], p);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], linear_slope<ACT>(p[e]));
            if (dv) *reinterpret_cast<uint4*>(dv + (size_t)(r + i * kWarps) * n + col) = pack8(v);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], v[e]);
        }
    }
  if (parts) {
#pragma unroll
    for (int e = 0; e < 4; ++e) split(sum[e], sums[warp][8 * lane + 2 * e], sums[warp][8 * lane + 2 * e + 1]);
    __syncthreads();
    const int c = blockIdx.x * kCols + threadIdx.x;   // a thread to a column
    if (c < n) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w][threadIdx.x];
      parts[(size_t)blockIdx.y * n + c] = s;
    }
  }
  pdl_trigger();
}

__global__ void __launch_bounds__(kWarps * 32) linear_dbias_kernel(const BiasParts b) {
  pdl_wait();
  bias_sums(b, blockIdx.x * kWarps + (threadIdx.x >> 5), gridDim.x * kWarps, threadIdx.x & 31);
  pdl_trigger();
}

}  // namespace

int linear_bias_parts(int n, int T) {
  const int columns = cdiv(n, kCols), most = cdiv(4 * sm_count(), columns), least = cdiv(T, kWarps * kAhead);
  return least < most ? least : most;
}

cudaError_t launch_linear_dbias(const BiasParts& b, cudaStream_t s) {
  return launch_pdl(linear_dbias_kernel, dim3(cdiv(b.n, 2 * kWarps)), dim3(kWarps * 32), 0, s, b);
}

cudaError_t launch_linear_dv(int act, const uint16_t* dy, const uint16_t* pre, int T, int n, uint16_t* dv, float* parts,
                             uint32_t* status, uint32_t* clear, int zeros, cudaStream_t s) {
  const int rows = linear_bias_parts(n, T);
  auto run = [&](auto kernel) {
    return launch_pdl(kernel, dim3(cdiv(n, kCols), rows), dim3(kWarps * 32), 0, s, dy, pre, T, n, dv, parts, status,
                       clear, zeros);
  };
  return act == MOE_LINEAR_SILU        ? run(linear_dv_kernel<MOE_LINEAR_SILU>)
         : act == MOE_LINEAR_GELU      ? run(linear_dv_kernel<MOE_LINEAR_GELU>)
         : act == MOE_LINEAR_GELU_TANH ? run(linear_dv_kernel<MOE_LINEAR_GELU_TANH>)
                                       : run(linear_dv_kernel<MOE_LINEAR_NONE>);
}

}  // namespace moe
