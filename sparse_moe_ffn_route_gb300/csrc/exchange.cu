// The exchange around a sparse layer's experts (moe_exchange.h): slots sorted by expert with the
// tokens' rows copied along, and the weighted sum of the rows back at their token, with the
// gradients of both.
//
// Everything here is bound by memory, and goes by token, not by sorted row: a token's row
// is read (or written) once and its k sorted rows are written (or read) once.
#include "../../include/moe_exchange.h"
#include "abi_check.h"
#include "common.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- the sort
// The slots are cut into chunks, one CTA each.  First every chunk counts its slots of each
// expert; then each CTA knows where its chunk's slots of an expert begin (all slots of the
// experts before, and the expert's slots in the chunks before), and places them in order:
// 1024 slots at a time, a warp 32 of them, a slot's place among those of its warp by
// match_any, and the warps' counts added up in a table.
constexpr int kSortThreads = 1024, kChunk = 2048, kMostChunks = 128;

struct SortArgs {
  const int32_t* ids;
  int S, E, chunks, chunk;   // slots, experts; chunks of so many slots
  int32_t *hist;             // [chunks][E]
  int32_t *offsets, *rows;
};

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a) {
  __shared__ int count[kMaxExperts];
  pdl_wait();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int s0 = blockIdx.x * a.chunk, s1 = min(a.S, s0 + a.chunk);
  for (int s = s0 + threadIdx.x; s < s1; s += kSortThreads) {
    const int e = a.ids[s];
    if (e >= 0 && e < a.E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.hist[(size_t)blockIdx.x * a.E + e] = count[e];
  pdl_trigger();
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortArgs a) {
  __shared__ int cursor[kMaxExperts], warp_sum[32];
  __shared__ __align__(16) uint8_t table[kMaxExperts][32];   // an expert's slots in each warp
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // thread e: expert e's slots in all chunks, and in those before this one
  int all = 0, before = 0;
  if (tid < a.E)
    for (int c = 0; c < a.chunks; ++c) {
      const int n = a.hist[(size_t)c * a.E + tid];
      all += n;
      before += c < (int)blockIdx.x ? n : 0;
    }
  int inc = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int base = inc - all;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  if (tid < a.E) {
    cursor[tid] = base + before;
    if (blockIdx.x == 0) {
      a.offsets[tid] = base;
      if (tid == a.E - 1) a.offsets[a.E] = base + all;
    }
  }
  const int s0 = blockIdx.x * a.chunk, s1 = min(a.S, s0 + a.chunk);
  for (int from = s0; from < s1; from += kSortThreads) {
    for (int i = tid; i < a.E * 8; i += kSortThreads) reinterpret_cast<uint32_t*>(table)[i] = 0u;
    const int s = from + tid;
    int e = s < s1 ? a.ids[s] : -1;
    if (e < 0 || e >= a.E) e = -1;
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    __syncthreads();
    if (e >= 0 && rank == 0) table[e][warp] = (uint8_t)__popc(peers);
    __syncthreads();
    if (s < s1) {
      int row = -1;
      if (e >= 0) {
        const uint32_t* t = reinterpret_cast<const uint32_t*>(table[e]);
        uint32_t earlier = 0;
        for (int q = 0; q < (warp >> 2); ++q) earlier = __dp4a(t[q], 0x01010101u, earlier);
        if (warp & 3) earlier = __dp4a(t[warp >> 2] & ((1u << (8 * (warp & 3))) - 1u), 0x01010101u, earlier);
        row = cursor[e] + (int)earlier + rank;
      }
      a.rows[s] = row;
    }
    __syncthreads();
    for (int i = tid; i < a.E; i += kSortThreads) {   // the next slots come behind
      const uint32_t* t = reinterpret_cast<const uint32_t*>(table[i]);
      uint32_t n = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) n = __dp4a(t[q], 0x01010101u, n);
      cursor[i] += (int)n;
    }
    __syncthreads();
  }
  pdl_trigger();
}

// ---------------------------------------------------------------- rows
// A token's row is cut over `parts` warps, so that few tokens still fill the GPU; warp w of all
// takes part w % parts of token w / parts, then those behind.
struct RowArgs {
  const int32_t* rows;       // [T, k]
  int T, k, S;
  int vecs, parts;           // 16-byte vectors of a row; warps to a row
};

constexpr int kRowWarps = 8;

// xs[rows[t, j]] = x[t]
__global__ void __launch_bounds__(kRowWarps * 32) dispatch_rows_kernel(const RowArgs a, const uint4* __restrict__ x,
                                                                       const float* __restrict__ x_scale, uint4* xs,
                                                                       float* xs_scale) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long units = (long long)a.T * a.parts, step = (long long)gridDim.x * kRowWarps;
  for (long long u = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < units; u += step) {
    const int t = (int)(u / a.parts), part = (int)(u - (long long)t * a.parts);
    const int mine = lane < a.k ? a.rows[(size_t)t * a.k + lane] : -1;   // k is 32 at most
    for (int v0 = part * 32; v0 < a.vecs; v0 += 128 * a.parts) {
      uint4 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = v0 + 32 * i * a.parts + lane;
        if (v < a.vecs) q[i] = __ldg(x + (size_t)t * a.vecs + v);
      }
      for (int j = 0; j < a.k; ++j) {
        const int r = __shfl_sync(0xffffffffu, mine, j);
        if ((unsigned)r >= (unsigned)a.S) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int v = v0 + 32 * i * a.parts + lane;
          if (v < a.vecs) xs[(size_t)r * a.vecs + v] = q[i];
        }
      }
    }
    if (xs_scale && part == 0 && (unsigned)mine < (unsigned)a.S) xs_scale[mine] = x_scale[t];
  }
  pdl_trigger();
}

__device__ __forceinline__ void unpack8(const uint4& q, float (&f)[8]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(u[i]);
    f[2 * i + 1] = bf16_hi(u[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// y[t] = residual[t] + sum_j w[t, j] z[rows[t, j]]
__global__ void __launch_bounds__(kRowWarps * 32) combine_rows_kernel(const RowArgs a, const uint4* __restrict__ z,
                                                                      const float* __restrict__ w, const uint4* residual,
                                                                      uint4* y) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long units = (long long)a.T * a.parts, step = (long long)gridDim.x * kRowWarps;
  for (long long u = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < units; u += step) {
    const int t = (int)(u / a.parts), part = (int)(u - (long long)t * a.parts);
    const int mine = lane < a.k ? a.rows[(size_t)t * a.k + lane] : -1;
    const float weight = w && lane < a.k ? w[(size_t)t * a.k + lane] : 1.f;
    for (int v = part * 32 + lane; v - lane < a.vecs; v += 32 * a.parts) {
      const bool in = v < a.vecs;
      float sum[8] = {};
      if (residual && in) unpack8(residual[(size_t)t * a.vecs + v], sum);
      for (int j0 = 0; j0 < a.k; j0 += 4) {
        uint4 q[4];
        bool has[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = __shfl_sync(0xffffffffu, mine, (j0 + i) & 31);
          has[i] = in && j0 + i < a.k && (unsigned)r < (unsigned)a.S;
          if (has[i]) q[i] = __ldg(z + (size_t)r * a.vecs + v);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = __shfl_sync(0xffffffffu, weight, (j0 + i) & 31);
          if (has[i]) {
            float f[8];
            unpack8(q[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = fmaf(c, f[e], sum[e]);
          }
        }
      }
      if (in) y[(size_t)t * a.vecs + v] = pack8(sum);
    }
  }
  pdl_trigger();
}

// dz[rows[t, j]] = w[t, j] dy[t];  dw[t, j] = dy[t] . z[rows[t, j]].  A CTA of parts warps takes
// a token at a time.
__global__ void __launch_bounds__(kRowWarps * 32) combine_backward_kernel(const RowArgs a, const uint4* __restrict__ dy,
                                                                          const uint4* __restrict__ z,
                                                                          const float* __restrict__ w, uint4* dz, float* dw) {
  __shared__ float part_sum[2][kRowWarps][kMaxTopK];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int turn = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const int mine = lane < a.k ? a.rows[(size_t)t * a.k + lane] : -1;
    const float weight = lane < a.k ? w[(size_t)t * a.k + lane] : 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int r = __shfl_sync(0xffffffffu, mine, j);
      const float c = __shfl_sync(0xffffffffu, weight, j);
      float sum = 0.f;
      if ((unsigned)r < (unsigned)a.S)
        for (int v = warp * 32 + lane; v < a.vecs; v += 32 * a.parts) {
          float g[8];
          unpack8(__ldg(dy + (size_t)t * a.vecs + v), g);
          if (dw) {
            float f[8];
            unpack8(__ldg(z + (size_t)r * a.vecs + v), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(g[e], f[e], sum);
          }
          if (dz) {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] *= c;
            dz[(size_t)r * a.vecs + v] = pack8(g);
          }
        }
      if (dw) {
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) part_sum[turn][warp][j] = sum;
      }
    }
    if (dw) {
      __syncthreads();
      if (warp == 0 && lane < a.k) {
        float s = 0.f;
        for (int p = 0; p < a.parts; ++p) s += part_sum[turn][p][lane];
        dw[(size_t)t * a.k + lane] = s;
      }
    }
  }
  pdl_trigger();
}

// ---------------------------------------------------------------- host
int cdiv(long long a, int b) { return (int)((a + b - 1) / b); }

int chunk_slots(int S) { return S <= kChunk * kMostChunks ? kChunk : cdiv(cdiv(S, kMostChunks), kSortThreads) * kSortThreads; }
int chunk_count(int S) { return S ? cdiv(S, chunk_slots(S)) : 1; }

RowArgs row_args(const moe_exchange_cfg_t& c, const int32_t* rows, int T) {
  RowArgs a{};
  a.rows = rows;
  a.T = T;
  a.k = c.top_k;
  a.S = T * c.top_k;
  a.vecs = c.d_model * (c.format == MOE_ROWS_E4M3 ? 1 : 2) / 16;
  const int most = cdiv(a.vecs, 32), want = cdiv(48LL * sm_count(), T);
  a.parts = want < most ? (want > 1 ? want : 1) : most;
  return a;
}

int row_grid(const RowArgs& a) {
  const long long blocks = ((long long)a.T * a.parts + kRowWarps - 1) / kRowWarps, most = 64LL * sm_count();
  return (int)(blocks < most ? blocks : most);
}

int check_cfg(const moe_exchange_cfg_t* c, int T, bool bf16) {
  if (!c || c->d_model <= 0 || c->n_experts <= 0 || c->top_k <= 0 || T < 0) return MOE_ERR_INVALID_ARG;
  if (c->format != MOE_ROWS_BF16 && c->format != MOE_ROWS_E4M3) return MOE_ERR_INVALID_ARG;
  for (int r : c->reserved)
    if (r) return MOE_ERR_INVALID_ARG;
  if (c->n_experts > kMaxExperts || c->top_k > kMaxTopK || c->d_model > kMaxInputs) return MOE_ERR_UNSUPPORTED;
  if (c->d_model % (c->format == MOE_ROWS_E4M3 ? 16 : 8)) return MOE_ERR_UNSUPPORTED;
  if (bf16 && c->format != MOE_ROWS_BF16) return MOE_ERR_UNSUPPORTED;
  return (long long)T * c->top_k > kMaxTokens ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

#define EXCHANGE_CUDA(call)                         \
  do {                                              \
    if ((call) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

int sum_rows(const moe_exchange_cfg_t* cfg, const void* z, const int32_t* rows, const float* w, const void* residual,
             int32_t T, void* y, void* stream) {
  const int st = check_cfg(cfg, T, true);
  if (st != MOE_OK || T == 0) return st;
  if (!z || !rows || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned16(z, rows, w, residual, y)) return MOE_ERR_ALIGNMENT;
  const size_t S = (size_t)T * cfg->top_k, row = (size_t)cfg->d_model * 2;
  const Span out[] = {{y, T * row}};
  const Span in[] = {{z, S * row}, {rows, S * 4}, {w, S * 4}, {residual == y ? nullptr : residual, T * row}};
  if (overlap(out, in)) return MOE_ERR_INVALID_ARG;
  const RowArgs a = row_args(*cfg, rows, T);
  EXCHANGE_CUDA(launch_pdl(combine_rows_kernel, dim3(row_grid(a)), dim3(kRowWarps * 32), 0, static_cast<cudaStream_t>(stream), a,
                           static_cast<const uint4*>(z), w, static_cast<const uint4*>(residual), static_cast<uint4*>(y)));
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_dispatch_workspace_bytes(const moe_exchange_cfg_t* cfg, int32_t T) {
  if (check_cfg(cfg, T, false) != MOE_OK) return 0;
  return align_up((size_t)chunk_count(T * cfg->top_k) * cfg->n_experts * 4);
}

int moe_dispatch_forward(const moe_exchange_cfg_t* cfg, const int32_t* topk_ids, const void* x, const float* x_scale,
                         int32_t T, int32_t* offsets, int32_t* rows, void* xs, float* xs_scale, void* ws,
                         size_t ws_bytes, void* stream) {
  const int st = check_cfg(cfg, T, false);
  if (st != MOE_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!offsets) return MOE_ERR_INVALID_ARG;
  if (!aligned16(offsets)) return MOE_ERR_ALIGNMENT;
  const size_t ends = ((size_t)cfg->n_experts + 1) * 4;
  if (T == 0) {
    EXCHANGE_CUDA(cudaMemsetAsync(offsets, 0, ends, s));
    return MOE_OK;
  }
  const bool eight = cfg->format == MOE_ROWS_E4M3 && xs;
  if (!topk_ids || !rows || !ws || (x != nullptr) != (xs != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((x_scale != nullptr) != eight || (xs_scale != nullptr) != eight) return MOE_ERR_INVALID_ARG;
  if (!aligned16(topk_ids, x, x_scale, rows, xs, xs_scale, ws)) return MOE_ERR_ALIGNMENT;
  const size_t need = moe_dispatch_workspace_bytes(cfg, T);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  const size_t S = (size_t)T * cfg->top_k, row = (size_t)cfg->d_model * (eight ? 1 : 2);
  const Span out[] = {{offsets, ends}, {rows, S * 4}, {xs, S * row}, {xs_scale, S * 4}, {ws, need}};
  const Span in[] = {{topk_ids, S * 4}, {x, T * row}, {x_scale, (size_t)T * 4}};
  if (overlap(out, in)) return MOE_ERR_INVALID_ARG;
  SortArgs a{};
  a.ids = topk_ids;
  a.S = (int)S;
  a.E = cfg->n_experts;
  a.chunk = chunk_slots(a.S);
  a.chunks = chunk_count(a.S);
  a.hist = static_cast<int32_t*>(ws);
  a.offsets = offsets;
  a.rows = rows;
  EXCHANGE_CUDA(launch_pdl(sort_count_kernel, dim3(a.chunks), dim3(kSortThreads), 0, s, a));
  EXCHANGE_CUDA(launch_pdl(sort_place_kernel, dim3(a.chunks), dim3(kSortThreads), 0, s, a));
  if (xs) {
    const RowArgs r = row_args(*cfg, rows, T);
    EXCHANGE_CUDA(launch_pdl(dispatch_rows_kernel, dim3(row_grid(r)), dim3(kRowWarps * 32), 0, s, r, static_cast<const uint4*>(x),
                             x_scale, static_cast<uint4*>(xs), xs_scale));
  }
  return MOE_OK;
}

int moe_dispatch_backward(const moe_exchange_cfg_t* cfg, const void* dxs, const int32_t* rows, int32_t T, void* dx,
                          void* stream) {
  return sum_rows(cfg, dxs, rows, nullptr, nullptr, T, dx, stream);
}

int moe_combine_forward(const moe_exchange_cfg_t* cfg, const void* z, const int32_t* rows, const float* w,
                        const void* residual, int32_t T, void* y, void* stream) {
  return sum_rows(cfg, z, rows, w, residual, T, y, stream);
}

int moe_combine_backward(const moe_exchange_cfg_t* cfg, const void* dy, const void* z, const int32_t* rows,
                         const float* w, int32_t T, void* dz, float* dw, void* stream) {
  const int st = check_cfg(cfg, T, true);
  if (st != MOE_OK || T == 0) return st;
  if ((!dz && !dw) || !dy || !rows || !w || (dw && !z)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy, z, rows, w, dz, dw)) return MOE_ERR_ALIGNMENT;
  const size_t S = (size_t)T * cfg->top_k, row = (size_t)cfg->d_model * 2;
  const Span out[] = {{dz, S * row}, {dw, S * 4}};
  const Span in[] = {{dy, T * row}, {dw ? z : nullptr, S * row}, {rows, S * 4}, {w, S * 4}};
  if (overlap(out, in)) return MOE_ERR_INVALID_ARG;
  RowArgs a = row_args(*cfg, rows, T);
  a.parts = cdiv(a.vecs, 64) < kRowWarps ? cdiv(a.vecs, 64) : kRowWarps;
  const int most = 16 * sm_count();
  EXCHANGE_CUDA(launch_pdl(combine_backward_kernel, dim3(T < most ? T : most), dim3(a.parts * 32), 0,
                           static_cast<cudaStream_t>(stream), a, static_cast<const uint4*>(dy), static_cast<const uint4*>(z), w,
                           static_cast<uint4*>(dz), dw));
  return MOE_OK;
}

}  // extern "C"
