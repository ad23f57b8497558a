// The exchange around a sparse layer's experts (moe_exchange.h): slots sorted by expert with the
// tokens' rows copied along, and the weighted sum of the rows back at their token, with the
// gradients of both.
//
// Everything here is bound by memory, and goes by token, not by sorted row: a token's row
// is read (or written) once and its k sorted rows are written (or read) once.
//
// Measured, 4096 tokens of 2048 in bf16, 8 experts each of 256 (151 MB a kernel, the combine's
// gradient 285; a copy's rate is 6.8 TB/s): sort and copy 29.1 us with the count's launch, rows
// back 27.4 (168 MB with the residual: 6.1 TB/s), their gradient 49.6 (5.75 TB/s),
// the first's gradient 24.9 (6.1).  1001 tokens of 2880, 4 experts each of 32, where
// the launches show: 7.5, 4.1, 9.4 and 4.0 us from L2.  A few tokens take one launch's 3.1 to 3.6 us.
#include <algorithm>

#include "../../include/moe_exchange.h"
#include "abi_check.h"
#include "block.h"
#include "f32x2.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- out: sort and copy
// Each CTA takes a run of tokens, finds where its slots go and copies its tokens' rows there.
// A slot's row is (all slots of the experts before) + (its expert's slots before this
// run) + (those before it in the run).  The first two come from counts: of all ids themselves
// where these are few (one launch), else of chunks of slots, which a launch before has counted,
// and of the ids between the chunk's start and the run's.  The third comes tile by tile, a
// thread to a slot: the slot's place among those of its warp by match_any, and the warps'
// counts added up in a table.
constexpr int kCountThreads = 1024, kMostChunks = 128;
// Slots up to which every CTA counts all ids, and slots of a chunk beyond.  (Every CTA reads
// kDirect ids at most, or a chunk and the chunks' counts.)
constexpr int kDirect = 8192, kChunk = 2048;

struct SortArgs {
  const int32_t* ids;
  int T, k, S, E;            // S = T k slots
  int chunks, chunk;         // 0: count all ids
  int32_t* hist;             // [chunks][E]
  int32_t *offsets, *rows;
  int vecs;                  // 16-byte vectors of a row; 0: sort alone
  const uint4* x;
  uint4* xs;
  const float* x_scale;
  float* xs_scale;
  uint32_t* status;          // cleared by the call's first kernel
};

__global__ void __launch_bounds__(kCountThreads) sort_count_kernel(const SortArgs a) {
  __shared__ int count[kMaxExperts];
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0u;
  pdl_trigger();   // what does not need the counts may start
  for (int e = threadIdx.x; e < a.E; e += kCountThreads) count[e] = 0;
  __syncthreads();
  const int s0 = blockIdx.x * a.chunk, s1 = min(a.S, s0 + a.chunk);
  for (int s = s0 + threadIdx.x; s < s1; s += kCountThreads) {
    const int e = a.ids[s];
    if (e >= 0 && e < a.E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kCountThreads) a.hist[(size_t)blockIdx.x * a.E + e] = count[e];
}

// Sum of four bytes of counts.
__device__ __forceinline__ uint32_t add_bytes(uint32_t w, uint32_t sum) { return __dp4a(w, 0x01010101u, sum); }

// NT threads, W = NT / 32 warps.
template <int NT>
__global__ void __launch_bounds__(NT) dispatch_kernel(const SortArgs a) {
  constexpr int W = NT / 32, PER = kMaxExperts / NT;   // experts of a thread in the scan
  __shared__ int all[kMaxExperts], cursor[kMaxExperts], warp_sum[W], tile_rows[NT];
  __shared__ __align__(16) uint8_t table[kMaxExperts][W];   // an expert's slots in each warp of a tile
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = (int)((long long)a.T * blockIdx.x / gridDim.x), t1 = (int)((long long)a.T * (blockIdx.x + 1) / gridDim.x);
  const int s0 = t0 * a.k;
  for (int e = tid; e < a.E; e += NT) all[e] = cursor[e] = 0;
  __syncthreads();
  // With counts to come, only these have to be waited for: the launch that makes them has itself
  // waited for what is before it on the stream.
  if (!a.chunks) {
    pdl_wait();
    if (blockIdx.x == 0 && tid == 0) *a.status = 0u;
  }
  // A warp copies up to 4 x 32 vectors of a token at a time; its first ones are asked for now.
  const int pieces = (a.vecs + 127) / 128, piece = pieces ? (a.vecs + 32 * pieces - 1) / (32 * pieces) * 32 : 0;
  uint4 q[4];
  auto load = [&](int u) {   // unit u of the run
    const int i = u / pieces, v0 = (u - i * pieces) * piece;
    const uint4* src = a.x + (size_t)(t0 + i) * a.vecs;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int v = v0 + 32 * h + lane;
      if (32 * h < piece && v < a.vecs) q[h] = __ldg(src + v);
    }
  };
  int unit = warp;
  if (a.vecs && unit < (t1 - t0) * pieces) load(unit);
  const int chunk = a.chunks ? s0 / a.chunk : 0;
  for (int s = (a.chunks ? chunk * a.chunk : 0) + tid, end = a.chunks ? s0 : a.S; s < end; s += NT) {
    const int e = a.ids[s];
    if (e >= 0 && e < a.E) {
      if (!a.chunks) atomicAdd(&all[e], 1);
      if (s < s0) atomicAdd(&cursor[e], 1);
    }
  }
  __syncthreads();
  if (a.chunks) {
    pdl_wait();
    for (int e = tid; e < a.E; e += NT) {
      int sum = 0, before = 0;
      for (int c0 = 0; c0 < a.chunks; c0 += 16) {
        int n[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) n[i] = c0 + i < a.chunks ? a.hist[(size_t)(c0 + i) * a.E + e] : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          sum += n[i];
          before += c0 + i < chunk ? n[i] : 0;
        }
      }
      all[e] = sum;
      cursor[e] += before;
    }
    __syncthreads();
  }
  // where each expert's rows begin: an exclusive scan, PER experts to a thread
  int mine[PER], run = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = PER * tid + i;
    mine[i] = run;
    run += e < a.E ? all[e] : 0;
  }
  int inc = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int base = inc - run;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = PER * tid + i;
    if (e < a.E) {
      cursor[e] += base + mine[i];
      if (blockIdx.x == 0) {
        a.offsets[e] = base + mine[i];
        if (e == a.E - 1) a.offsets[a.E] = base + run;
      }
    }
  }
  // tiles of whole tokens
  const int per_tile = NT / a.k;
  for (int t = t0; t < t1; t += per_tile) {
    const int tokens = min(per_tile, t1 - t), slots = tokens * a.k;
    for (int i = tid; i < a.E * (W / 4); i += NT) reinterpret_cast<uint32_t*>(table)[i] = 0u;
    const int s = t * a.k + tid;
    int e = tid < slots ? a.ids[s] : -1;
    if (e < 0 || e >= a.E) e = -1;
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    __syncthreads();
    if (e >= 0 && rank == 0) table[e][warp] = (uint8_t)__popc(peers);
    __syncthreads();
    int row = -1;
    if (e >= 0) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(table[e]);
      uint32_t earlier = 0;
      for (int q = 0; q < (warp >> 2); ++q) earlier = add_bytes(w[q], earlier);
      if (warp & 3) earlier = add_bytes(w[warp >> 2] & ((1u << (8 * (warp & 3))) - 1u), earlier);
      row = cursor[e] + (int)earlier + rank;
    }
    if (tid < slots) a.rows[s] = tile_rows[tid] = row;
    __syncthreads();
    if (t + per_tile < t1)
      for (int i = tid; i < a.E; i += NT) {   // the next tile's slots come behind
        const uint32_t* w = reinterpret_cast<const uint32_t*>(table[i]);
        uint32_t n = 0;
#pragma unroll
        for (int q = 0; q < W / 4; ++q) n = add_bytes(w[q], n);
        cursor[i] += (int)n;
      }
    if (a.vecs) {
      for (; unit < (t + tokens - t0) * pieces; unit += W) {
        const int i = unit / pieces, v0 = (unit - i * pieces) * piece;
        uint4 p[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) p[h] = q[h];
        if (unit + W < (t1 - t0) * pieces) load(unit + W);
        const int* to = tile_rows + (t0 + i - t) * a.k;
        for (int j = 0; j < a.k; ++j) {
          const int r = to[j];
          if (r < 0) continue;
          uint4* dst = a.xs + (size_t)r * a.vecs;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int v = v0 + 32 * h + lane;
            if (32 * h < piece && v < a.vecs) dst[v] = p[h];
          }
        }
      }
      if (a.xs_scale && row >= 0) a.xs_scale[row] = a.x_scale[t + tid / a.k];
    }
    __syncthreads();
  }
  pdl_trigger();
}

// ---------------------------------------------------------------- back: rows to their tokens
struct RowArgs {
  const int32_t* rows;       // [T, k]
  int T, k, S;
  int vecs, groups;          // 16-byte vectors of a row; groups of 32 of them
};

// y[t] = residual[t] + sum_j w[t, j] z[rows[t, j]].  threadIdx.y: tokens of a CTA (whole warps
// each); threadIdx.x and blockIdx.y: vectors of the row.  A thread has the vectors of KT rows
// in flight, of more than 8 four at a time (2000 x 4096, 12 rows: 39 us, eight at a time 45), and
// as many CTAs as their registers allow hide the way to a row, its number first.
// Smaller CTAs begin and end less at one time: with 128 threads instead of 256, 8 rows at
// 1001 x 2880 take 10.6 us instead of 12.8, 3 at 4096 x 2048 14.8 instead of 15.6, but 1 at
// 8000 x 1024, where a CTA has too little to do, 9.9 instead of 8.6.
// Persistent warps that copied units of 32 vectors ahead through shared memory took 27.7 us
// (here 27.4) at 4096 x 2048 with 8 rows a token, 54 (34) at 8192 x 4096 with one and 6.8 (4.1) at
// 1001 x 2880 with 4: each unit then waits for its row's number.  Row
// numbers and weights by shuffles from a lane's register: 50 us at the first of these sizes, the loads
// wait for one another.
constexpr int combine_threads(int kt, bool more) { return kt <= 2 || more ? 256 : 128; }
template <int KT, bool MORE>
__global__ void __launch_bounds__(combine_threads(KT, MORE), MORE ? 5 : KT == 8 ? 7 : KT == 4 ? 10 : 8)
combine_kernel(const RowArgs a, const uint4* __restrict__ z, const float* __restrict__ w, const uint4* residual, uint4* y) {
  pdl_wait();
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.T) return;
  int r[KT];
  float c[KT];
  auto look = [&](int j0) {
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      r[j] = j0 + j < a.k ? a.rows[t * a.k + j0 + j] : -1;
      if (KT <= 4) c[j] = w && j0 + j < a.k ? w[t * a.k + j0 + j] : 1.f;
      if ((unsigned)r[j] >= (unsigned)a.S) r[j] = -1;
    }
  };
  if (!MORE) look(0);
  for (int v = blockIdx.y * blockDim.x + threadIdx.x; v < a.vecs; v += blockDim.x * gridDim.y) {
    F2 sum[4] = {};
    if (residual) unpack8(residual[t * a.vecs + v], sum);
    for (int j0 = 0; j0 < (MORE ? a.k : 1); j0 += KT) {
      if (MORE) look(j0);
      uint4 q[KT];
#pragma unroll
      for (int j = 0; j < KT; ++j)
        if (r[j] >= 0) q[j] = __ldg(z + (size_t)r[j] * a.vecs + v);
#pragma unroll
      for (int j = 0; j < KT; ++j)
        if (r[j] >= 0) {
          F2 f[4];
          const F2 by = f2(KT <= 4 ? c[j] : w ? __ldg(w + t * a.k + j0 + j) : 1.f);   // (8 would spill)
          unpack8(q[j], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = fma2(by, f[e], sum[e]);
        }
    }
    y[t * a.vecs + v] = pack8(sum);
  }
  pdl_trigger();
}

// dz[rows[t, j]] = w[t, j] dy[t];  dw[t, j] = dy[t] . z[rows[t, j]].  threadIdx.y: tokens of
// a CTA (short rows); a token's warps take its vectors in turn, KB rows at a time in registers, and
// add their parts of the dot products up at the end.  Half of the bytes are writes, and many CTAs per
// SM keep both ways busy: 4096 x 2048 with 8 rows a token takes 50 us, 1001 x 2880 with 4 9 us;
// through rings in shared memory 51 to 59 us and 15 to 19.  One row a token, 8192 x 4096: 35 us, 52
// with the registers of four.  Row numbers and weights by shuffles from a lane's register instead of the
// same loads by all threads: 9.6 instead of 9.1 us at 1001 x 2880, 74 instead of 70 at 2000 x 4096
// with 12 rows.
constexpr int kBackWarps = 8;
template <int KB>
__global__ void __launch_bounds__(kBackWarps * 32, KB == 8 ? 3 : KB == 4 ? 4 : KB == 2 ? 5 : 7)
combine_backward_kernel(const RowArgs a, const uint4* __restrict__ dy, const uint4* __restrict__ z, const float* __restrict__ w,
                        uint4* dz, float* dw) {
  __shared__ float part_sum[kBackWarps][kMaxTopK];
  const int lane = threadIdx.x & 31, W = blockDim.x >> 5, first = threadIdx.y * W, warp = first + (threadIdx.x >> 5);
  pdl_wait();
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const int k = t < a.T ? a.k : 0;
  for (int j0 = 0; j0 < k; j0 += KB) {
    int r[KB];
    float c[KB];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const long long at = t * a.k + j0 + i;
      r[i] = j0 + i < k ? a.rows[at] : -1;
      if (KB <= 4) c[i] = j0 + i < k ? w[at] : 0.f;
      if ((unsigned)r[i] >= (unsigned)a.S) r[i] = -1;
    }
    F2 acc[KB] = {};
    for (int v = threadIdx.x; v < a.vecs; v += blockDim.x) {
      uint4 q[KB];
#pragma unroll
      for (int i = 0; i < KB; ++i)
        if (dw && r[i] >= 0) q[i] = __ldg(z + (size_t)r[i] * a.vecs + v);
      F2 d[4];
      unpack8(__ldg(dy + t * a.vecs + v), d);
#pragma unroll
      for (int i = 0; i < KB; ++i)
        if (r[i] >= 0) {
          if (dz) {
            const F2 by = f2(KB <= 4 ? c[i] : __ldg(w + t * a.k + j0 + i));   // (8 would spill)
            F2 o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = mul2(by, d[e]);
            dz[(size_t)r[i] * a.vecs + v] = pack8(o);
          }
          if (dw) {
            F2 f[4];
            unpack8(q[i], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i] = fma2(d[e], f[e], acc[i]);
          }
        }
    }
    if (dw) {
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        float v = both(acc[i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0 && j0 + i < k) part_sum[warp][j0 + i] = v;
      }
    }
  }
  if (dw) {
    __syncthreads();
    if (warp == first && lane < k) {
      float s = 0.f;
      for (int p = first; p < first + W; ++p) s += part_sum[p][lane];
      dw[t * a.k + lane] = s;   // (without a row: 0)
    }
  }
  pdl_trigger();
}

// ---------------------------------------------------------------- host
int cdiv(long long a, int b) { return (int)((a + b - 1) / b); }

int chunk_slots(int S) { return S <= kChunk * kMostChunks ? kChunk : cdiv(S, kMostChunks); }
int chunk_count(int S) { return S <= kDirect ? 0 : cdiv(S, chunk_slots(S)); }

RowArgs row_args(const moe_exchange_cfg_t& c, const int32_t* rows, int T) {
  RowArgs a{};
  a.rows = rows;
  a.T = T;
  a.k = c.top_k;
  a.S = T * c.top_k;
  a.vecs = c.d_model / 8;
  a.groups = cdiv(a.vecs, 32);
  return a;
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
  // short rows' CTAs take several tokens; with few tokens several take a row
  const int k = cfg->top_k, threads = combine_threads(k, k > 8);
  const int x = std::min(threads, a.groups * 32), ty = threads / x, ctas = cdiv(T, ty);
  const int pieces = std::max(1, std::min(cdiv(a.vecs, x), 1024 / threads * sm_count() / ctas));
  auto* kernel = k == 1   ? combine_kernel<1, false>
                 : k == 2 ? combine_kernel<2, false>
                 : k <= 4 ? combine_kernel<4, false>
                 : k <= 8 ? combine_kernel<8, false>
                          : combine_kernel<4, true>;
  EXCHANGE_CUDA(launch_pdl(kernel, dim3(ctas, pieces), dim3(x, ty), 0, static_cast<cudaStream_t>(stream), a,
                           static_cast<const uint4*>(z), w, static_cast<const uint4*>(residual), static_cast<uint4*>(y)));
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_dispatch_workspace_bytes(const moe_exchange_cfg_t* cfg, int32_t T) {
  if (check_cfg(cfg, T, false) != MOE_OK) return 0;
  return 256 + align_up((size_t)chunk_count(T * cfg->top_k) * cfg->n_experts * 4);
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
  a.T = T;
  a.k = cfg->top_k;
  a.S = (int)S;
  a.E = cfg->n_experts;
  a.chunks = chunk_count(a.S);
  a.chunk = chunk_slots(a.S);
  a.hist = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + 256);   // behind the status word
  a.status = static_cast<uint32_t*>(ws);
  a.offsets = offsets;
  a.rows = rows;
  a.vecs = xs ? (int)(row / 16) : 0;
  a.x = static_cast<const uint4*>(x);
  a.xs = static_cast<uint4*>(xs);
  a.x_scale = x_scale;
  a.xs_scale = xs_scale;
  if (a.chunks) EXCHANGE_CUDA(launch_pdl(sort_count_kernel, dim3(a.chunks), dim3(kCountThreads), 0, s, a));
  const int most = sm_count();
  // a token or two to a CTA: small CTAs start and meet sooner (8 tokens of 2048: 3.6 us, of
  // 1024 threads 4.2; 512 tokens: 6.3, 6.3; 1000: 13.3, 10.4)
  if (T <= 2 * most)
    EXCHANGE_CUDA(launch_pdl(dispatch_kernel<256>, dim3(T < most ? T : most), dim3(256), 0, s, a));
  else
    EXCHANGE_CUDA(launch_pdl(dispatch_kernel<1024>, dim3(most), dim3(1024), 0, s, a));
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
  const RowArgs a = row_args(*cfg, rows, T);
  // CTAs of at least 4 warps (20000 x 256, 2 rows a token: 9.5 us, with a CTA to a token 22; 16000 x 512,
  // 4 rows: 25.2, with 8 warps 26)
  const int warps = cdiv(a.groups, cdiv(a.groups, kBackWarps)), tokens = std::max(1, kBackWarps / 2 / warps);
  const int k = cfg->top_k;
  auto* kernel = k == 1   ? combine_backward_kernel<1>
                 : k == 2 ? combine_backward_kernel<2>
                 : k <= 4 ? combine_backward_kernel<4>
                          : combine_backward_kernel<8>;
  EXCHANGE_CUDA(launch_pdl(kernel, dim3(cdiv(T, tokens)), dim3(warps * 32, tokens), 0, static_cast<cudaStream_t>(stream), a,
                           static_cast<const uint4*>(dy), static_cast<const uint4*>(z), w, static_cast<uint4*>(dz), dw));
  return MOE_OK;
}

}  // extern "C"
