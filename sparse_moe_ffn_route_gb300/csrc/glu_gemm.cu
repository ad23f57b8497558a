// The dense gated FFN on the 5th-generation tensor cores: its two forward products and
// the six of its backward pass, all D[128 x N] = A[128 x K] . B[N x K]^T tiles with fp32
// accumulators in TMEM, fed by TMA through an mbarrier ring.
//
//   gate/up:  g = x Wg^T, u = x Wu^T in one tile (the B tile holds nf rows of each), so
//             that the epilogue has both and writes h = act(g, u) (and, in training, g, u)
//   down:     y = h Wd^T
//   dact:     dh = dy Wd, whose epilogue turns it into dg and du with the saved g and u
//             (dh never reaches memory and is never rounded)
//   grads:    dx = dg Wg + du Wu (one sum over two runs of k), dWg = dg^T x,
//             dWu = du^T x, dWd = dy^T h, all in one launch so that the tiles of the
//             small products fill the SMs that the large ones leave
//
// An operand's k runs along its rows ("K-major": x Wg^T) or down its columns
// ("MN-major": both operands of dg^T x).  Both are read as they lie: a K-major tile is
// one box of 64 k (128 bytes, swizzled) per row, an MN-major one a box of 64 k rows per
// 64 columns; the tensor core's descriptors name the form.  Rows and columns past an
// edge are filled with zeros by the TMA unit, so d, ff and T need no padding.
//
// Warp roles of the persistent CTA: warp 0 TMA producer, warp 1 MMA issuer and owner of
// TMEM (two accumulators of up to 256 columns, so that a tile's epilogue runs under the
// next tile's MMAs), warps 2..5 epilogue.  Every wait is bounded (see tc::mbar_wait).
#include <cuda.h>

#include <cstring>

#include "block.h"
#include "common.cuh"
#include "glu_act.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kBM = 128, kBK = 64, kMaxN = 256;
constexpr int kTileA = kBM * kBK * 2;
constexpr int kStageBytes = kTileA + kMaxN * kBK * 2;   // 48 KiB
constexpr int kStages = 4;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
constexpr int kThreads = 192;
constexpr int kMaxProblems = 4;

enum : int { kEpiGlu = 0, kEpiStore = 1, kEpiDact = 2 };

// One product: D [M, N] over `segs` runs of `nkc` chunks of 64 k.  Run s multiplies
// a[s] and b[s]; with `pair` (gate/up) every chunk instead takes N / 2 rows of b[0] and
// N / 2 rows of b[1].
struct Problem {
  CUtensorMap a[2], b[2];
  int M, N;             // rows and columns of the output (pair: columns of h)
  int nkc, segs, pair;
  int a_mn, b_mn;       // 1: MN-major
  int tn;               // columns of B per tile (MMA N)
  int mt, nt;           // tiles
  uint16_t* out;        // bf16 [M, N]
};

struct GemmParams {
  Problem p[kMaxProblems];
  int n_problems, tiles;
  GluAct act;
  float *g, *u;         // saved (kEpiGlu: written when non-null; kEpiDact: read)
  uint16_t* out2;       // kEpiDact: du (out: dg)
  uint32_t* status;
  int clear_status;     // this is the call's first kernel
};

struct Tile {
  int pi, m, n;
};

// Tiles run in groups of 8 m tiles: the CTAs working at one time share a few A tiles and
// a few B tiles through L2.
__device__ __forceinline__ Tile tile_at(const GemmParams& g, int t) {
  Tile tl;
  tl.pi = 0;
  while (tl.pi + 1 < g.n_problems && t >= g.p[tl.pi].mt * g.p[tl.pi].nt) {
    t -= g.p[tl.pi].mt * g.p[tl.pi].nt;
    ++tl.pi;
  }
  const Problem& p = g.p[tl.pi];
  constexpr int kGroup = 8;
  const int per = kGroup * p.nt;
  const int grp = t / per, r = t - grp * per;
  const int m0 = grp * kGroup, rows = min(kGroup, p.mt - m0);
  tl.n = r / rows;
  tl.m = m0 + (r - tl.n * rows);
  return tl;
}

// Descriptor of an MN-major tile of 128-byte-swizzled boxes [64 k][64 mn]: 8 k rows are
// 1024 bytes, the boxes of successive 64 mn lie 8192 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(8192 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// 16 fp32 -> 16 bf16 at dst (two 16-byte stores; cols: how many are in range, a multiple of 8).
__device__ __forceinline__ void store_bf16x16(uint16_t* dst, const float (&v)[16], int cols) {
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  if (cols > 0) reinterpret_cast<uint4*>(dst)[0] = make_uint4(q[0], q[1], q[2], q[3]);
  if (cols > 8) reinterpret_cast<uint4*>(dst)[1] = make_uint4(q[4], q[5], q[6], q[7]);
}

template <int EPI>
__global__ void __launch_bounds__(kThreads, 1) glu_gemm_kernel(const __grid_constant__ GemmParams g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tc::smem_align1024(smem_raw);
  __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages], tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s, consumed_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &abort_s;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(tc::smem_u32(&full_bar[s]), 1);
      tc::mbar_init(tc::smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tc::smem_u32(&tfull_bar[b]), 1);
      tc::mbar_init(tc::smem_u32(&tempty_bar[b]), 4);
    }
    tc::mbar_init(tc::smem_u32(&drain_bar), 1);
    abort_s = 0;
    consumed_s = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(tc::smem_u32(&tmem_base_s), 512);
  pdl_wait();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  if (g.clear_status && blockIdx.x == 0 && threadIdx.x == 0) *g.status = 0u;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (tc::elect_one()) {
      int s = 0, issued = 0, withheld = -1;
      uint32_t ph = 0;
      for (int t = blockIdx.x; t < g.tiles && !*abort; t += gridDim.x) {
        const Tile tl = tile_at(g, t);
        const Problem& p = g.p[tl.pi];
        const int m0 = tl.m * kBM;
        const uint32_t bytes = (uint32_t)kTileA + (uint32_t)p.tn * 128u;
        for (int c = 0; c < p.nkc * p.segs; ++c) {
          if (!tc::mbar_wait(tc::smem_u32(&empty_bar[s]), ph ^ 1, abort, g.status)) break;
          if (*abort) break;   // a slot freed by an abort is not refilled
          if (tc::withheld_load(issued, blockIdx.x == 0)) {
            withheld = issued++;
          } else {
            const int seg = c >= p.nkc;
            const int k0 = (c - seg * p.nkc) * kBK;
            const uint32_t fb = tc::smem_u32(&full_bar[s]);
            const uint32_t sa = tc::smem_u32(smem + s * kStageBytes), sb = sa + kTileA;
            tc::mbar_arrive_expect_tx(fb, bytes);
            if (p.a_mn) {
              tc::tma_load_2d(sa, &p.a[seg], m0, k0, fb);
              tc::tma_load_2d(sa + 8192, &p.a[seg], m0 + 64, k0, fb);
            } else {
              tc::tma_load_2d(sa, &p.a[seg], k0, m0, fb);
            }
            if (p.pair) {
              const int nf = p.tn >> 1;
              tc::tma_load_2d(sb, &p.b[0], k0, tl.n * nf, fb);
              tc::tma_load_2d(sb + (uint32_t)nf * 128u, &p.b[1], k0, tl.n * nf, fb);
            } else if (p.b_mn) {
              for (int j = 0; j < p.tn / 64; ++j)
                tc::tma_load_2d(sb + 8192u * j, &p.b[seg], tl.n * p.tn + 64 * j, k0, fb);
            } else {
              tc::tma_load_2d(sb, &p.b[seg], k0, tl.n * p.tn, fb);
            }
            ++issued;
          }
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (*abort) {
        // Drain: wait (bounded, whatever the abort flag says) for the loads still in flight.
        int zero = 0;
        volatile int* never = &zero;
        for (int i = consumed_s; i < issued; ++i)
          if (i != withheld)
            tc::mbar_wait(tc::smem_u32(&full_bar[i % kStages]), (i / kStages) & 1, never, g.status);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (tc::elect_one()) {
      int s = 0, b = 0;
      uint32_t ph = 0, aph = 0;
      bool any = false;
      for (int t = blockIdx.x; t < g.tiles && !*abort; t += gridDim.x) {
        const Tile tl = tile_at(g, t);
        const Problem& p = g.p[tl.pi];
        const uint32_t idesc =
            tc::idesc_bf16_f32(kBM, p.tn) | ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16);
        const uint32_t astep = p.a_mn ? 128u : 2u, bstep = p.b_mn ? 128u : 2u;   // 16 k, in 16-byte units
        if (!tc::mbar_wait(tc::smem_u32(&tempty_bar[b]), aph ^ 1, abort, g.status)) break;
        tc::tc_fence_after();
        const uint32_t dt = tmem + (uint32_t)b * 256u;
        bool ok = true;
        const int chunks = p.nkc * p.segs;
        for (int c = 0; c < chunks; ++c) {
          if (!tc::mbar_wait(tc::smem_u32(&full_bar[s]), ph, abort, g.status)) {
            ok = false;
            break;
          }
          consumed_s = consumed_s + 1;
          tc::tc_fence_after();
          const uint32_t sa = tc::smem_u32(smem + s * kStageBytes), sb = sa + kTileA;
          const uint64_t ad = p.a_mn ? sdesc_mn_sw128(sa) : tc::sdesc_sw128(sa);
          const uint64_t bd = p.b_mn ? sdesc_mn_sw128(sb) : tc::sdesc_sw128(sb);
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j)
            tc::umma_bf16(dt, ad + j * astep, bd + j * bstep, idesc, (c | j) != 0);
          tc::umma_commit(tc::smem_u32(&empty_bar[s]));
          any = true;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        tc::umma_commit(tc::smem_u32(&tfull_bar[b]));
        if (++b == 2) {
          b = 0;
          aph ^= 1;
        }
      }
      if (*abort && any) {
        // Let every MMA issued so far finish before TMEM is released.
        tc::umma_commit(tc::smem_u32(&drain_bar));
        int zero = 0;
        volatile int* never = &zero;
        tc::mbar_wait(tc::smem_u32(&drain_bar), 0, never, g.status);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;                 // TMEM lane quarter this warp may read
    const int row = 32 * q + lane;
    int b = 0;
    uint32_t aph = 0;
    for (int t = blockIdx.x; t < g.tiles && !*abort; t += gridDim.x) {
      const Tile tl = tile_at(g, t);
      const Problem& p = g.p[tl.pi];
      if (!tc::mbar_wait(tc::smem_u32(&tfull_bar[b]), aph, abort, g.status)) break;
      tc::tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)b * 256u;
      const int m = tl.m * kBM + row;
      const bool valid = m < p.M;
      const int tn = p.pair ? p.tn >> 1 : p.tn;
      const int n0 = tl.n * tn, cols = min(tn, p.N - n0);
      uint16_t* orow = p.out + (size_t)m * p.N + n0;
      const size_t blk = ((size_t)tl.m * (p.N / 4) + n0 / 4) * 128 + row;   // saved g, u: float4 index
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
        tc::tmem_ld16(taddr + (uint32_t)c0, v);
        const int left = cols - c0;
        if (EPI == kEpiGlu) {
          float w[16];
          tc::tmem_ld16(taddr + (uint32_t)(tn + c0), w);
          if (valid) {
            if (g.g) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (4 * i < left) {
                  const size_t at = blk + (size_t)(c0 / 4 + i) * 128;
                  reinterpret_cast<float4*>(g.g)[at] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                  reinterpret_cast<float4*>(g.u)[at] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = glu_value(g.act, v[i], w[i]);
            store_bf16x16(orow + c0, v, left);
          }
        } else if (EPI == kEpiDact) {
          if (valid) {
            float du[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float4 gv = make_float4(0.f, 0.f, 0.f, 0.f), uv = gv;
              if (4 * i < left) {
                const size_t at = blk + (size_t)(c0 / 4 + i) * 128;
                gv = reinterpret_cast<const float4*>(g.g)[at];
                uv = reinterpret_cast<const float4*>(g.u)[at];
              }
              glu_grad(g.act, gv.x, uv.x, v[4 * i], v[4 * i], du[4 * i]);
              glu_grad(g.act, gv.y, uv.y, v[4 * i + 1], v[4 * i + 1], du[4 * i + 1]);
              glu_grad(g.act, gv.z, uv.z, v[4 * i + 2], v[4 * i + 2], du[4 * i + 2]);
              glu_grad(g.act, gv.w, uv.w, v[4 * i + 3], v[4 * i + 3], du[4 * i + 3]);
            }
            store_bf16x16(orow + c0, v, left);
            store_bf16x16(g.out2 + (size_t)m * p.N + n0 + c0, du, left);
          }
        } else if (valid) {
          store_bf16x16(orow + c0, v, left);
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&tempty_bar[b]));
      if (++b == 2) {
        b = 0;
        aph ^= 1;
      }
    }
  }

  pdl_trigger();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- host
bool map_bf16(CUtensorMap* m, const uint16_t* base, int rows, int cols, int box_rows) {
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, (uint64_t)rows, (uint64_t)cols, (uint64_t)cols * 2,
                  (uint32_t)box_rows, kBK, CU_TENSOR_MAP_SWIZZLE_128B);
}

int cdiv(int a, int b) { return (a + b - 1) / b; }

// Columns of B per tile: the widest of 256, 128, 64 (32) whose tiles still give every SM
// one.  `cols` output columns; a tile covers tn / per of them.
int pick_tn(int mt, int cols, int per, int least) {
  const int sms = sm_count();
  int tn = kMaxN;
  while (tn > least && (long long)mt * cdiv(cols, tn / per) < sms) tn >>= 1;
  return tn;
}

template <int EPI>
cudaError_t launch(GemmParams& g, cudaStream_t s) {
  static bool done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(glu_gemm_kernel<EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  g.tiles = 0;
  for (int i = 0; i < g.n_problems; ++i) g.tiles += g.p[i].mt * g.p[i].nt;
  const int sms = sm_count();
  return launch_pdl(glu_gemm_kernel<EPI>, dim3(g.tiles < sms ? g.tiles : sms), dim3(kThreads), kSmemBytes, s, g);
}

// D [M, N] = sum over segments of A_s B_s^T, k of length K in each.  a_mn / b_mn: the
// operand is stored [K, M] / [K, N].
bool set_problem(Problem& p, int M, int N, int K, const uint16_t* a0, const uint16_t* a1, bool a_mn,
                 const uint16_t* b0, const uint16_t* b1, bool b_mn, uint16_t* out) {
  p.M = M;
  p.N = N;
  p.nkc = cdiv(K, kBK);
  p.segs = a1 ? 2 : 1;
  p.pair = 0;
  p.a_mn = a_mn;
  p.b_mn = b_mn;
  p.mt = cdiv(M, kBM);
  p.tn = pick_tn(p.mt, N, 1, 64);
  p.nt = cdiv(N, p.tn);
  p.out = out;
  const uint16_t* a[2] = {a0, a1};
  const uint16_t* b[2] = {b0, b1};
  for (int i = 0; i < p.segs; ++i) {
    if (!(a_mn ? map_bf16(&p.a[i], a[i], K, M, 64) : map_bf16(&p.a[i], a[i], M, K, kBM))) return false;
    if (!(b_mn ? map_bf16(&p.b[i], b[i], K, N, 64) : map_bf16(&p.b[i], b[i], N, K, p.tn))) return false;
  }
  return true;
}

}  // namespace

cudaError_t launch_glu_gate_up(const GluParams& w, const uint16_t* x, int T, uint16_t* h, float* sg, float* su,
                               uint32_t* status, cudaStream_t s) {
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  g.n_problems = 1;
  Problem& p = g.p[0];
  p.M = T;
  p.N = w.ff;
  p.nkc = cdiv(w.d, kBK);
  p.segs = 1;
  p.pair = 1;
  p.mt = cdiv(T, kBM);
  p.tn = pick_tn(p.mt, w.ff, 2, 32);
  p.nt = cdiv(w.ff, p.tn / 2);
  p.out = h;
  if (!map_bf16(&p.a[0], x, T, w.d, kBM) || !map_bf16(&p.b[0], w.gate, w.ff, w.d, p.tn / 2) ||
      !map_bf16(&p.b[1], w.up, w.ff, w.d, p.tn / 2))
    return cudaErrorInvalidValue;
  g.act = GluAct{w.act, w.limit, w.alpha};
  g.g = sg;
  g.u = su;
  g.status = status;
  g.clear_status = 1;
  return launch<kEpiGlu>(g, s);
}

cudaError_t launch_glu_down(const GluParams& w, const uint16_t* h, int T, uint16_t* y, uint32_t* status,
                            cudaStream_t s) {
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  g.n_problems = 1;
  if (!set_problem(g.p[0], T, w.d, w.ff, h, nullptr, false, w.down, nullptr, false, y)) return cudaErrorInvalidValue;
  g.status = status;
  return launch<kEpiStore>(g, s);
}

cudaError_t launch_glu_dact(const GluParams& w, const uint16_t* dy, int T, const GluSaved& sv, uint16_t* dg,
                            uint16_t* du, uint32_t* status, cudaStream_t s) {
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  g.n_problems = 1;
  if (!set_problem(g.p[0], T, w.ff, w.d, dy, nullptr, false, w.down, nullptr, true, dg)) return cudaErrorInvalidValue;
  g.act = GluAct{w.act, w.limit, w.alpha};
  g.g = sv.g;
  g.u = sv.u;
  g.out2 = du;
  g.status = status;
  g.clear_status = 1;
  return launch<kEpiDact>(g, s);
}

cudaError_t launch_glu_grads(const GluParams& w, const uint16_t* x, const uint16_t* dy, int T, const GluSaved& sv,
                             const uint16_t* dg, const uint16_t* du, uint16_t* dx, uint16_t* dwg, uint16_t* dwu,
                             uint16_t* dwd, uint32_t* status, cudaStream_t s) {
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  bool ok = true;
  // the weights' gradients first: their sums over the tokens are the longest tiles
  if (dwg) ok = ok && set_problem(g.p[g.n_problems++], w.ff, w.d, T, dg, nullptr, true, x, nullptr, true, dwg);
  if (dwu) ok = ok && set_problem(g.p[g.n_problems++], w.ff, w.d, T, du, nullptr, true, x, nullptr, true, dwu);
  if (dwd) ok = ok && set_problem(g.p[g.n_problems++], w.d, w.ff, T, dy, nullptr, true, sv.h, nullptr, true, dwd);
  if (dx) ok = ok && set_problem(g.p[g.n_problems++], T, w.d, w.ff, dg, du, false, w.gate, w.up, true, dx);
  if (!ok) return cudaErrorInvalidValue;
  if (!g.n_problems) return cudaSuccess;
  g.status = status;
  return launch<kEpiStore>(g, s);
}

cudaError_t glu_set_wait_test(uint32_t polls, int withhold) { return tc::set_wait_test(polls, withhold); }

}  // namespace moe
