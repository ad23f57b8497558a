// The dense gated FFN on the 5th-generation tensor cores, its two forward products and
// the six of its backward pass, and the linear layer (moe_linear.h), all
// D[M x N] = A[M x K] . B[N x K]^T tiles with fp32 accumulators in TMEM, fed by TMA through an
// mbarrier ring.
//
//   gate/up:  g = x Wg^T, u = x Wu^T in one tile (the B tile holds tn / 2 rows of each), so
//             that the epilogue has both and writes h = act(g, u) (and, in training, g, u;
//             clamped ones near the border are settled there, with the rows' norms of a
//             launch before)
//   down:     y = h Wd^T
//   dact:     dh = dy Wd, whose epilogue turns it into dg and du with the saved g and u
//             (dh never reaches memory and is never rounded)
//             (dWd = dy^T h may ride along in that launch)
//   grads:    dx = dg Wg + du Wu (one sum over two runs of k), dWg = dg^T x and
//             dWu = du^T x in one launch, so that the tiles of the small products fill the
//             SMs that the large ones leave
//   linear:   act(x W^T + bias) + residual, or a gated layer's two halves as gate/up; bf16, or
//             e4m3 with a scale per row of x and of W (kind::f8f6f4; two values are moved as one
//             of 16 bits, so that a chunk is 128 of k in the same 128 bytes)
//   its gradients: dx = dv W and dW = dv^T x in one launch, with dv from linear_dv.cu
//
// An operand's k runs along its rows ("K-major": x Wg^T) or down its columns
// ("MN-major": both operands of dg^T x).  Both are read as they lie: a K-major tile is
// one box of 64 k (128 bytes, swizzled) per row, an MN-major one a box of 64 k rows per
// 64 columns; the tensor core's descriptors name the form.  Rows and columns past an
// edge are filled with zeros by the TMA unit, so d, ff and T need no padding.
//
// CG = 2: two CTAs of a cluster share one tile of 256 rows (cta_group::2).  Each holds its
// 128 rows of A and half of the B tile, and the accumulators of its rows; the tensor cores
// read the other half of B from the peer.  Against CG = 1 a chunk of 64 k moves 32 KiB
// into each SM instead of 48 KiB for the same MMAs (278 ns a chunk of 256 columns instead
// of 307), but a launch of pairs costs 1.4 us more, so that single CTAs serve short sums
// and few rows.
//
// SPLIT: when the tiles are too few for the SMs (few tokens), the 2, 4 or 8 CTAs of a
// cluster take consecutive parts of one tile's k.  Each CTA finishes a share of the columns:
// the others write their partial sums of these into its shared memory, and it adds them up
// in order (reading them from the others instead cost up to 5 us of round trips).
//
// parts (of a Problem): with many tokens and few weights the k of a weight gradient's tile is
// cut into parts that are units' work like tiles; the last part to end adds the sums up.
//
// Warp roles of the persistent CTA: warps 0 and 11 TMA producers; warp 1 owner of TMEM and,
// in the first CTA of a pair, MMA issuer (two accumulators of up to 256 columns, so that a tile's
// epilogue runs under the next tile's MMAs); warps 2..9 epilogue, two per TMEM lane
// quarter on alternate column chunks; warp 10 works out the coming tiles (list, divisions,
// cold reads of the constant bank: about 1700 clocks, in which the producers issued nothing
// and the MMAs ran dry) and leaves them in a ring for warps 0, 1 and 11; dact: warp 12 copies
// the saved g and u of the coming chunks into a shared-memory ring, since their latency
// would otherwise be paid at every chunk.  Every wait is bounded (see tc::mbar_wait).
//
// Measured at 8192 tokens, d 2048, ff 8192 (tensor cores under the power limit; a library's
// bf16 product reaches 1.87 PFLOP/s): gate/up 280 us (1.96 PFLOP/s; 325 with g and u kept,
// 0.5 GB), down 165 us (1.67: 256 tiles on 76 pairs), dact 211 us, grads with dWd 724 us
// (1.90).  At 4096, 2048, 512 the four launches take 20, 14, 19 and 32 us: one wave each,
// bound by the first loads' latency and the open epilogue.  Linear: 4096 x 2048 x 2048 25 us
// with its bias (1.37 PFLOP/s, one wave), 30 with SiLU, residual and v kept, its gradients 42.5
// (1.62); 8192 x 4096 x 4096 144 us (1.91), in 8 bits 79 (3.5); 8192 x 2880 x 8192 gated in 8 bits
// 220 to 245 us by the power limit (3.5 to 3.2 PFLOP/s).  16 epilogue warps with 16 columns
// at a time in place of 8 with 32 took 26.5 instead of 27.2 us with an activation, but 29.1
// instead of 27.9 with a residual, since a row's pieces are then 32 bytes.
#include <cuda.h>

#include <algorithm>
#include <cstring>
#include <utility>

#include "block.h"
#include "common.cuh"
#include "glu_act.cuh"
#include "linear_act.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kBM = 128, kBK = 64, kMaxN = 256;
constexpr int kTileA = kBM * kBK * 2;
constexpr int kMaxProblems = 4;
constexpr int kEpiWarps = 8, kProducer1 = 3 + kEpiWarps;

// The epilogue of a launch's first product (any others: kEpiStore).
enum : int { kEpiGlu = 0, kEpiStore = 1, kEpiDact = 2, kEpiLinear = 3, kEpiLinear8 = 4 };
__host__ __device__ constexpr bool is_linear(int epi) { return epi >= kEpiLinear; }

constexpr int kLinearCols = 128 * 8;   // bias and scale of 128 columns in fp32

constexpr int kMaxStages = 20;
constexpr int kInfos = 4;   // tiles worked out ahead

// Shared memory: the ring of operand stages (A 16 KiB | B rows of this CTA, as many as the
// launch's widest tile has, so that narrow tiles get more stages), then, for dact, kSlots
// slots of 16 columns of g and u (128 rows x 16 x 4 bytes each).
template <int EPI>
struct Lay {
  static constexpr int kSlots = EPI == kEpiDact ? 4 : 0;
  static constexpr int kRing = kSlots ? kSlots : 1;
  static constexpr int kSlotBytes = 2 * 128 * 16 * 4;
  // the linear layer's epilogue warps keep their columns' bias and scale behind the stages
  static constexpr int kStageSpace = is_linear(EPI) ? 216 * 1024 : 225 * 1024 - kSlots * kSlotBytes;
  static constexpr int kSmemBytes = kStageSpace + (is_linear(EPI) ? kEpiWarps * kLinearCols : kSlots * kSlotBytes) + 1024;
  static constexpr int kThreads = 32 * (4 + kEpiWarps + (EPI == kEpiDact ? 1 : 0));
};

// One product: D [M, N] over `segs` runs of `nkc` chunks of 64 k.  Run s multiplies
// a[s] and b[s]; with `pair` (gate/up) the B tile instead takes tn / 2 rows of b[0] and
// tn / 2 rows of b[1].
struct Problem {
  CUtensorMap a[2], b[2];
  int M, N;             // rows and columns of the output (pair: columns of h)
  int nkc, segs, pair;
  int a_mn, b_mn;       // 1: MN-major
  int a_blocks, b_blocks;   // MN-major, 1: maps of [block of 64][k][64], one load per chunk
  int tn;               // columns of B per tile (MMA N)
  int mt, nt;           // tiles (of 128 CG rows)
  int parts, base;      // of a tile's k, each a unit's work; tiles of the problems before it
  int wide;             // output rows and base allow 32-byte stores
  uint16_t* out;        // bf16 [M, N]
};

// Launches of several products list each unit's tiles (see list_tiles); the others give unit
// u the tiles u, u + units, ...
constexpr int kMaxListed = 2048, kMaxUnits = 160;

struct GemmParams {
  Problem p[kMaxProblems];
  int n_problems, tiles, listed;
  int stages, stage_bytes;   // of the ring
  uint16_t first[kMaxUnits + 1], list[kMaxListed];
  float4* partial;      // sums of the parts of split tiles (parts > 1)
  uint32_t* arrived;    // parts that have written theirs, per tile, CTA and epilogue warp
  int zeros;            // kEpiDact: so many of `arrived` to clear for the launch that splits
  GluAct act;
  float *g, *u;         // saved (kEpiGlu: written when non-null; kEpiDact: read)
  uint16_t* out2;       // kEpiDact: du (out: dg)
  // kEpiGlu, clamped, with g: clamp inputs nearer to their border than the sum may be off
  // (see border_gap) are computed again from these; norm: of the rows of x, wg and wu
  const uint16_t *x, *wg, *wu;
  int d;
  const float* norm;    // [M] | [N] | [N]; null where nothing is settled
  float gap;
  LinearEpi lin;        // kEpiLinear, kEpiLinear8
  int tile_a;           // and the bytes of a stage's rows of x: as many as there are, where fewer than 128
  BiasParts bias;       // kEpiStore: partial sums to add up on the way, or none
  uint32_t* status;
  int clear_status;     // this is the call's first kernel
};

struct Tile {
  int pi, m, n;
  int idx, part;   // within its problem; of its k
};

// Tiles run in groups of 8 m tiles: the CTAs working at one time share a few A tiles and
// a few B tiles through L2.
// PARTS: some products' k may be split over units.
template <bool PARTS>
__device__ __forceinline__ Tile tile_at(const GemmParams& g, int t) {
  Tile tl;
  tl.pi = 0;
  while (tl.pi + 1 < g.n_problems) {
    const int n = g.p[tl.pi].mt * g.p[tl.pi].nt * (PARTS ? g.p[tl.pi].parts : 1);
    if (t < n) break;
    t -= n;
    ++tl.pi;
  }
  const Problem& p = g.p[tl.pi];
  tl.part = 0;
  if (PARTS && p.parts > 1) {
    tl.part = t % p.parts;
    t /= p.parts;
  }
  tl.idx = t;
  constexpr int kGroup = 8;
  const int per = kGroup * p.nt;
  const int grp = t / per, r = t - grp * per;
  const int m0 = grp * kGroup, rows = min(kGroup, p.mt - m0);
  tl.n = r / rows;
  tl.m = m0 + (r - tl.n * rows);
  return tl;
}

// What the producer and the MMA issuer of a CTA need to know of a tile.
struct alignas(16) TileInfo {
  const CUtensorMap *a[2], *b[2];   // of either run of k (pair, CG 1: b of gate, of up)
  int m0, n0;                       // first row of A, of B
  int nkc, from, to;                // chunks of a run; those to take, over both runs (to 0: no tile is left)
  int half, boxes;                  // rows of gate, of up; boxes of an MN-major B
  uint32_t bytes, idesc;
  int a_mn, b_mn, a_blocks, b_blocks, two_b;
};

// The i-th tile of a unit, or -1.
__device__ __forceinline__ int nth_tile(const GemmParams& g, int unit, int units, int i) {
  if (g.listed) {
    i += g.first[unit];
    return i < g.first[unit + 1] ? g.list[i] : -1;
  }
  const long long t = unit + (long long)units * i;
  return t < g.tiles ? (int)t : -1;
}

// Four fp32 of shared memory as two pairs.
struct alignas(16) F2x2 {
  F2 a, b;
};

__device__ __forceinline__ uint32_t pack_pair(F2 v) {
  float lo, hi;
  split(v, lo, hi);
  return pack_bf16x2(lo, hi);
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

// 16 fp32 -> 16 bf16 at dst; cols: how many are in range, a multiple of 8; wide: dst is
// 32-byte aligned (one store per thread writes a whole sector).
__device__ __forceinline__ void store_bf16x16(uint16_t* dst, const float (&v)[16], int cols, bool wide) {
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  if (wide && cols > 8) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(q[0]), "r"(q[1]), "r"(q[2]),
                 "r"(q[3]), "r"(q[4]), "r"(q[5]), "r"(q[6]), "r"(q[7])
                 : "memory");
    return;
  }
  if (cols > 0) reinterpret_cast<uint4*>(dst)[0] = make_uint4(q[0], q[1], q[2], q[3]);
  if (cols > 8) reinterpret_cast<uint4*>(dst)[1] = make_uint4(q[4], q[5], q[6], q[7]);
}

__device__ __forceinline__ void pack16(const float (&v)[16], uint32_t* z) {
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
}

// A warp's 32 rows x 32 columns of bf16, a row per lane (z: 4 runs of 8 columns).  Every 4
// lanes exchange their runs, so that a store writes 64 bytes of each of 8 rows instead of a
// sector of each of 32: the stores hold up the next tile's operands less (2206 x 456 x 1000
// backward: 38.3 -> 37.3 us; 128 or 256 bytes of a row, and bulk stores, gained no more; the
// epilogues that compute keep a row per lane, since there the exchange cost what it gained).
// dst: the first row's first column; rows, cols: how many are in range (cols a multiple of 8).
__device__ __forceinline__ void store_32x32(uint16_t* dst, size_t pitch, uint32_t (&z)[16], int rows, int cols, int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool high = lane & bit;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & bit) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // run j of the odd lane for run j + bit of the even one
        uint32_t &lo = z[4 * j + i], &hi = z[4 * (j + bit) + i];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? lo : hi, bit);
        if (high) lo = got;
        else hi = got;
      }
    }
  }
  const int r0 = lane & ~3, c = 8 * (lane & 3);
  uint16_t* at = dst + (size_t)r0 * pitch + c;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (r0 + j < rows && c < cols)
      *reinterpret_cast<uint4*>(at + j * pitch) = make_uint4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
}

// 2 x 16 fp32 accumulator columns of this thread's row, at columns a and b.
__device__ __forceinline__ void tmem_ld_2x16(uint32_t a, uint32_t b, float (&v)[16], float (&w)[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a), "r"(b)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = __uint_as_float(r[i]);
    w[i] = __uint_as_float(r[16 + i]);
  }
}

// ---- the pair forms (PTX ISA, cta_group::2): operands and barriers of two CTAs
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The address of the same shared-memory location in the first CTA of the pair.
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Whether phase `parity` of `bar` is over, without waiting.
__device__ __forceinline__ bool mbar_over(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(done)
               : "r"(bar), "r"(parity)
               : "memory");
  return done != 0;
}

// A wait of a whole warp whose lanes go on together: each lane polls for itself, and one that
// sees the barrier's phase end while another sees the abort flag would leave the rest of the
// warp alone in the collective instructions that follow.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort, status));
}

template <int CG>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  if (CG == 1) {
    tc::tma_load_2d(dst, map, c0, c1, bar);
  } else {
    // into this CTA's shared memory, counted on a barrier of the pair's first CTA
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  }
}

// The same for a box of [blocks of 64 columns][64 k][64 columns]: k0, first block.
template <int CG>
__device__ __forceinline__ void load_blocks(uint32_t dst, const CUtensorMap* map, int k0, int block, uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(k0), "r"(block), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(k0), "r"(block), "r"(bar)
        : "memory");
}

// EIGHT: 32 bytes of k are 32 e4m3 values and not 16 bf16 ones.
template <int CG, bool EIGHT>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (EIGHT && CG == 1) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0;"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  } else if (EIGHT) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0;"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  } else if (CG == 1) {
    tc::umma_bf16(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0;"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// Arrive on `bar` (CG 2: in both CTAs) once every MMA issued so far has completed.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if (CG == 1) {
    tc::umma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  }
}

template <int CG>
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  if (CG == 1)
    tc::mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_leader(bar)) : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t dst) {
  if (CG == 1) {
    tc::tmem_alloc(dst, 512);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(dst) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}

template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr) {
  if (CG == 1)
    tc::tmem_dealloc(addr, 512);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(addr) : "memory");
}

// Plain copy of `bytes` (a multiple of 16) contiguous bytes into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// a + b as the rounded sum and what the rounding lost (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float& s, float& lost, float v) {
  const float t = __fadd_rn(s, v), z = __fsub_rn(t, s);
  lost = __fadd_rn(lost, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(v, z)));
  s = t;
}

// x . w over k by the whole warp: the products of bf16 values are exact in fp32, and the
// sums (four, whose additions do not wait for one another) keep what their roundings lose.
__device__ __noinline__ float exact_dot(const uint16_t* x, const uint16_t* w, int k, int lane) {
  float s[4] = {}, lost[4] = {};
  for (int i = 8 * lane; i < k; i += 1024) {
    uint4 a[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = i + 256 * j < k;
      a[j] = in ? *reinterpret_cast<const uint4*>(x + i + 256 * j) : make_uint4(0u, 0u, 0u, 0u);
      b[j] = in ? *reinterpret_cast<const uint4*>(w + i + 256 * j) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t av = e == 0 ? a[j].x : e == 1 ? a[j].y : e == 2 ? a[j].z : a[j].w;
        const uint32_t bv = e == 0 ? b[j].x : e == 1 ? b[j].y : e == 2 ? b[j].z : b[j].w;
        two_sum(s[j], lost[j], __fmul_rn(bf16_lo(av), bf16_lo(bv)));
        two_sum(s[j], lost[j], __fmul_rn(bf16_hi(av), bf16_hi(bv)));
      }
  }
#pragma unroll
  for (int j = 1; j < 4; ++j) {
    two_sum(s[0], lost[0], s[j]);
    lost[0] = __fadd_rn(lost[0], lost[j]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, s[0], o), l = __shfl_xor_sync(0xffffffffu, lost[0], o);
    two_sum(s[0], lost[0], other);
    lost[0] = __fadd_rn(lost[0], l);
  }
  return __fadd_rn(__shfl_sync(0xffffffffu, s[0], 0), __shfl_sync(0xffffffffu, lost[0], 0));
}

// How far the tensor cores' sum of x . w may be from the exact one near the clamp's border.
// They truncate the sum at every step of 16 products, by at most 2^-23 of the larger of the
// sum and the products (taken from measurements: the instruction's documents leave the
// rounding open).  By Cauchy and Schwarz a sum S_i of the first i products is at most
// p_i = |x[:i]| |w[:i]|, and, since the whole sum is near the limit L, at most L + q_i, q_i
// that of the products still to come; p_i + q_i <= |x| |w|.  So |S_i| <= (|x| |w| + L) / 2, and
// all steps together are off by at most (d / 16) 2^-24 (|x| |w| + L); `gap` is that factor,
// with 9 steps more for the rounding of the norms and, in split tiles, of the parts' sum.
// Measured at d 72 to 8192: at most 0.54 of it, where the first products alone make the sum
// (half of 2^-23 on average at each step), 0.26 for terms of one sign, 0.13 where large terms
// cancel, 0.08 for random operands (0.006 at d 2880).  A fixed share of the limit, without the
// norms, let values cross the border whose terms cancel, or with a limit below the terms'
// size.  Rows of zeros have no gap and no error.
__device__ __forceinline__ float border_gap(const GemmParams& g, float x_norm, float w_norm) {
  return g.gap * fmaf(x_norm, w_norm, x_norm > 0.f ? g.act.limit : 0.f);
}

// Whether v, at a distance from its border, is nearer than gap.  A gap that is infinite or NaN
// belongs to a row or feature whose sums are, or leave fp32's range on the way.
__device__ __forceinline__ bool nearer(float distance, float gap) { return distance < gap && gap < 3.0e38f; }

// Values of a clamp's input nearer to its border than that, one per lane: computed again, so
// that the backward pass takes the side that the exact value takes.  row0: the warp's
// first row.
__device__ __forceinline__ void settle(float& v, bool near, const uint16_t* x, const uint16_t* w, int k, int row0,
                                       int lane) {
  unsigned todo = __ballot_sync(0xffffffffu, near);
  while (todo) {
    const int l = __ffs(todo) - 1;
    todo &= todo - 1;
    const float r = exact_dot(x + (size_t)(row0 + l) * k, w, k, lane);
    if (lane == l) v = r;
  }
}

// The address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}

// 8 finished columns of one row of a split tile: the sums v (gate/up: v gate, w up).
template <int EPI>
__device__ __forceinline__ void finish8(const GemmParams& g, const Problem& p, int mb, int row, int n, float (&v)[8],
                                        float (&w)[8]) {
  const bool clamped = g.act.act == MOE_ACT_CLAMPED_GLU;
  const int m = mb * kBM + row, lane = row & 31;
  const bool valid = m < p.M;
  const size_t blk = ((size_t)mb * (p.N / 4) + n / 4) * 128 + row;   // saved g, u: float4 index
  if (EPI == kEpiGlu) {
    if (g.norm) {
      const float xn = valid ? g.norm[m] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const size_t f = (size_t)(n + i) * g.d;
        settle(v[i], nearer(fabsf(v[i] - g.act.limit), border_gap(g, xn, g.norm[p.M + n + i])), g.x, g.wg + f, g.d, m - lane, lane);
        settle(w[i], nearer(fabsf(fabsf(w[i]) - g.act.limit), border_gap(g, xn, g.norm[p.M + p.N + n + i])), g.x, g.wu + f,
               g.d, m - lane, lane);
      }
    }
    if (!valid) return;
    if (g.g) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        reinterpret_cast<float4*>(g.g)[blk + 128 * i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        reinterpret_cast<float4*>(g.u)[blk + 128 * i] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = glu_value(g.act, v[i], w[i]);
  } else if (EPI == kEpiDact) {
    if (!valid) return;
    float gv[8], uv[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<float4*>(gv + 4 * i) = reinterpret_cast<const float4*>(g.g)[blk + 128 * i];
      *reinterpret_cast<float4*>(uv + 4 * i) = reinterpret_cast<const float4*>(g.u)[blk + 128 * i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (clamped) glu_grad<true>(g.act, gv[i], uv[i], v[i], v[i], w[i]);
      else glu_grad<false>(g.act, gv[i], uv[i], v[i], v[i], w[i]);
    }
    *reinterpret_cast<uint4*>(g.out2 + (size_t)m * p.N + n) =
        make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7]));
  }
  if constexpr (is_linear(EPI)) {
    if (!valid) return;
    constexpr bool kEight = EPI == kEpiLinear8;
    const float xs = kEight ? g.lin.x_scale[m] : 1.f;
    const size_t at = (size_t)m * p.N + n;
    F2 a[4] = {f2(v[0], v[1]), f2(v[2], v[3]), f2(v[4], v[5]), f2(v[6], v[7])};
    linear_affine8<kEight>(g.lin, xs, n, a);
    if (p.pair) {
      F2 u[4] = {f2(w[0], w[1]), f2(w[2], w[3]), f2(w[4], w[5]), f2(w[6], w[7])};
      linear_affine8<kEight>(g.lin, xs, p.N + n, u);
      gated_values(g.lin.gated, a, u);
    } else {
      if (g.lin.pre) *reinterpret_cast<uint4*>(g.lin.pre + at) = pack8(a);
      linear_values(g.lin.act, a);
    }
    if (g.lin.residual) {
      F2 r[4];
      unpack8(*reinterpret_cast<const uint4*>(g.lin.residual + at), r);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = add2(a[i], r[i]);
    }
    *reinterpret_cast<uint4*>(p.out + at) = pack8(a);
    return;
  }
  if (valid)
    *reinterpret_cast<uint4*>(p.out + (size_t)m * p.N + n) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

template <int CG, int EPI, bool SPLIT>
__global__ void __launch_bounds__(Lay<EPI>::kThreads, 1) glu_gemm_kernel(const __grid_constant__ GemmParams g) {
  using L = Lay<EPI>;
  const int kStages = g.stages, kStageBytes = g.stage_bytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tc::smem_align1024(smem_raw);
  __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ __align__(8) uint64_t sfull_bar[L::kRing], sempty_bar[L::kRing];
  __shared__ __align__(8) uint64_t ifull_bar[kInfos], iempty_bar[kInfos];
  __shared__ TileInfo infos[kInfos];
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)cluster_rank() : 0;
  // SPLIT: a cluster is a unit with one tile, of which this CTA takes part `part`
  const int parts = SPLIT ? (int)cluster_size() : 1, part = SPLIT ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / (CG * parts), units = gridDim.x / (CG * parts);
  volatile int* abort = &abort_s;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(tc::smem_u32(&full_bar[s]), 1);
      tc::mbar_init(tc::smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tc::smem_u32(&tfull_bar[b]), 1);
      tc::mbar_init(tc::smem_u32(&tempty_bar[b]), kEpiWarps * CG);
    }
    for (int s = 0; s < L::kSlots; ++s) {
      tc::mbar_init(tc::smem_u32(&sfull_bar[s]), 1);
      tc::mbar_init(tc::smem_u32(&sempty_bar[s]), kEpiWarps / 2);
    }
    for (int i = 0; i < kInfos; ++i) {
      tc::mbar_init(tc::smem_u32(&ifull_bar[i]), 1);
      tc::mbar_init(tc::smem_u32(&iempty_bar[i]), rank == 0 ? 3 : 2);   // the producers and the issuer
    }
    tc::mbar_init(tc::smem_u32(&drain_bar), 1);
    abort_s = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) tmem_alloc<CG>(tc::smem_u32(&tmem_base_s));
  tc::tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();   // the peer's barriers and TMEM are ready
  if (SPLIT) cluster_arrive();   // this CTA runs: the others may write to it
  bool all_run = false;
  tc::tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  // Each role waits for the kernel before this one only where it first touches global
  // memory: the barriers, TMEM and the first tile's parameters (cold reads of the constant
  // bank: about 1 us) are then ready.

  if (warp == 0 || warp == kProducer1) {
    // ---------------------------------------------------------------- TMA producers
    // A thread takes about 390 clocks for a chunk's loads and barriers, although all that it
    // needs is in registers and it asks for its next stage before the loads go out: less
    // than the MMAs of a 256-column tile (512), more than those of a narrow one.  So two
    // take the chunks in turn.
    if (tc::elect_one()) {
      const int me = warp == 0 ? 0 : 1;
      bool free = true;   // this producer's next stage is
      int s = 0, issued = 0, withheld = tc::withheld_load(0, blockIdx.x == 0) ? 0 : -1;
      uint32_t ph = 0;
      const uint32_t full0 = tc::smem_u32(&full_bar[0]), empty0 = tc::smem_u32(&empty_bar[0]);
      const uint32_t lead0 = CG == 2 ? in_leader(full0) : full0, stage0 = tc::smem_u32(smem);
      for (int nth = 0; !*abort; ++nth) {
        if (!tc::mbar_wait(tc::smem_u32(&ifull_bar[nth % kInfos]), (nth / kInfos) & 1, abort, g.status)) break;
        const TileInfo in = infos[nth % kInfos];
        tc::mbar_arrive(tc::smem_u32(&iempty_bar[nth % kInfos]));
        if (nth == 0) {
          pdl_wait();
          if (g.clear_status && blockIdx.x == 0 && me == 0) *g.status = 0u;
        }
        if (in.to == 0) break;
        const bool a_mn = in.a_mn, b_mn = in.b_mn, a_blocks = in.a_blocks, b_blocks = in.b_blocks, two_b = in.two_b;
        const int m0 = in.m0, n0 = in.n0, half = in.half, boxes = in.boxes;
        const uint32_t bytes = in.bytes;
        bool ok = true;
        for (int seg = 0; seg < 2 && ok; ++seg) {
          const CUtensorMap *ma = seg ? in.a[1] : in.a[0], *mb = seg ? in.b[1] : in.b[0], *mb1 = in.b[1];
          const int c0 = max(in.from - seg * in.nkc, 0), c1 = min(in.to - seg * in.nkc, in.nkc);
          for (int c = c0, k0 = c0 * kBK; c < c1; ++c, k0 += kBK) {
            if ((issued & 1) == me) {
              if (!free && !tc::mbar_wait(empty0 + 8u * s, ph ^ 1, abort, g.status)) {
                ok = false;
                break;
              }
              const uint32_t fb = lead0 + 8u * s, sa = stage0 + (uint32_t)s * kStageBytes, sb = sa + (is_linear(EPI) ? (uint32_t)g.tile_a : kTileA);
              const bool now = issued != withheld;
              if (now && rank == 0) tc::mbar_arrive_expect_tx(full0 + 8u * s, bytes);   // the peer's loads count here too
              const bool wraps = s + 2 >= kStages;
              free = mbar_over(empty0 + 8u * (wraps ? s + 2 - kStages : s + 2), ph ^ (wraps ? 0 : 1));
              if (now) {
                if (a_blocks) {
                  load_blocks<CG>(sa, ma, k0, m0 >> 6, fb);
                } else if (a_mn) {
                  load_tile<CG>(sa, ma, m0, k0, fb);
                  load_tile<CG>(sa + 8192, ma, m0 + 64, k0, fb);
                } else {
                  load_tile<CG>(sa, ma, k0, m0, fb);
                }
                if (b_blocks) {
                  load_blocks<CG>(sb, mb, k0, n0 >> 6, fb);
                } else if (b_mn) {
                  for (int j = 0; j < boxes; ++j) load_tile<CG>(sb + 8192u * j, mb, n0 + 64 * j, k0, fb);
                } else {
                  load_tile<CG>(sb, mb, k0, n0, fb);
                  if (two_b) load_tile<CG>(sb + (uint32_t)half * 128u, mb1, k0, n0, fb);
                }
              }
            }
            if (++s == kStages) {
              s = 0;
              ph ^= 1;
            }
            ++issued;
          }
        }
        if (!ok) break;
      }
      if (*abort && rank == 0) {
        // Drain: wait (bounded, whatever the abort flag says) for the last load of each
        // stage; the peer's are counted on the same barriers, and the cluster barrier at
        // the end keeps it here meanwhile.
        int zero = 0;
        volatile int* never = &zero;
        for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
          if ((i & 1) == me && i != withheld) tc::mbar_wait(full0 + 8u * (i % kStages), (i / kStages) & 1, never, g.status);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (rank == 0 && tc::elect_one()) {
      int s = 0, b = 0;
      uint32_t ph = 0, aph = 0;
      bool any = false, full = false;   // stage s is (asked for before the MMAs of the one before)
      const uint32_t full0 = tc::smem_u32(&full_bar[0]), empty0 = tc::smem_u32(&empty_bar[0]);
      const uint32_t stage0 = tc::smem_u32(smem);
      for (int nth = 0; !*abort; ++nth) {
        if (!tc::mbar_wait(tc::smem_u32(&ifull_bar[nth % kInfos]), (nth / kInfos) & 1, abort, g.status)) break;
        const TileInfo& in = infos[nth % kInfos];
        const bool a_mn = in.a_mn, b_mn = in.b_mn;
        const uint32_t idesc = in.idesc;
        const int chunks = in.to - in.from;
        tc::mbar_arrive(tc::smem_u32(&iempty_bar[nth % kInfos]));
        if (chunks == 0) break;
        const uint32_t astep = a_mn ? 128u : 2u, bstep = b_mn ? 128u : 2u;   // 16 k, in 16-byte units
        const uint64_t ad0 = a_mn ? sdesc_mn_sw128(stage0) : tc::sdesc_sw128(stage0);
        const uint32_t stage_b = stage0 + (is_linear(EPI) ? (uint32_t)g.tile_a : kTileA);
        const uint64_t bd0 = b_mn ? sdesc_mn_sw128(stage_b) : tc::sdesc_sw128(stage_b);
        if (!tc::mbar_wait(tc::smem_u32(&tempty_bar[b]), aph ^ 1, abort, g.status)) break;
        tc::tc_fence_after();
        const uint32_t dt = tmem + (uint32_t)b * 256u;
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
          if (!full && !tc::mbar_wait(full0 + 8u * s, ph, abort, g.status)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint64_t ad = ad0 + (uint32_t)s * (kStageBytes >> 4), bd = bd0 + (uint32_t)s * (kStageBytes >> 4);
          const uint32_t done = empty0 + 8u * s;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
          full = mbar_over(full0 + 8u * s, ph);
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j) mma<CG, EPI == kEpiLinear8>(dt, ad + j * astep, bd + j * bstep, idesc, (c | j) != 0);
          commit<CG>(done);
          any = true;
        }
        if (!ok) break;
        commit<CG>(tc::smem_u32(&tfull_bar[b]));
        if (++b == 2) {
          b = 0;
          aph ^= 1;
        }
      }
      if (*abort && any) {
        // Let every MMA issued so far finish before TMEM is released.
        commit<CG>(tc::smem_u32(&drain_bar));
        int zero = 0;
        volatile int* never = &zero;
        tc::mbar_wait(tc::smem_u32(&drain_bar), 0, never, g.status);
      }
    }
  } else if (warp == 2 + kEpiWarps) {
    // ---------------------------------------------------------------- the coming tiles
    if (tc::elect_one()) {
      for (int nth = 0, t = 0; t >= 0 && !*abort; ++nth) {
        t = nth_tile(g, unit, units, nth);
        TileInfo in;
        in.to = in.from = 0;
        if (t >= 0) {
          const Tile tl = tile_at<EPI == kEpiStore && !SPLIT>(g, t);
          const Problem& p = g.p[tl.pi];
          const int brows = p.tn / CG;   // rows of B in this CTA
          for (int i = 0; i < 2; ++i) {
            in.a[i] = &p.a[i];
            in.b[i] = &p.b[p.pair && CG == 2 ? rank : i];   // a pair of CTAs: one takes gate, one up
          }
          in.half = p.tn >> 1;
          in.m0 = (tl.m * CG + rank) * kBM;
          in.n0 = p.pair ? tl.n * in.half : tl.n * p.tn + rank * brows;
          in.a_mn = p.a_mn;
          in.b_mn = p.b_mn;
          in.a_blocks = p.a_blocks;
          in.b_blocks = p.b_blocks;
          in.two_b = CG == 1 && p.pair;
          in.boxes = in.b_mn ? (brows + 63) / 64 : 0;
          in.bytes = CG * ((is_linear(EPI) ? (uint32_t)g.tile_a : (uint32_t)kTileA) + (in.b_mn ? (uint32_t)in.boxes * 8192u : (uint32_t)brows * 128u));
          in.idesc = (EPI == kEpiLinear8 ? tc::idesc_e4m3_f32(kBM * CG, p.tn) : tc::idesc_bf16_f32(kBM * CG, p.tn)) | ((uint32_t)in.a_mn << 15) | ((uint32_t)in.b_mn << 16);
          in.nkc = p.nkc;
          const int all = p.nkc * p.segs;
          const int pt = SPLIT ? part : tl.part, pts = SPLIT ? parts : EPI == kEpiStore ? p.parts : 1;
          in.from = all * pt / pts;
          in.to = all * (pt + 1) / pts;
        }
        if (!tc::mbar_wait(tc::smem_u32(&iempty_bar[nth % kInfos]), (nth / kInfos & 1) ^ 1, abort, g.status)) break;
        infos[nth % kInfos] = in;
        tc::mbar_arrive(tc::smem_u32(&ifull_bar[nth % kInfos]));
      }
    }
  } else if (EPI == kEpiDact && warp == 4 + kEpiWarps) {
    // ---------------------------------------------------------------- saved g, u
    // 16 columns of the CTA's 128 rows are 8 KiB of g and 8 KiB of u, contiguous each.
    if (!SPLIT && tc::elect_one()) {
      int slot = 0, filled = 0;
      uint32_t ph = 0;
      for (int nth = 0, t; (t = nth_tile(g, unit, units, nth)) >= 0 && !*abort; ++nth) {
        const Tile tl = tile_at<EPI == kEpiStore && !SPLIT>(g, t);
        const Problem& p = g.p[tl.pi];
        if (nth == 0) pdl_wait();
        if (tl.pi) continue;
        const int mb = tl.m * CG + rank;
        const int n0 = tl.n * p.tn, cols = min(p.tn, p.N - n0);
        for (int c0 = 0; c0 < cols; c0 += 16) {
          if (!tc::mbar_wait(tc::smem_u32(&sempty_bar[slot]), ph ^ 1, abort, g.status) || *abort) break;
          const uint32_t fb = tc::smem_u32(&sfull_bar[slot]);
          if (mb * kBM < p.M) {
            const uint32_t n = (uint32_t)min(16, cols - c0) * 512u;
            const size_t at = ((size_t)mb * p.N + n0 + c0) * 128;   // floats
            const uint32_t dst = tc::smem_u32(smem + kStages * kStageBytes + slot * L::kSlotBytes);
            tc::mbar_arrive_expect_tx(fb, 2 * n);
            bulk_load(dst, g.g + at, n, fb);
            bulk_load(dst + L::kSlotBytes / 2, g.u + at, n, fb);
          } else {
            tc::mbar_arrive(fb);   // a tile row block past the last token
          }
          ++filled;
          if (++slot == L::kSlots) {
            slot = 0;
            ph ^= 1;
          }
        }
      }
      if (*abort) {
        int zero = 0;
        volatile int* never = &zero;
        for (int i = filled > L::kSlots ? filled - L::kSlots : 0; i < filled; ++i)
          tc::mbar_wait(tc::smem_u32(&sfull_bar[i % L::kRing]), (i / L::kRing) & 1, never, g.status);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;                 // TMEM lane quarter this warp may read
    const int par = (warp - 2) >> 2;        // takes column chunks of this parity
    const int row = 32 * q + lane;
    const bool clamped = g.act.act == MOE_ACT_CLAMPED_GLU;
    int b = 0, sl = 0;                      // sl: dact, chunks seen (slot sl % kSlots)
    uint32_t aph = 0;
    if (EPI == kEpiStore && g.bias.parts) {
      // a linear layer's bias gradient, under the first tile's MMAs
      pdl_wait();
      bias_sums(g.bias, blockIdx.x * kEpiWarps + warp - 2, gridDim.x * kEpiWarps, lane);
    }
    for (int nth = 0, t; (t = nth_tile(g, unit, units, nth)) >= 0 && __all_sync(0xffffffffu, !*abort); ++nth) {
      const Tile tl = tile_at<EPI == kEpiStore && !SPLIT>(g, t);
      const Problem& p = g.p[tl.pi];
      const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)b * 256u;
      const int mb = tl.m * CG + rank;
      const int m = mb * kBM + row;
      const bool valid = m < p.M, wide = p.wide;
      const int tn = p.pair ? p.tn >> 1 : p.tn;
      const int n0 = tl.n * tn, cols = min(tn, p.N - n0);
      uint16_t* orow = p.out + (size_t)m * p.N + n0;
      if (nth == 0) {
        pdl_wait();
        if (EPI == kEpiDact && blockIdx.x == 0)
          for (int i = threadIdx.x - 64; i < g.zeros; i += 32 * kEpiWarps) g.arrived[i] = 0u;
      }
      // The norms that the border's gaps depend on, asked for under the tile's MMAs: of this
      // lane's row of x, and of this warp's chunks of columns (at most 4) of gate's row of
      // column i in lane i, of up's in lane 16 + i.  A feature whose own sums are not finite
      // has none, so that the widest gap is the others'.
      float xn = 0.f, wn[4] = {};
      if (EPI == kEpiGlu && !SPLIT && g.norm) {
        if (valid) xn = g.norm[m];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = 16 * par + 32 * k + (lane & 15);
          const float n = c < cols ? g.norm[p.M + (lane & 16 ? p.N : 0) + n0 + c] : 0.f;
          wn[k] = n < 3.0e38f ? n : 0.f;
        }
      }
      // Linear layer, asked for under the tile's MMAs as well: bias and scale of this warp's
      // columns, 4 to a lane in the order of its chunks (gated: the gate's, then the up's); the
      // row's scale; and the residual of the first chunk (then always the next one's).
      uint2 lin_bias = make_uint2(0u, 0u);
      float4 lin_scale = make_float4(0.f, 0.f, 0.f, 0.f);
      float xs = 1.f;
      uint4 res[4] = {};
      const uint16_t* rrow = is_linear(EPI) && !SPLIT && g.lin.residual ? g.lin.residual + (size_t)m * p.N + n0 : nullptr;
      auto ask = [&](int c0) {
        if (!rrow || !valid) return;
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if ((h < 2 || !p.pair) && c0 + 8 * h < cols) res[h] = *reinterpret_cast<const uint4*>(rrow + c0 + 8 * h);
      };
      F2* mine_cols = nullptr;
      if (is_linear(EPI) && !SPLIT) {
        mine_cols = reinterpret_cast<F2*>(smem + L::kStageSpace + (warp - 2) * kLinearCols);
        const int l = lane & 15;
        const int c = p.pair ? 32 * (l >> 2) + 16 * par + 4 * (l & 3) : 64 * (lane >> 3) + 32 * par + 4 * (lane & 7);
        const int wr = n0 + c + (p.pair && lane >= 16 ? p.N : 0);
        if (c < cols) {
          if (g.lin.bias) lin_bias = __ldg(reinterpret_cast<const uint2*>(g.lin.bias + wr));
          if (EPI == kEpiLinear8) lin_scale = __ldg(reinterpret_cast<const float4*>(g.lin.w_scale + wr));
        }
        if (EPI == kEpiLinear8 && valid) xs = g.lin.x_scale[m];
        ask((p.pair ? 16 : 32) * par);
        if (rrow && valid)   // the later chunks' into L2
          for (int c0 = (p.pair ? 48 : 96) - (p.pair ? 16 : 32) * (1 - par); c0 < cols; c0 += p.pair ? 32 : 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(rrow + c0));
      }
      if (!warp_wait(tc::smem_u32(&tfull_bar[b]), aph, abort, g.status)) break;
      tc::tc_fence_after();
      if (SPLIT) {
        // every 8 columns to the CTA that finishes them: [its share][part][8 (pair: 16)][row]
        cluster_wait();
        all_run = true;
        const uint32_t ex = tc::smem_u32(smem) + (uint32_t)(kStages * kStageBytes + 4 * row);
        const bool pairs = EPI == kEpiGlu || (is_linear(EPI) && p.pair);
        const int shares = tn / 8, each = pairs ? 16 : 8;
        if (m - lane < p.M)   // of a row block past the last row nothing is needed
          for (int c0 = 16 * par; c0 < p.tn; c0 += 32) {
            float v[16];
            tc::tmem_ld16(taddr + (uint32_t)c0, v);
            const int up = pairs && c0 >= tn, c = up ? c0 - tn : c0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int u = c / 8 + k, owner = ((u + 1) * parts - 1) / shares, nth_of = u - shares * owner / parts;
              const uint32_t to =
                  in_cta(ex + (uint32_t)(((nth_of * parts + part) * each + 8 * up) * kBM * 4), (uint32_t)owner);
#pragma unroll
              for (int i = 0; i < 8; ++i) st_cluster(to + (uint32_t)(i * kBM * 4), v[8 * k + i]);
            }
          }
      } else if (EPI == kEpiGlu) {
        const size_t blk = ((size_t)mb * (p.N / 4) + n0 / 4) * 128 + row;   // saved g, u: float4 index
        for (int c0 = 16 * par; c0 < cols; c0 += 32) {
          float v[16], w[16];
          tmem_ld_2x16(taddr + (uint32_t)c0, taddr + (uint32_t)(tn + c0), v, w);
          const int left = cols - c0;
          if (g.norm) {
            // against the widest gap of the 32 columns first
            const float lim = g.act.limit, top = border_gap(g, xn, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(wn[0]))));
            bool any = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) any |= fabsf(v[i] - lim) < top || fabsf(fabsf(w[i]) - lim) < top;
            if (__any_sync(0xffffffffu, any)) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float gn = __shfl_sync(0xffffffffu, wn[0], i), un = __shfl_sync(0xffffffffu, wn[0], 16 + i);
                const bool in = i < left;
                const size_t f = (size_t)(n0 + c0 + i) * g.d;
                settle(v[i], in && nearer(fabsf(v[i] - lim), border_gap(g, xn, gn)), g.x, g.wg + f, g.d, m - lane, lane);
                settle(w[i], in && nearer(fabsf(fabsf(w[i]) - lim), border_gap(g, xn, un)), g.x, g.wu + f, g.d, m - lane, lane);
              }
            }
          }
          wn[0] = wn[1], wn[1] = wn[2], wn[2] = wn[3];   // the next chunk's
          if (valid) {
            if (g.g) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (4 * i < left) {
                  const size_t at = blk + (size_t)(c0 / 4 + i) * 128;
                  __stcs(reinterpret_cast<float4*>(g.g) + at, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                  __stcs(reinterpret_cast<float4*>(g.u) + at, make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
                }
            }
            if (clamped) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = glu_value<true>(g.act, v[i], w[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = glu_value<false>(g.act, v[i], w[i]);
            }
            store_bf16x16(orow + c0, v, left, wide);
          }
        }
      } else if constexpr (is_linear(EPI)) {
        constexpr bool kEight = EPI == kEpiLinear8;
        __syncwarp();
        mine_cols[2 * lane] = f2(bf16_lo(lin_bias.x), bf16_hi(lin_bias.x));
        mine_cols[2 * lane + 1] = f2(bf16_lo(lin_bias.y), bf16_hi(lin_bias.y));
        if (kEight) *reinterpret_cast<float4*>(mine_cols + 64 + 2 * lane) = lin_scale;
        __syncwarp();
        const int rows = p.M - (m - lane);
        // 2 N columns of the parameters' place i on
        auto affine = [&](int i, auto& v) {
#pragma unroll
          for (int j = 0; j < (int)(sizeof(v) / sizeof(F2)); j += 2) {
            const F2x2 bias = *reinterpret_cast<const F2x2*>(mine_cols + (i >> 1) + j);
            if (kEight) {
              const F2x2 scale = *reinterpret_cast<const F2x2*>(mine_cols + 64 + (i >> 1) + j);
              v[j] = fma2(mul2(v[j], f2(xs)), scale.a, bias.a);   // (the scales' product could underflow)
              v[j + 1] = fma2(mul2(v[j + 1], f2(xs)), scale.b, bias.b);
            } else {
              v[j] = add2(v[j], bias.a);
              v[j + 1] = add2(v[j + 1], bias.b);
            }
          }
        };
        if (p.pair) {
          for (int c0 = 16 * par, i = 0; c0 < cols; c0 += 32, i += 16) {
            const uint4 now[2] = {res[0], res[1]};
            ask(c0 + 32);
            float x[16], y[16];
            tmem_ld_2x16(taddr + (uint32_t)c0, taddr + (uint32_t)(tn + c0), x, y);
            F2 v[8], u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[j] = f2(x[2 * j], x[2 * j + 1]);
              u[j] = f2(y[2 * j], y[2 * j + 1]);
            }
            affine(i, v);
            affine(64 + i, u);
            gated_values(g.lin.gated, v, u);
            if (rrow) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                F2 r[4];
                unpack8(now[h], r);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * h + j] = add2(v[4 * h + j], r[j]);
              }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) split(v[j], x[2 * j], x[2 * j + 1]);
            if (valid) store_bf16x16(orow + c0, x, cols - c0, wide);
          }
        } else {
          for (int c0 = 32 * par, i = 0; c0 < cols; c0 += 64, i += 32) {
            const uint4 now[4] = {res[0], res[1], res[2], res[3]};
            ask(c0 + 64);
            float x[16], y[16];
            tmem_ld_2x16(taddr + (uint32_t)c0, taddr + (uint32_t)(c0 + 16), x, y);
            F2 v[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[j] = f2(x[2 * j], x[2 * j + 1]);
              v[8 + j] = f2(y[2 * j], y[2 * j + 1]);
            }
            affine(i, v);
            uint32_t z[16];
            if (g.lin.pre) {
#pragma unroll
              for (int j = 0; j < 16; ++j) z[j] = pack_pair(v[j]);
              store_32x32(g.lin.pre + (size_t)(m - lane) * p.N + n0 + c0, p.N, z, rows, cols - c0, lane);
            }
            linear_values(g.lin.act, v);
            if (rrow) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                F2 r[4];
                unpack8(now[h], r);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * h + j] = add2(v[4 * h + j], r[j]);
              }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] = pack_pair(v[j]);
            store_32x32(orow + c0 - (size_t)lane * p.N, p.N, z, rows, cols - c0, lane);
          }
        }
      } else if (EPI == kEpiDact && tl.pi == 0) {
        const int n_chunks = (cols + 15) / 16;
        for (int j = 0; j < n_chunks; ++j) {
          const int n = sl + j;
          if ((n & 1) != par) continue;
          const int slot = n % L::kRing, c0 = 16 * j;
          float v[16], du[16];
          tc::tmem_ld16(taddr + (uint32_t)c0, v);
          if (!warp_wait(tc::smem_u32(&sfull_bar[slot]), (n / L::kRing) & 1, abort, g.status)) break;
          const float4* gs = reinterpret_cast<const float4*>(smem + kStages * kStageBytes + slot * L::kSlotBytes) + row;
          const float4* us = gs + L::kSlotBytes / 32;
          const int left = cols - c0;
          float gv[16], uv[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // past the last column the slot holds old values, not stored
            *reinterpret_cast<float4*>(gv + 4 * i) = gs[128 * i];
            *reinterpret_cast<float4*>(uv + 4 * i) = us[128 * i];
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sempty_bar[slot]));
          if (valid) {
            if (clamped) {
#pragma unroll
              for (int i = 0; i < 16; ++i) glu_grad<true>(g.act, gv[i], uv[i], v[i], v[i], du[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) glu_grad<false>(g.act, gv[i], uv[i], v[i], v[i], du[i]);
            }
            store_bf16x16(orow + c0, v, left, wide);
            store_bf16x16(g.out2 + (size_t)m * p.N + n0 + c0, du, left, wide);
          }
        }
        sl += n_chunks;
      } else if (EPI == kEpiStore && !SPLIT && p.parts > 1) {
        // This warp's share of the part's sums, [part][CTA][columns / 4][row], goes to
        // memory.  The warp that does so last of all parts' adds the shares up in order, so
        // that the result does not depend on who that is, and finishes the tile.
        const size_t each = (size_t)kBM * kMaxN / 4;
        float4* all = g.partial + ((size_t)(p.base + tl.idx) * p.parts * CG + rank) * each + row;
        float4* mine = all + (size_t)tl.part * CG * each;
        for (int c0 = 32 * par; c0 < cols; c0 += 64) {
          float v[16], w[16];
          tmem_ld_2x16(taddr + (uint32_t)c0, taddr + (uint32_t)(c0 + 16), v, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mine[(c0 / 4 + i) * kBM] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            mine[(c0 / 4 + 4 + i) * kBM] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
        __threadfence();
        __syncwarp();
        int before = 0;
        if (lane == 0) before = (int)atomicAdd(g.arrived + ((p.base + tl.idx) * CG + rank) * kEpiWarps + warp - 2, 1u);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before == p.parts - 1) {
          __threadfence();
          for (int c0 = 32 * par; c0 < cols; c0 += 64) {
            float v[32] = {};
            for (int r = 0; r < p.parts; r += 2) {   // two parts in flight
              const float4* from = all + (size_t)r * CG * each + (c0 / 4) * kBM;
              const bool two = r + 1 < p.parts;
              float4 x[16];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                x[i] = __ldcg(from + i * kBM);
                x[8 + i] = two ? __ldcg(from + CG * each + i * kBM) : make_float4(0.f, 0.f, 0.f, 0.f);
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int j = 4 * (i & 7);
                v[j] += x[i].x;
                v[j + 1] += x[i].y;
                v[j + 2] += x[i].z;
                v[j + 3] += x[i].w;
              }
            }
            uint32_t z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            store_32x32(orow + c0 - (size_t)lane * p.N, p.N, z, p.M - (m - lane), cols - c0, lane);
          }
        }
      } else {
        for (int c0 = 32 * par; c0 < cols; c0 += 64) {
          float v[16], w[16];
          tmem_ld_2x16(taddr + (uint32_t)c0, taddr + (uint32_t)(c0 + 16), v, w);
          uint32_t z[16];
          pack16(v, z);
          pack16(w, z + 8);
          store_32x32(orow + c0 - (size_t)lane * p.N, p.N, z, p.M - (m - lane), cols - c0, lane);
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader<CG>(tc::smem_u32(&tempty_bar[b]));
      if (++b == 2) {
        b = 0;
        aph ^= 1;
      }
    }
  }

  if (SPLIT) {
    if (!all_run) cluster_wait();
    cluster_sync();   // every part has arrived
    if (warp >= 2 && warp < 2 + kEpiWarps) {
      const int q = warp & 3, par = (warp - 2) >> 2, row = 32 * q + lane;
      const Tile tl = tile_at<false>(g, unit);
      const Problem& p = g.p[tl.pi];
      const int tn = p.pair ? p.tn >> 1 : p.tn, n0 = tl.n * tn, shares = tn / 8;
      const bool pairs = EPI == kEpiGlu || (is_linear(EPI) && p.pair);
      const int each = pairs ? 16 : 8;
      const float* ex = reinterpret_cast<const float*>(smem + kStages * kStageBytes) + row;
      const int u0 = shares * part / parts, u1 = shares * (part + 1) / parts;
      for (int u = u0 + par; u < u1; u += 2) {
        if (n0 + 8 * u >= p.N || tl.m * kBM + 32 * q >= p.M) break;
        float v[8] = {}, w[8] = {};
        for (int r = 0; r < parts; ++r) {
          const float* x = ex + ((u - u0) * parts + r) * each * kBM;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[i] += x[i * kBM];
            if (pairs) w[i] += x[(8 + i) * kBM];
          }
        }
        finish8<EPI>(g, p, tl.m, row, n0 + 8 * u, v, w);
      }
    }
  }
  pdl_trigger();
  tc::tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();   // neither CTA leaves while the other's MMAs or arrivals may reach it
  tc::tc_fence_after();
  if (warp == 1) tmem_dealloc<CG>(tmem);
}

// ---------------------------------------------------------------- norms
// out[r] = |row r| of x (rows of x first), wg and wu: a warp per row, bound by the reads.  A
// sum of squares that leaves fp32's range, or comes near its smallest numbers, is formed again
// from the row times 2^-80 or 2^80.  At 1001 x 2880 x 2880 it takes 10 us of a training step's
// 138 (39 MB).  As four more warps of the gate/up kernel it cost nothing, but came too late
// for that kernel's epilogue, and settled in the backward pass, whose ring of g and u then
// stalls, the step took 161 us.
constexpr int kNormWarps = 8, kNormLoads = 6;
__global__ void __launch_bounds__(kNormWarps * 32, 6) glu_norm_kernel(const uint16_t* x, const uint16_t* wg, const uint16_t* wu,
                                                                      int T, int ff, int d, float* out) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long rows = T + 2LL * ff;
  for (long long r = (long long)blockIdx.x * kNormWarps + (threadIdx.x >> 5); r < rows; r += (long long)gridDim.x * kNormWarps) {
    const uint16_t* row = r < T ? x + r * d : r < T + (long long)ff ? wg + (r - T) * d : wu + (r - T - ff) * d;
    float by = 1.f, sum = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
      float s = 0.f;
      for (int i = 8 * lane; i < d; i += 256 * kNormLoads) {
        uint4 q[kNormLoads];
#pragma unroll
        for (int j = 0; j < kNormLoads; ++j)
          q[j] = i + 256 * j < d ? *reinterpret_cast<const uint4*>(row + i + 256 * j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < kNormLoads; ++j) {
          const uint32_t u[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = bf16_lo(u[e]) * by, hi = bf16_hi(u[e]) * by;
            s = fmaf(lo, lo, s);
            s = fmaf(hi, hi, s);
          }
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      sum = s;
      if (pass || (s > 1e-30f && s < 1e30f)) break;
      by = s < 1.f ? 0x1p80f : 0x1p-80f;
    }
    if (lane == 0) out[r] = sqrtf(sum) / by;
  }
}

// ---------------------------------------------------------------- host
bool map_bf16(CUtensorMap* m, const uint16_t* base, int rows, int cols, int box_rows) {
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, (uint64_t)rows, (uint64_t)cols, (uint64_t)cols * 2,
                  (uint32_t)box_rows, kBK, CU_TENSOR_MAP_SWIZZLE_128B);
}

int cdiv(int a, int b) { return (a + b - 1) / b; }

// A matrix [k, cols], cols a multiple of 64, seen as [cols / 64][k][64]: an MN-major tile of
// `blocks` x 64 columns and 64 k is one box.  (With a ragged last block its rows would run
// into the next row of the matrix, and past its end: those go by boxes of the plain map.)
bool map_blocks(CUtensorMap* m, const uint16_t* base, int k, int cols, int blocks) {
  const EncodeTiled fn = encode_tiled();
  if (!fn || !base) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)k, (cuuint64_t)(cols / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, 128};
  const cuuint32_t box[3] = {64, kBK, (cuuint32_t)blocks}, step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <int CG, int EPI, bool SPLIT>
cudaError_t prepare_kernel() {
  return allow_smem<glu_gemm_kernel<CG, EPI, SPLIT>>(Lay<EPI>::kSmemBytes);
}

// How many clusters of n = 1, 2, 4, 8 CTAs (one CTA per SM) the GPU holds at one time: [n].
struct ClusterCounts {
  int of[9];
  int operator[](int n) const { return of[n]; }
};

// Asked of the runtime once per device.
ClusterCounts cluster_counts() {
  static PerDevice<9> counts;
  int dev = 0;
  cudaGetDevice(&dev);
  ClusterCounts found;
  counts.get(dev, found.of, [](int (&of)[9]) {
    const int sms = sm_count();
    for (int n = 0; n < 9; ++n) of[n] = n ? std::max(1, sms / n) : 0;
    const bool ready = prepare_kernel<2, kEpiStore, false>() == cudaSuccess;
    for (int n = 2; n <= 8; n <<= 1) {
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)n;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(sms / n * n);
      cfg.blockDim = dim3(Lay<kEpiStore>::kThreads);
      cfg.dynamicSmemBytes = Lay<kEpiStore>::kSmemBytes;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int c = 0;
      if (ready && cudaOccupancyMaxActiveClusters(&c, glu_gemm_kernel<2, kEpiStore, false>, &cfg) == cudaSuccess && c > 0)
        of[n] = c;
    }
    return true;
  });
  return found;
}

// How a launch runs: single CTAs or pairs (cg), or clusters of `parts` CTAs that split k.
struct Way {
  int cg, parts, tn;
};

template <int CG, int EPI, bool SPLIT>
cudaError_t launch_as(const GemmParams& g, const Way& w, cudaStream_t s) {
  const cudaError_t e = prepare_kernel<CG, EPI, SPLIT>();
  if (e != cudaSuccess) return e;
  const int size = CG * w.parts;   // CTAs of a unit
  const int units = SPLIT ? g.tiles : cluster_counts()[size];
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)size;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size * (g.tiles < units ? g.tiles : units));
  cfg.blockDim = dim3(Lay<EPI>::kThreads);
  cfg.dynamicSmemBytes = Lay<EPI>::kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = size > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, glu_gemm_kernel<CG, EPI, SPLIT>, g);
}

int stage_bytes(int cg, int tn, bool b_mn) {
  return kTileA + (b_mn ? cdiv(tn / cg, 64) * 8192 : tn / cg * 128);
}

int stages_for(int bytes, int space, int most = 10) { return std::min(most, space / bytes); }

// Clocks of one chunk of 64 k with tn columns of B: the MMAs (2 per column for the 128
// rows of an SM, and 1 in 22 more), its operands' way into shared memory (86 bytes a clock),
// or the MMA issuer's own 330.  Fitted to launches of one wave of tiles at k 512 to 4096, as
// are the clocks below (one CTA at 256 columns: 307 ns a chunk, 128: 196, 32: 168; pairs:
// 278, 183, 176).  space: shared memory for the stages, given for MN-major operands, whose
// loads take up to 2600 clocks (one CTA at 256 columns, 4 stages: 657 a chunk).
int chunk_clocks(int cg, int tn, int space) {
  const int mma = 2 * tn * 23 / 22, feed = (kTileA + tn * 128 / cg) / 86;
  const int wait = space ? 2600 / stages_for(stage_bytes(cg, tn, true), space) : 0;
  return std::max(std::max(mma, wait), std::max(feed, 330));
}

// What a tile of tn columns adds to its chunks (its epilogue, as far as nothing hides it),
// and what a launch of pairs costs more than one of single CTAs (1.4 us).
int tile_fixed(int tn) { return 1000 + 8 * tn; }
constexpr int kPairClocks = 2100, kLaunchClocks = 2500;

// Split tiles of the weight gradients: at most 8 parts, and so many parts in all (two per
// pair of SMs; the sums of all are 40 MB, which L2 holds).
constexpr int kMaxParts = 8, kMaxSplit = 152;

// The way to run one product [M, N] (per = 2: gate/up, N columns of each) alone on the GPU
// for which
//   waves of tiles x (chunks of a unit x clocks per chunk + a tile's fixed cost)
// is least.  A long launch (kLongClocks: 100 us) runs against the power limit, where what
// the last wave leaves idle speeds the others up: there only the tiles count (8192 x
// 2048 x 8192 forward with y in pairs' tiles of 256 columns, 3.4 waves: 485 us, of 192, 4.6
// waves: 493 us; no more apart than two boxes are, so the rule is a weak one).  A part of a split tile pays for the exchange (two parts of 128 columns 2.7 us,
// of 32 columns 1.3 us).
constexpr long long kLongClocks = 200000;
// finer: widths between 128 and 256 columns in steps of 16 (the linear layer's; 4096 x 2048 x
// 2048 takes 144 tiles of 240 columns instead of 128 of 256 on 76 pairs, 25.0 us instead of 27.4).
Way pick_way(int M, int N, int chunks, int per, int space, long long* clocks = nullptr, bool finer = false) {
  Way best{1, 1, kMaxN};
  long long least = -1;
  const ClusterCounts counts = cluster_counts();
  auto consider = [&](int cg, int parts, int tn) {
    const int units = counts[cg * parts];
    const long long tiles = (long long)cdiv(M, kBM * cg) * cdiv(N, tn / per);
    const int exchange = parts > 1 ? 1500 + 29 * tn + 500 * (parts - 2) : 0;
    const long long each = (long long)cdiv(chunks, parts) * chunk_clocks(cg, tn, space) + tile_fixed(tn) + exchange;
    long long cost = (tiles + units - 1) / units * each;
    if (cost > kLongClocks) cost = tiles * each / units;
    cost += cg == 2 ? kPairClocks : 0;
    if (least < 0 || cost < least) {
      least = cost;
      best = Way{cg, parts, tn};
    }
  };
  for (int cg = 1; cg <= 2; ++cg)
    // boxes of 16 rows of gate and of up are too small for few tokens (16 x 1080 x 1520:
    // 18.6 us, of 32 rows 15.6; 126 x 376 x 1216: 9.9, 10.4)
    for (int tn = 256; tn >= 32 * per; tn -= finer && tn > 128 ? 16 : 32) consider(cg, 1, tn);
  for (int parts = 2; parts <= 8 && parts <= chunks; parts <<= 1)
    // up to 128 columns: the exchange's space leaves the ring three stages at least
    for (int tn = 128; tn >= 8 * per * parts && tn >= 32; tn >>= 1) consider(1, parts, tn);
  if (clocks) *clocks = least;
  return best;
}

// Clocks of a unit's work on a tile: its chunks, and what its epilogue adds to the next
// tile's start.  A part of a split tile writes its sums (128 KiB a CTA) and the last one reads
// all parts' at about 60 bytes a clock: 2500 clocks a part, and as long as four of these go
// by in memory fences and in what is late for the last (measured: a weak rule at the border,
// 1500 x 1024 x 512 backward is 23.3 us whole and 26.2 in two parts; 16384 x 512 x 512 is
// 161 us whole, 73 in two parts, 61 in four and 68 in six).
constexpr int kPartClocks = 2500;
long long tile_clocks(int chunks, int parts, int cg, int tn, int space) {
  return (long long)cdiv(chunks, parts) * chunk_clocks(cg, tn, space) + tile_fixed(tn) + (parts > 1 ? (parts + 4LL) * kPartClocks : 0);
}
long long tile_clocks(const Problem& p, int cg) { return tile_clocks(p.nkc * p.segs, p.parts, cg, p.tn, Lay<kEpiStore>::kStageSpace); }

// Gives the tiles of several products, the longest first, each to the unit that is done
// first.  With more tiles than the list holds (then there are many per unit) they go round
// in turn.
void list_tiles(GemmParams& g, int cg) {
  const int units = cluster_counts()[cg];
  g.tiles = 0;
  for (int i = 0; i < g.n_problems; ++i) g.tiles += g.p[i].mt * g.p[i].nt * g.p[i].parts;
  g.listed = g.n_problems > 1 && g.tiles <= kMaxListed && units <= kMaxUnits;
  if (!g.listed) return;
  int order[kMaxProblems], start[kMaxProblems], n = 0;
  for (int i = 0; i < g.n_problems; ++i) {
    order[i] = i;
    start[i] = n;
    n += g.p[i].mt * g.p[i].nt * g.p[i].parts;
  }
  std::sort(order, order + g.n_problems, [&](int a, int b) { return tile_clocks(g.p[a], cg) > tile_clocks(g.p[b], cg); });
  // a heap of (clocks so far, unit); who took which tile
  std::pair<long long, int> heap[kMaxUnits];
  for (int u = 0; u < units; ++u) heap[u] = {0, -u};   // equal loads: the lowest unit first
  auto later = [](const std::pair<long long, int>& a, const std::pair<long long, int>& b) {
    return a.first != b.first ? a.first > b.first : a.second < b.second;
  };
  std::make_heap(heap, heap + units, later);
  uint16_t taken_by[kMaxListed], count[kMaxUnits] = {};
  for (int i = 0; i < g.n_problems; ++i) {
    const Problem& p = g.p[order[i]];
    const long long c = tile_clocks(p, cg);
    for (int t = 0; t < p.mt * p.nt * p.parts; ++t) {
      std::pop_heap(heap, heap + units, later);
      auto& least = heap[units - 1];
      least.first += c;
      taken_by[start[order[i]] + t] = (uint16_t)(-least.second);
      ++count[-least.second];
      std::push_heap(heap, heap + units, later);
    }
  }
  g.first[0] = 0;
  for (int u = 0; u < units; ++u) g.first[u + 1] = (uint16_t)(g.first[u] + count[u]);
  uint16_t at[kMaxUnits];
  std::copy(g.first, g.first + units, at);
  for (int i = 0; i < g.n_problems; ++i)   // a unit's tiles in the order it took them
    for (int t = start[order[i]], e = t + g.p[order[i]].mt * g.p[order[i]].nt * g.p[order[i]].parts; t < e; ++t) g.list[at[taken_by[t]]++] = (uint16_t)t;
}

template <int EPI>
cudaError_t launch(GemmParams& g, const Way& w, cudaStream_t s) {
  g.stage_bytes = 0;
  for (int i = 0; i < g.n_problems; ++i) g.stage_bytes = std::max(g.stage_bytes, stage_bytes(w.cg, g.p[i].tn, g.p[i].b_mn));
  g.stage_bytes = (g.stage_bytes + 1023) / 1024 * 1024;
  // a split tile's exchange takes the partial sums of 128 rows x its columns
  int space = Lay<EPI>::kStageSpace - (w.parts > 1 ? kBM * w.tn * 4 : 0), most = 10;
  if (is_linear(EPI) && g.tile_a < kTileA) {
    // the MMAs read 128 rows all the same: what comes behind the last stage's has to be there
    g.stage_bytes -= kTileA - g.tile_a;
    space -= std::max(0, kTileA - g.stage_bytes);
    most = kMaxStages;
  }
  g.stages = stages_for(g.stage_bytes, space, most);
  list_tiles(g, w.cg);
  if (w.parts > 1) return launch_as<1, EPI, true>(g, w, s);
  return w.cg == 2 ? launch_as<2, EPI, false>(g, w, s) : launch_as<1, EPI, false>(g, w, s);
}

// D [M, N] = sum over segments of A_s B_s^T, k of length K in each.  a_mn / b_mn: the
// operand is stored [K, M] / [K, N].
bool set_problem(Problem& p, int cg, int tn, int M, int N, int K, const uint16_t* a0, const uint16_t* a1, bool a_mn,
                 const uint16_t* b0, const uint16_t* b1, bool b_mn, uint16_t* out) {
  p.M = M;
  p.N = N;
  p.nkc = cdiv(K, kBK);
  p.segs = a1 ? 2 : 1;
  p.pair = 0;
  p.parts = 1;
  p.a_mn = a_mn;
  p.b_mn = b_mn;
  p.mt = cdiv(M, kBM * cg);
  p.tn = tn;
  p.nt = cdiv(N, tn);
  p.wide = N % 16 == 0 && aligned32(out);
  p.out = out;
  const uint16_t* a[2] = {a0, a1};
  const uint16_t* b[2] = {b0, b1};
  const int brows = tn / cg;
  p.a_blocks = a_mn && M % 64 == 0;
  p.b_blocks = b_mn && N % 64 == 0 && brows % 64 == 0;
  for (int i = 0; i < p.segs; ++i) {
    if (!(p.a_blocks ? map_blocks(&p.a[i], a[i], K, M, 2)
          : a_mn     ? map_bf16(&p.a[i], a[i], K, M, 64)
                     : map_bf16(&p.a[i], a[i], M, K, kBM)))
      return false;
    if (!(p.b_blocks ? map_blocks(&p.b[i], b[i], K, N, brows / 64)
          : b_mn     ? map_bf16(&p.b[i], b[i], K, N, 64)
                     : map_bf16(&p.b[i], b[i], N, K, brows)))
      return false;
  }
  return true;
}

}  // namespace

cudaError_t launch_glu_gate_up(const GluParams& w, const uint16_t* x, int T, uint16_t* h, float* sg, float* su,
                               float* norms, uint32_t* status, cudaStream_t s) {
  // Only what the backward pass will need to know: without it h is continuous at the border.
  const bool settled = sg && w.act == MOE_ACT_CLAMPED_GLU;
  if (settled) {
    const long long blocks = (T + 2LL * w.ff + kNormWarps - 1) / kNormWarps, most = 6LL * sm_count();
    const cudaError_t e = launch_pdl(glu_norm_kernel, dim3((unsigned)std::min(blocks, most)), dim3(kNormWarps * 32), 0, s, x,
                                     w.gate, w.up, T, w.ff, w.d, norms);
    if (e != cudaSuccess) return e;
  }
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  g.n_problems = 1;
  Problem& p = g.p[0];
  p.M = T;
  p.N = w.ff;
  p.nkc = cdiv(w.d, kBK);
  p.segs = 1;
  p.pair = 1;
  p.parts = 1;
  const Way way = pick_way(T, w.ff, p.nkc, 2, 0);
  p.tn = way.tn;
  p.mt = cdiv(T, kBM * way.cg);
  p.nt = cdiv(w.ff, p.tn / 2);
  p.wide = w.ff % 16 == 0 && aligned32(h);
  p.out = h;
  if (!map_bf16(&p.a[0], x, T, w.d, kBM) || !map_bf16(&p.b[0], w.gate, w.ff, w.d, p.tn / 2) ||
      !map_bf16(&p.b[1], w.up, w.ff, w.d, p.tn / 2))
    return cudaErrorInvalidValue;
  g.act = GluAct{w.act, w.limit, w.alpha};
  g.g = sg;
  g.u = su;
  g.x = x;
  g.wg = w.gate;
  g.wu = w.up;
  g.d = w.d;
  g.norm = settled ? norms : nullptr;
  g.gap = (float)(w.d / 16 + 9) * 0x1p-24f;
  g.status = status;
  g.clear_status = 1;
  return launch<kEpiGlu>(g, way, s);
}

cudaError_t launch_glu_down(const GluParams& w, const uint16_t* h, int T, uint16_t* y, uint32_t* status,
                            cudaStream_t s) {
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  g.n_problems = 1;
  const Way way = pick_way(T, w.d, cdiv(w.ff, kBK), 1, 0);
  if (!set_problem(g.p[0], way.cg, way.tn, T, w.d, w.ff, h, nullptr, false, w.down, nullptr, false, y)) return cudaErrorInvalidValue;
  g.status = status;
  return launch<kEpiStore>(g, way, s);
}

namespace {

// The tiles of a launch that are alike: how many, and the clocks of each.
struct Alike {
  int tiles;
  long long clocks;
};

// When the last of `units` is done if the longest tiles go out first, each to the unit that
// is free first.
long long span(int units, Alike* a, int n) {
  std::sort(a, a + n, [](const Alike& x, const Alike& y) { return x.clocks > y.clocks; });
  std::pair<long long, int> level[64];   // busy until, units: in order
  int levels = 1;
  level[0] = {0, units};
  for (int i = 0; i < n; ++i) {
    int left = a[i].tiles;
    while (left > 0) {
      const int k = std::min(level[0].second, left);
      const long long until = level[0].first + a[i].clocks;
      left -= k;
      if ((level[0].second -= k) == 0) std::copy(level + 1, level + levels--, level);
      int at = 0;
      while (at < levels && level[at].first < until) ++at;
      if (at < levels && level[at].first == until) {
        level[at].second += k;
      } else if (levels < 64) {
        std::copy_backward(level + at, level + levels, level + levels + 1);
        level[at] = {until, k};
        ++levels;
      } else {
        return until;   // more levels than any few kinds of tiles give
      }
    }
  }
  return level[levels - 1].first;
}

// How a backward pass is laid out: whether dWd = dy^T h, which waits for nothing that the
// pass computes, fills up the SMs beside dg and du; dx in a launch of its own, its long sum
// over few tiles split; and over how many units the k (tokens) of a weight gradient's tile.
struct Backward {
  Way dact, dx;
  int cg, parts, tn;   // of the launch of dx and the weight gradients
  bool down_first, dx_alone;
};

Backward plan_backward(const GluParams& w, int T, bool dx, bool dwg, bool dwu, bool dwd) {
  constexpr int kDactSpace = Lay<kEpiDact>::kStageSpace, kSpace = Lay<kEpiStore>::kStageSpace;
  const ClusterCounts counts = cluster_counts();
  const int k = cdiv(T, kBK), kd = cdiv(w.d, kBK), kff = cdiv(w.ff, kBK);
  auto tiles = [&](int M, int N, int cg, int tn) { return (int)std::min<long long>((long long)cdiv(M, kBM * cg) * cdiv(N, tn), 1 << 28); };
  auto pairs = [](int cg) { return cg == 2 ? kPairClocks : 0; };
  Alike a[2];
  // dg and du alone, or with dWd beside them (a launch that splits k has no other tiles)
  long long dact[2], alone_dx = 0, least = -1;
  Way way[2];
  way[0] = pick_way(T, w.ff, kd, 1, kDactSpace, &dact[0]);
  dact[1] = -1;
  for (int cg = 1; dwd && cg <= 2; ++cg)
    for (int tn = kMaxN; tn >= 64; tn -= 32) {
      a[0] = Alike{tiles(T, w.ff, cg, tn), tile_clocks(kd, 1, cg, tn, kDactSpace)};
      a[1] = Alike{tiles(w.d, w.ff, cg, kMaxN), tile_clocks(k, 1, cg, kMaxN, kDactSpace)};
      const long long clocks = span(counts[cg], a, 2) + pairs(cg);
      if (dact[1] < 0 || clocks < dact[1]) {
        dact[1] = clocks;
        way[1] = Way{cg, 1, tn};
      }
    }
  Backward b{};
  if (dx) b.dx = pick_way(T, w.d, 2 * kff, 1, kSpace, &alone_dx);
  const int most = glu_split_tiles(w.d, w.ff, T);   // no split over more tiles: there are many per unit
  auto consider = [&](int cg, int tn, int parts) {
    for (int first = dwd ? 1 : 0; first >= 0; --first)
      for (int alone = 0; alone <= (dx && b.dx.parts > 1 ? 1 : 0); ++alone) {
        const int products = dwg + dwu + (dwd && !first), each = tiles(w.d, w.ff, cg, tn);
        if (parts > 1 && (long long)products * each * parts > most) continue;
        int n = 0;
        if (dx && !alone) a[n++] = Alike{tiles(T, w.d, cg, tn), tile_clocks(2 * kff, 1, cg, tn, kSpace)};
        if (products) a[n++] = Alike{products * each * parts, tile_clocks(k, parts, cg, tn, kSpace)};
        long long clocks = dact[first] + (alone ? alone_dx + kLaunchClocks : 0);
        if (n) clocks += span(counts[cg], a, n) + kLaunchClocks + pairs(cg);
        if (least < 0 || clocks < least) {
          least = clocks;
          b = Backward{way[first], b.dx, cg, parts, tn, first == 1, alone == 1};
        }
      }
  };
  for (int cg = 1; cg <= 2; ++cg)
    for (int tn = kMaxN; tn >= 128; tn >>= 1) consider(cg, tn, 1);
  for (int parts = 2; parts <= kMaxParts && k >= 4 * parts; ++parts) consider(2, kMaxN, parts);
  return b;
}

}  // namespace

// A pair's tile of a split product is 256 x 256 fp32 sums.
int glu_split_tiles(int d, int ff, int T) {
  const long long tiles = 3LL * cdiv(d, 2 * kBM) * cdiv(ff, kMaxN);
  if (T < 8 * kBK || 2 * tiles > kMaxSplit) return 0;
  return (int)std::min<long long>(kMaxParts * tiles, kMaxSplit);
}

cudaError_t launch_glu_backward(const GluParams& w, const uint16_t* x, const uint16_t* dy, int T, const GluSaved& sv,
                                uint16_t* dg, uint16_t* du, uint16_t* dx, uint16_t* dwg, uint16_t* dwu, uint16_t* dwd,
                                const GluSplit& split, uint32_t* status, cudaStream_t s) {
  const Backward b = plan_backward(w, T, dx, dwg, dwu, dwd);
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  if (!set_problem(g.p[g.n_problems++], b.dact.cg, b.dact.tn, T, w.ff, w.d, dy, nullptr, false, w.down, nullptr, true, dg))
    return cudaErrorInvalidValue;
  g.p[0].wide = g.p[0].wide && aligned32(du);
  g.act = GluAct{w.act, w.limit, w.alpha};
  g.g = sv.g;
  g.u = sv.u;
  g.out2 = du;
  g.status = status;
  g.clear_status = 1;
  g.arrived = split.arrived;
  g.zeros = b.parts > 1 ? kMaxSplit * 2 * kEpiWarps : 0;
  if (b.down_first &&
      !set_problem(g.p[g.n_problems++], b.dact.cg, kMaxN, w.d, w.ff, T, dy, nullptr, true, sv.h, nullptr, true, dwd))
    return cudaErrorInvalidValue;
  cudaError_t e = launch<kEpiDact>(g, b.dact, s);
  if (e != cudaSuccess) return e;

  std::memset(&g, 0, sizeof(g));
  g.status = status;
  if (b.dx_alone) {
    if (!set_problem(g.p[g.n_problems++], b.dx.cg, b.dx.tn, T, w.d, w.ff, dg, du, false, w.gate, w.up, true, dx))
      return cudaErrorInvalidValue;
    e = launch<kEpiStore>(g, b.dx, s);
    if (e != cudaSuccess) return e;
    g.n_problems = 0;
    dx = nullptr;
  }
  bool ok = true;
  int base = 0;
  auto product = [&](int M, int N, int K, const uint16_t* a0, const uint16_t* a1, bool a_mn, const uint16_t* b0,
                     const uint16_t* b1, int parts, uint16_t* out) {
    Problem& p = g.p[g.n_problems++];
    ok = ok && set_problem(p, b.cg, b.tn, M, N, K, a0, a1, a_mn, b0, b1, true, out);
    p.parts = parts;
    p.base = base;
    if (parts > 1) base += p.mt * p.nt;
  };
  if (dx) product(T, w.d, w.ff, dg, du, false, w.gate, w.up, 1, dx);
  if (dwg) product(w.ff, w.d, T, dg, nullptr, true, x, nullptr, b.parts, dwg);
  if (dwu) product(w.ff, w.d, T, du, nullptr, true, x, nullptr, b.parts, dwu);
  if (dwd && !b.down_first) product(w.d, w.ff, T, dy, nullptr, true, sv.h, nullptr, b.parts, dwd);
  if (!ok) return cudaErrorInvalidValue;
  if (!g.n_problems) return cudaSuccess;
  g.partial = reinterpret_cast<float4*>(split.partial);
  g.arrived = split.arrived;
  return launch<kEpiStore>(g, Way{b.cg, 1, b.tn}, s);
}

// ---------------------------------------------------------------- the linear layer
namespace {

// The way for T <= 128 tokens, one row of tiles: the weights' stream bounds what pick_way's
// clocks do not, epilogues and exchanges take the rows that there are, 32 to a warp, and x no
// more of a stage than its rows (a_bytes), so that more weights are under way: 32 tokens, 8192 x
// 8192, bf16 33.0 us with stages of 128 rows of x, 28.6 with 32, 27.4 in the way that this picks;
// e4m3 21.1, 18.8 and 16.0; 8192 x 1024 10.7 and 8.6.
Way pick_few(int T, int N, int chunks, int per, int a_bytes) {
  constexpr long long kStream = 3370;   // bytes a clock from memory: 6.4 TB/s
  Way best{1, 1, kMaxN};
  long long least = -1;
  const ClusterCounts counts = cluster_counts();
  const int warps = cdiv(T, 32);
  auto consider = [&](int parts, int tn) {
    const int units = counts[parts], feed = (a_bytes + tn * 128) / 86;
    const long long waves = (cdiv(N, tn / per) + units - 1) / units;
    const int chunk = std::max(std::max(2 * tn * 23 / 22, feed), 330);
    const int exchange = parts > 1 ? 1500 + 29 * tn * warps / 4 + 500 * (parts - 2) : 0;
    const long long work = waves * cdiv(chunks, parts) * chunk, stream = (long long)N * per * chunks * 128 / kStream;
    const long long cost = std::max(work, stream) + waves * (1000 + 2 * tn * warps + exchange);
    if (least < 0 || cost < least) {
      least = cost;
      best = Way{1, parts, tn};
    }
  };
  for (int tn = 256; tn >= 32 * per; tn -= 32) consider(1, tn);
  for (int parts = 2; parts <= 8 && parts <= chunks; parts <<= 1)
    for (int tn = 128; tn >= 8 * per * parts && tn >= 32; tn >>= 1) consider(parts, tn);
  return best;
}

}  // namespace

cudaError_t launch_linear_gemm(const LinearShape& l, const void* x, int T, const void* weights, uint16_t* y,
                               const LinearEpi& epi, uint32_t* status, cudaStream_t s) {
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  g.n_problems = 1;
  // e4m3 values are moved two at a time: to TMA both formats are rows of n_in bytes or 2 n_in
  const int k = l.eight ? l.n_in / 2 : l.n_in, per = epi.glu ? 2 : 1;
  const uint16_t *a = static_cast<const uint16_t*>(x), *b = static_cast<const uint16_t*>(weights);
  Problem& p = g.p[0];
  p.M = T;
  p.N = l.n_out;
  p.nkc = cdiv(k, kBK);
  p.segs = 1;
  p.pair = epi.glu;
  p.parts = 1;
  const int arows = std::min(kBM, (T + 7) / 8 * 8);
  g.tile_a = arows * kBK * 2;
  const Way way = T <= kBM ? pick_few(T, l.n_out, p.nkc, per, g.tile_a) : pick_way(T, l.n_out, p.nkc, per, 0, nullptr, per == 1);
  p.tn = way.tn;
  p.mt = cdiv(T, kBM * way.cg);
  p.nt = cdiv(l.n_out, p.tn / per);
  p.wide = l.n_out % 16 == 0 && aligned32(y);
  p.out = y;
  const int brows = epi.glu ? p.tn / 2 : p.tn / way.cg;
  if (!map_bf16(&p.a[0], a, T, k, arows) || !map_bf16(&p.b[0], b, l.n_out, k, brows) ||
      (epi.glu && !map_bf16(&p.b[1], b + (size_t)l.n_out * k, l.n_out, k, brows)))
    return cudaErrorInvalidValue;
  g.lin = epi;
  g.status = status;
  g.clear_status = 1;
  return l.eight ? launch<kEpiLinear8>(g, way, s) : launch<kEpiLinear>(g, way, s);
}

LinearPlan plan_linear_backward(const LinearShape& l, int T, bool dx, bool dw) {
  const int n_in = l.n_in, n_out = l.n_out;
  constexpr int kSpace = Lay<kEpiStore>::kStageSpace;
  const ClusterCounts counts = cluster_counts();
  const int k = cdiv(T, kBK), ko = cdiv(n_out, kBK);
  auto tiles = [&](int M, int N, int cg, int tn) { return (int)std::min<long long>((long long)cdiv(M, kBM * cg) * cdiv(N, tn), 1 << 28); };
  LinearPlan b{};
  long long least = -1, alone_dx = 0;
  Way own{1, 1, kMaxN};
  if (dx) own = pick_way(T, n_in, ko, 1, kSpace, &alone_dx);
  b.dx_cg = own.cg;
  b.dx_parts = own.parts;
  b.dx_tn = own.tn;
  const int most = linear_split_tiles(n_in, n_out, T);
  Alike a[2];
  auto consider = [&](int cg, int tn, int parts) {
    for (int alone = 0; alone <= (dx && (!dw || own.parts > 1) ? 1 : 0); ++alone) {
      const int each = tiles(n_out, n_in, cg, tn);
      if (parts > 1 && (!dw || (long long)each * parts > most)) continue;
      int n = 0;
      if (dx && !alone) a[n++] = Alike{tiles(T, n_in, cg, tn), tile_clocks(ko, 1, cg, tn, kSpace)};
      if (dw) a[n++] = Alike{each * parts, tile_clocks(k, parts, cg, tn, kSpace)};
      long long clocks = alone ? alone_dx + kLaunchClocks : 0;
      if (n) clocks += span(counts[cg], a, n) + kLaunchClocks + (cg == 2 ? kPairClocks : 0);
      if (least < 0 || clocks < least) {
        least = clocks;
        b.cg = cg;
        b.parts = parts;
        b.tn = tn;
        b.dx_alone = alone == 1;
      }
    }
  };
  for (int cg = 1; cg <= 2; ++cg)
    for (int tn = kMaxN; tn >= 128; tn >>= 1) consider(cg, tn, 1);
  for (int parts = 2; parts <= kMaxParts && k >= 4 * parts; ++parts) consider(2, kMaxN, parts);
  return b;
}

int linear_split_tiles(int n_in, int n_out, int T) {
  const long long tiles = (long long)cdiv(n_out, 2 * kBM) * cdiv(n_in, kMaxN);
  if (T < 8 * kBK || 2 * tiles > kMaxSplit) return 0;
  return (int)std::min<long long>(kMaxParts * tiles, kMaxSplit);
}

cudaError_t launch_linear_backward(const LinearShape& l, const LinearPlan& b, const uint16_t* x, int T, const uint16_t* w, const uint16_t* dv,
                                   uint16_t* dx, uint16_t* dw, const GluSplit& split, const BiasParts& bias, uint32_t* status,
                                   cudaStream_t s) {
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  g.status = status;
  g.clear_status = 1;
  g.bias = bias;
  if (b.dx_alone) {
    if (!set_problem(g.p[g.n_problems++], b.dx_cg, b.dx_tn, T, l.n_in, l.n_out, dv, nullptr, false, w, nullptr, true, dx))
      return cudaErrorInvalidValue;
    const cudaError_t e = launch<kEpiStore>(g, Way{b.dx_cg, b.dx_parts, b.dx_tn}, s);
    if (e != cudaSuccess || !dw) return e;
    g.n_problems = g.clear_status = 0;
    g.bias.parts = nullptr;
    dx = nullptr;
  }
  if (dx && !set_problem(g.p[g.n_problems++], b.cg, b.tn, T, l.n_in, l.n_out, dv, nullptr, false, w, nullptr, true, dx))
    return cudaErrorInvalidValue;
  if (dw) {
    Problem& p = g.p[g.n_problems++];
    if (!set_problem(p, b.cg, b.tn, l.n_out, l.n_in, T, dv, nullptr, true, x, nullptr, true, dw)) return cudaErrorInvalidValue;
    p.parts = b.parts;
    p.base = 0;
  }
  g.partial = reinterpret_cast<float4*>(split.partial);
  g.arrived = split.arrived;
  return launch<kEpiStore>(g, Way{b.cg, 1, b.tn}, s);
}

cudaError_t glu_set_wait_test(uint32_t polls, int withhold) { return tc::set_wait_test(polls, withhold); }

}  // namespace moe
