// Internal contract between the dense block's C-ABI host code (block_abi.cu) and its
// kernel translation units.
#pragma once

#include "../../include/moe_linear.h"
#include "internal.h"
#include "per_device.h"

namespace moe {

// Lets KERNEL use up to `bytes` of dynamic shared memory; asked of the runtime once per
// device (`bytes` is the same at every call).
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
  static PerDevice<1> allowed;
  int dev = 0, got[1];
  cudaGetDevice(&dev);
  cudaError_t e = cudaSuccess;
  allowed.get(dev, got, [&](int (&out)[1]) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    out[0] = bytes;
    return e == cudaSuccess;
  });
  return e;
}

// The gated FFN's shapes and weights.
struct GluParams {
  const uint16_t *gate, *up, *down;   // bf16 [ff, d], [ff, d], [d, ff]
  int d, ff;
  int act;
  float limit, alpha;
};

// What a training forward pass keeps: h row-major; g and u in blocks of 128 tokens x 4
// columns, [block of tokens][ff / 4][128][4], so that the threads of a warp, which hold
// one token row each, store and load whole lines.
struct GluSaved {
  uint16_t* h;     // bf16 [T, ff]
  float* g;        // fp32, 128-token blocks
  float* u;
};

// tcgen05 kernels (glu_gemm.cu).  Each clears or may set bits of *status.
// h = act(x Wg^T, x Wu^T); g, u non-null: kept as GluSaved describes; norms: scratch for the
// norms of x's rows and of both weights' (T + 2 ff floats; clamped, with g and u).
cudaError_t launch_glu_gate_up(const GluParams& p, const uint16_t* x, int T, uint16_t* h, float* g, float* u,
                               float* norms, uint32_t* status, cudaStream_t s);
// y = h Wd^T
cudaError_t launch_glu_down(const GluParams& p, const uint16_t* h, int T, uint16_t* y, uint32_t* status,
                            cudaStream_t s);
// Room for the weight gradients' products whose k (the tokens) several units share:
// glu_split_tiles(d, ff, T) x 256 KiB of partial sums (none for long weights or few tokens),
// and the counts of the parts that are there.
int glu_split_tiles(int d, int ff, int T);
constexpr size_t kGluSplitBytes = 256 * 256 * 4, kGluArrivedBytes = 152 * 16 * 4;
struct GluSplit {
  float* partial;
  uint32_t* arrived;
};
// dg, du [T, ff] (scratch) from dy and the saved g and u; then dx, dWg, dWu, dWd, each where
// its pointer is non-null
cudaError_t launch_glu_backward(const GluParams& p, const uint16_t* x, const uint16_t* dy, int T, const GluSaved& sv,
                                uint16_t* dg, uint16_t* du, uint16_t* dx, uint16_t* dwg, uint16_t* dwu, uint16_t* dwd,
                                const GluSplit& split, uint32_t* status, cudaStream_t s);
cudaError_t glu_set_wait_test(uint32_t polls, int withhold);

// Few tokens (skinny.cu): the weights stream through warp MMAs, every 16 tokens.
// x_lo, y_lo: the low halves of a two-part x or h (at most 8 tokens); a two-part h carries
// what rounding h to bf16 would lose into the down product.  early: the launch before it on
// the stream was this function's (the weights may be read before its results are there).
cudaError_t launch_skinny_bf16(const uint16_t* w0, const uint16_t* w1, int n_out, int n_in, const uint16_t* x,
                               const uint16_t* x_lo, int T, const GluParams* act, uint16_t* y, uint16_t* y_lo,
                               uint32_t* clear_status, bool early, cudaStream_t s);
cudaError_t launch_skinny_w4(const moe_w4_cfg_t& c, const moe_w4_weights_t& w, const uint16_t* x, int T, uint16_t* y,
                             cudaStream_t s);

// The linear layer (moe_linear.h).
struct LinearEpi;   // linear_act.cuh
struct LinearShape {
  int n_in, n_out;
  bool eight;       // operands in e4m3
};
// Many tokens (glu_gemm.cu): y = act(x W^T ...) as epi says.
cudaError_t launch_linear_gemm(const LinearShape& l, const void* x, int T, const void* w, uint16_t* y, const LinearEpi& epi,
                               uint32_t* status, cudaStream_t s);
// The same for few tokens (linear_stream.cu), and whether that is the faster way.
bool linear_streams(const LinearShape& l, int T, bool glu);
cudaError_t launch_linear_stream(const LinearShape& l, const void* x, int T, const void* w, uint16_t* y, const LinearEpi& epi,
                                 uint32_t* clear_status, cudaStream_t s);
// Room for a weight gradient whose tokens several units share, as glu_split_tiles.
int linear_split_tiles(int n_in, int n_out, int T);
// How the two products of a backward pass are laid out: dx in a launch of its own (where it is the
// only product, or its long sum over few tiles is split) or beside dW, and over how many
// units the tokens of a tile of dW (parts > 1: split.arrived has to be zero before).
struct LinearPlan {
  int dx_cg, dx_parts, dx_tn;
  int cg, parts, tn;
  bool dx_alone;
};
LinearPlan plan_linear_backward(const LinearShape& l, int T, bool dx, bool dw);
// Partial sums of a bias's gradient, [rows][n] floats (parts null: none), and where it goes.
struct BiasParts {
  const float* parts;
  int rows, n;
  uint16_t* out;
};
// dx = dv W, dW = dv^T x, each where its pointer is non-null (one of them is); the bias's gradient
// on the way.
cudaError_t launch_linear_backward(const LinearShape& l, const LinearPlan& plan, const uint16_t* x, int T, const uint16_t* w, const uint16_t* dv,
                                   uint16_t* dx, uint16_t* dw, const GluSplit& split, const BiasParts& bias, uint32_t* status,
                                   cudaStream_t s);
// dv = dy act'(pre) (dv null: not written) and partial sums of its rows, linear_bias_parts(n, T)
// x n floats (parts null: none), which the products' launch or the function after adds up; clears
// *status and `zeros` words at `clear`.
int linear_bias_parts(int n, int T);
cudaError_t launch_linear_dbias(const BiasParts& bias, cudaStream_t s);
cudaError_t launch_linear_dv(int act, const uint16_t* dy, const uint16_t* pre, int T, int n, uint16_t* dv, float* parts,
                             uint32_t* status, uint32_t* clear, int zeros, cudaStream_t s);

// Norms (block_norm.cu).
cudaError_t launch_block_norm_fwd(const moe_norm_cfg_t& c, const moe_norm_inputs_t& in, int T, uint16_t* y,
                                  uint16_t* a, cudaStream_t s);
// The same with a in e4m3 and a scale per row; without pre_w a = y.
cudaError_t launch_block_norm_quant(const moe_norm_cfg_t& c, const moe_norm_inputs_t& in, int T, uint16_t* y, uint8_t* q,
                                    float* scale, cudaStream_t s);
int block_norm_parts(int T);   // rows of the weight gradients' partial sums
cudaError_t launch_block_norm_bwd(const moe_norm_cfg_t& c, const moe_norm_inputs_t& in, int T, const uint16_t* dy,
                                  const uint16_t* da, const moe_norm_grads_t& g, float* parts, cudaStream_t s);

}  // namespace moe
