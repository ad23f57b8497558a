/*
 * moe_block.h -- C ABI of the dense block around the sparse MoE layer of moe.h, for
 * GB300 (sm_103a): the gated feed-forward network with its backward pass, the norms
 * either side of a block with its gate and residual scale (forward and backward), and
 * the linear layer with 4-bit weights and group scales.  Same library (libmoe.so),
 * status codes and conventions as moe.h: the caller owns every buffer, nothing
 * synchronises, work is enqueued on `stream` in order, bf16 tensors are raw bit
 * patterns in row-major order, weight matrices are row = output, column = input.
 * Every tensor pointer must be 16-byte aligned (MOE_ERR_ALIGNMENT).  On error nothing
 * has been enqueued unless the code is MOE_ERR_CUDA.  Reserved members must be zero.
 * The gated FFN and the norms take up to 2^30 tokens (MOE_ERR_UNSUPPORTED past that).
 *
 * Sums, norm statistics and activations are computed in fp32; results are rounded once
 * to their type (round to nearest even).  All reductions run in a fixed order, so equal
 * inputs give bit-identical results from run to run.  Infinities and NaN in an input
 * pass through as the formulas say.
 */
#ifndef MOE_BLOCK_H_
#define MOE_BLOCK_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ gated FFN
 *   g = x Wg^T;  u = x Wu^T;  h = act(g, u);  y = h Wd^T
 *   MOE_ACT_SWIGLU:       h = g sigmoid(g) u
 *   MOE_ACT_CLAMPED_GLU:  h = (clamp(u, +-limit) + 1) g' sigmoid(alpha g'), g' = min(g, limit)
 * h is rounded to bf16 between the two products (the operand type of the tensor cores);
 * with saved NULL, at most 8 tokens and ff <= 4096, where that rounding would show beside
 * y's own, h keeps its low half as a second bf16. */
typedef struct {
  int32_t d_model;     /* d, a positive multiple of 8, at most 2^29 */
  int32_t ff;          /* hidden width, a positive multiple of 8, at most 2^29 */
  int32_t act;         /* MOE_ACT_* */
  float glu_limit;     /* clamped GLU limit, >= 0 */
  float glu_alpha;     /* clamped GLU sigmoid slope */
  int32_t reserved[3];
} moe_glu_cfg_t;

/* bf16: gate, up [ff, d]; down [d, ff]. */
typedef struct {
  const void* gate;
  const void* up;
  const void* down;
} moe_glu_weights_t;

/* Gradients of the weights, bf16, laid out as the weights. */
typedef struct {
  void* gate;
  void* up;
  void* down;
} moe_glu_grads_t;

/* Bytes of workspace that moe_glu_forward and moe_glu_backward need for T tokens, and
 * bytes of the buffer that a training forward pass leaves for its backward pass (h in
 * bf16 and g, u in fp32, in an order of the library's own).  0 if cfg is invalid or
 * T < 0.  Pure host functions. */
size_t moe_glu_workspace_bytes(const moe_glu_cfg_t* cfg, int32_t T);
size_t moe_glu_saved_bytes(const moe_glu_cfg_t* cfg, int32_t T);

/* y [T, d] bf16 = FFN(x [T, d] bf16).  saved: NULL, or a buffer of saved_bytes >=
 * moe_glu_saved_bytes(cfg, T) that receives what moe_glu_backward needs.  With saved
 * NULL small batches stream the weights through warp MMAs (any T gives the same result
 * to within rounding).  T == 0 is a no-op. */
int moe_glu_forward(const moe_glu_cfg_t* cfg, const void* x, int32_t T, const moe_glu_weights_t* w, void* y,
                    void* saved, size_t saved_bytes, void* ws, size_t ws_bytes, void* stream);

/* Gradients of moe_glu_forward, from the same x and w, its saved buffer and dy [T, d] bf16:
 *   dh = dy Wd;  dg = dh dact/dg;  du = dh dact/du  (0 where a clamp holds the value, its
 *   one-sided derivative 1 at the border itself; a g or u so near the border that its sum's
 *   rounding could decide is summed again with compensation by the forward pass);
 *   dx = dg Wg + du Wu;  dWg = dg^T x;  dWu = du^T x;  dWd = dy^T h.
 * dh stays in fp32; dg and du are rounded to bf16 for the products that follow.
 * dx [T, d] bf16 or NULL; grads or any member of it NULL: not computed.  With many tokens
 * and few weights the sum over the tokens is cut into parts, and which cut is taken depends
 * on the outputs asked for (their last bits may, with it).  Gradients are written, not
 * added to.  No output may share memory with an input or another output
 * (MOE_ERR_INVALID_ARG).  T == 0 sets the weight gradients to zero. */
int moe_glu_backward(const moe_glu_cfg_t* cfg, const void* x, int32_t T, const moe_glu_weights_t* w,
                     const void* saved, size_t saved_bytes, const void* dy, void* dx,
                     const moe_glu_grads_t* grads, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ norms of a block
 * n(v) = v / sqrt(mean(v^2) + eps) per row of d.  With the block's output `branch` z:
 *   p = n(z) * post_w   (post_w given; else p = z)
 *   c = branch_scale * sigmoid(gate[t])   (gate given; else c = branch_scale)
 *   y = residual_scale * x + c * p        (z given; without z: y = x)
 *   a = n(y) * pre_w                      (pre_w given: the input of the next block)
 * a is computed from y before y is rounded. */
typedef struct {
  int32_t d_model;       /* d, a positive multiple of 8, at most 16384 */
  float eps;             /* finite, >= 0 */
  float residual_scale;  /* finite */
  float branch_scale;    /* finite */
  int32_t reserved[4];
} moe_norm_cfg_t;

/* What the forward and backward passes read.  x, branch [T, d] bf16; post_w, pre_w [d]
 * bf16; gate [T] fp32.  Everything but x may be NULL; post_w and gate need branch, and
 * without branch pre_w is needed. */
typedef struct {
  const void* x;
  const void* branch;
  const void* post_w;
  const float* gate;
  const void* pre_w;
} moe_norm_inputs_t;

/* y [T, d] bf16 (with branch, else NULL), a [T, d] bf16 (with pre_w, else NULL).  y may be
 * x's buffer, a may be branch's.  T == 0 is a no-op. */
int moe_block_norm_forward(const moe_norm_cfg_t* cfg, const moe_norm_inputs_t* in, int32_t T, void* y, void* a,
                           void* stream);

/* Gradients; each output that is not NULL is written. */
typedef struct {
  void* dx;          /* bf16 [T, d] */
  void* dbranch;     /* bf16 [T, d], with branch */
  float* dgate;      /* fp32 [T], with gate */
  float* dpost_w;    /* fp32 [d], with post_w */
  float* dpre_w;     /* fp32 [d], with pre_w */
} moe_norm_grads_t;

/* Bytes of workspace that moe_block_norm_backward needs (0 if cfg is invalid or T < 0). */
size_t moe_block_norm_workspace_bytes(const moe_norm_cfg_t* cfg, int32_t T);

/* Gradients from dy [T, d] bf16 (with branch; NULL: zero) and da [T, d] bf16 (with pre_w;
 * NULL: zero); at least one of them is given.  y is recomputed from the inputs.  dx may be
 * dy's buffer, dbranch may be da's.  T == 0 sets dpost_w and dpre_w to zero. */
int moe_block_norm_backward(const moe_norm_cfg_t* cfg, const moe_norm_inputs_t* in, int32_t T, const void* dy,
                            const void* da, const moe_norm_grads_t* grads, void* ws, size_t ws_bytes,
                            void* stream);

/* ------------------------------------------------------------------ 4-bit linear layer
 *   y[t, o] = sum_g scale[o, g] * (sum_{k in group g} x[t, k] * (code[o, k] - zero[o, g]))
 * glu = 1: the matrix has 2 n_out rows, gate rows first, and y = act(gate, up) [T, n_out]. */
typedef struct {
  int32_t n_in;        /* a positive multiple of group, at most 2^29 */
  int32_t n_out;       /* columns of y, 1 to 2^30 */
  int32_t group;       /* inputs per scale: 32, 64 or 128 */
  int32_t glu;         /* 0 or 1 */
  int32_t act;         /* MOE_ACT_*, with glu */
  float glu_limit;
  float glu_alpha;
  int32_t reserved[1];
} moe_w4_cfg_t;

/* rows = n_out, or 2 n_out with glu.
 *   codes   u8 [rows, n_in / 2]: 4-bit codes, the low half holds the even input
 *   scales  bf16 [rows, n_in / group]
 *   zeros   u8 [rows, n_in / group], each 0..15 (the low four bits are read), or NULL: 8 */
typedef struct {
  const void* codes;
  const void* scales;
  const void* zeros;
} moe_w4_weights_t;

/* y [T, n_out] bf16 from x [T, n_in] bf16.  Made for the few tokens of a decode step: the
 * weights are read once per 16 tokens.  Needs no workspace.  y may not share memory with x
 * (MOE_ERR_INVALID_ARG).  T == 0 is a no-op. */
int moe_w4_linear(const moe_w4_cfg_t* cfg, const void* x, int32_t T, const moe_w4_weights_t* w, void* y,
                  void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_BLOCK_H_ */
