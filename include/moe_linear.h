/*
 * moe_linear.h -- C ABI of the linear layer with bias, activation and residual in its
 * epilogue, for GB300 (sm_103a): in bf16, forward and backward, and with operands in 8
 * bits (e4m3 with a scale per row), which the norm here writes.  Same library
 * (libmoe.so), status codes and conventions as moe_block.h: the caller owns every buffer,
 * nothing synchronises, work is enqueued on `stream` in order, matrices are row-major,
 * weight matrices are row = output, column = input, and every tensor pointer is 16-byte
 * aligned (MOE_ERR_ALIGNMENT).  On error nothing has been enqueued unless the code is
 * MOE_ERR_CUDA.  Reserved members must be zero.  Up to 2^30 tokens (MOE_ERR_UNSUPPORTED
 * past that).  T == 0 is a no-op but for the weights' gradients, which are set to zero.
 *
 * Sums, statistics and activations are fp32; results are rounded once to their type, to
 * nearest even.  All reductions run in a fixed order, so equal inputs give equal bits.
 * Infinities and NaN in an input pass through as the formulas say.
 */
#ifndef MOE_LINEAR_H_
#define MOE_LINEAR_H_

#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ 8 bits
 * A row of d values a as e4m3 codes q with one fp32 scale:
 *   scale = max(max_i |a_i| / 448, 2^-126);  q_i = a_i / scale to the nearest e4m3 value
 * so that scale q_i stands for a_i.  A NaN is passed over by the maximum and keeps its own
 * place; an infinity makes its row's scale infinite (and the row, times it, NaN).
 *
 * moe_block_norm_forward (moe_block.h) whose a is written in 8 bits: the same configuration and
 * inputs, and y [T, d] bf16 (with branch, else NULL), q [T, d] e4m3, scale fp32 [T].
 * Without pre_w there is no second norm: a = y (or x, without branch), so that x alone is
 * a matrix taken to 8 bits.  a is not rounded to bf16 on the way.  y may be x's buffer. */
int moe_block_norm_quant(const moe_norm_cfg_t* cfg, const moe_norm_inputs_t* in, int32_t T, void* y, void* q,
                         float* scale, void* stream);

/* ------------------------------------------------------------------ linear layer
 *   v = x W^T + bias;  y = act(v) + residual
 * glu = 1: W has 2 n_out rows (and bias 2 n_out values), gate rows first, and
 *   y = act(v_gate, v_up) + residual, act as in moe_glu_forward.
 * MOE_LINEAR_E4M3: x and W are e4m3 with fp32 scales of their rows, which multiply the sums:
 *   v[t, o] = x_scale[t] w_scale[o] sum_k x[t, k] W[o, k] + bias[o] */
enum {
  MOE_LINEAR_BF16 = 0,
  MOE_LINEAR_E4M3 = 1
};
enum {
  MOE_LINEAR_NONE = 0,
  MOE_LINEAR_SILU = 1,      /* v sigmoid(v) */
  MOE_LINEAR_GELU = 2,      /* v (1 + erf(v / sqrt 2)) / 2 */
  MOE_LINEAR_GELU_TANH = 3  /* v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2 */
};

typedef struct {
  int32_t n_in;      /* a positive multiple of 8 (MOE_LINEAR_E4M3: of 16), at most 2^29 */
  int32_t n_out;     /* columns of y, a positive multiple of 8, at most 2^29 (glu: 2^28) */
  int32_t format;    /* MOE_LINEAR_BF16 or MOE_LINEAR_E4M3 */
  int32_t glu;       /* 0 or 1 */
  int32_t act;       /* MOE_LINEAR_NONE .. GELU_TANH, or, with glu, MOE_ACT_* */
  float glu_limit;   /* with glu: clamped GLU limit, >= 0 */
  float glu_alpha;   /* with glu: clamped GLU sigmoid slope */
  int32_t reserved[5];
} moe_linear_cfg_t;

typedef struct {
  const void* w;        /* bf16 or e4m3 [rows, n_in] */
  const float* scale;   /* fp32 [rows] with MOE_LINEAR_E4M3, else NULL */
  const void* bias;     /* bf16 [rows] or NULL */
} moe_linear_weights_t;

/* Bytes of workspace that moe_linear_forward and moe_linear_backward need for T tokens.
 * 0 if cfg is invalid or T < 0 or too many.  Pure host function. */
size_t moe_linear_workspace_bytes(const moe_linear_cfg_t* cfg, int32_t T);

/* y [T, n_out] bf16 from x [T, n_in] (x_scale fp32 [T] with MOE_LINEAR_E4M3, else NULL).
 * residual bf16 [T, n_out] or NULL; it may be y's buffer.  pre: NULL, or bf16 [T, n_out]
 * (glu = 0) that receives v rounded, for moe_linear_backward.  x_scale need only be aligned to
 * 4 bytes, so that a run of sorted rows (moe_exchange.h) can be passed.  Otherwise no output may share
 * memory with an input or another output (MOE_ERR_INVALID_ARG). */
int moe_linear_forward(const moe_linear_cfg_t* cfg, const void* x, const float* x_scale, int32_t T,
                       const moe_linear_weights_t* w, const void* residual, void* y, void* pre, void* ws,
                       size_t ws_bytes, void* stream);

/* Gradients, bf16, laid out as what they belong to. */
typedef struct {
  void* w;      /* [n_out, n_in] */
  void* bias;   /* [n_out] */
} moe_linear_grads_t;

/* Gradients of moe_linear_forward in bf16 without glu (others: MOE_ERR_UNSUPPORTED), from the
 * same x and w (its bias is not read), dy [T, n_out] bf16 and, with an activation, the pre of
 * the forward pass (else NULL):
 *   dv = dy act'(pre);  dx = dv W;  dW = dv^T x;  dbias = sum_t dv
 * (the residual's gradient is dy itself).  With an activation dv is rounded to bf16 for the
 * products; dbias sums it unrounded.  dx [T, n_in] bf16 or NULL; grads or any member of it
 * NULL: not computed.  x and w->w are needed whichever of them are asked for.  Gradients are
 * written, not added to.  With many tokens and few
 * weights the sum over the tokens is cut into parts, and which cut is taken depends on the
 * outputs asked for.  No output may share memory with an input or another output
 * (MOE_ERR_INVALID_ARG). */
int moe_linear_backward(const moe_linear_cfg_t* cfg, const void* x, int32_t T, const moe_linear_weights_t* w,
                        const void* pre, const void* dy, void* dx, const moe_linear_grads_t* grads, void* ws,
                        size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_LINEAR_H_ */
