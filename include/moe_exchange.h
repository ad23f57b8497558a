/*
 * moe_exchange.h -- C ABI of the exchange around a sparse layer's experts, for GB300
 * (sm_103a): tokens sorted by expert, and the experts' rows back to their tokens with the
 * routing weights applied, both with their gradients.  Same library (libmoe.so), status
 * codes and conventions as moe_block.h: the caller owns every buffer, nothing
 * synchronises, work is enqueued on `stream` in order, matrices are row-major and every
 * tensor pointer is 16-byte aligned (MOE_ERR_ALIGNMENT).  On error nothing has been
 * enqueued unless the code is MOE_ERR_CUDA.  T == 0 is a no-op but for the offsets of
 * moe_dispatch_forward, which are set to zero.
 *
 * Slot t k + j is token t's j-th choice; S = T k.  Row rows[t, j] of the sorted matrices is
 * that slot's: the slots of expert 0 first, then those of expert 1 and so on, the slots of
 * one expert in increasing order (what moe_group_by_expert's perm says from the other end).
 * A slot whose expert lies outside [0, n_experts) has no row: its entry of rows is -1, it
 * adds nothing to sums, and its weight's gradient is 0.  (An entry of a caller's rows that
 * is not in [0, S) is taken for -1; two equal ones are the caller's mistake, and the
 * backward pass of the combination then leaves either gradient in that row.)  Rows behind
 * the last slot's are left as they are.
 *
 * Sums are fp32, in the order of j, rounded once to bf16, and no atomic touches them (the
 * sort's counts are whole numbers), so equal inputs give equal bits.  No output may share memory with an input or another output,
 * but for y and residual (MOE_ERR_INVALID_ARG).
 */
#ifndef MOE_EXCHANGE_H_
#define MOE_EXCHANGE_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  MOE_ROWS_BF16 = 0, /* rows of d bf16 */
  MOE_ROWS_E4M3 = 1  /* rows of d e4m3 and an fp32 scale each (dispatch forward alone) */
};

typedef struct {
  int32_t d_model;     /* d, a positive multiple of 8 (MOE_ROWS_E4M3: of 16), at most 2^29 */
  int32_t n_experts;   /* 1..1024 */
  int32_t top_k;       /* k, 1..32 */
  int32_t format;      /* MOE_ROWS_* */
  int32_t reserved[4]; /* zero */
} moe_exchange_cfg_t;

/* Bytes of workspace that moe_dispatch_forward needs (0 if cfg is invalid, T < 0 or
 * T k > 2^30).  Pure host function.  The workspace begins with the status word, which the
 * call clears (moe_device_status; nothing in the dispatch sets it). */
size_t moe_dispatch_workspace_bytes(const moe_exchange_cfg_t* cfg, int32_t T);

/* Sorts the slots of topk_ids [T, k] int32 and copies the rows of x [T, d]:
 *   offsets  int32 [n_experts + 1], out: expert e's rows are offsets[e] .. offsets[e + 1] - 1
 *   rows     int32 [T, k], out
 *   xs       [S, d], out: xs[rows[t, j]] = x[t]; NULL (with x NULL): only the sort
 *   x_scale  fp32 [T] and xs_scale fp32 [S], out: with MOE_ROWS_E4M3 and xs, else NULL */
int moe_dispatch_forward(const moe_exchange_cfg_t* cfg, const int32_t* topk_ids, const void* x, const float* x_scale,
                         int32_t T, int32_t* offsets, int32_t* rows, void* xs, float* xs_scale, void* ws,
                         size_t ws_bytes, void* stream);

/* dx [T, d] bf16: dx[t] = sum_j dxs[rows[t, j]], from dxs [S, d] bf16. */
int moe_dispatch_backward(const moe_exchange_cfg_t* cfg, const void* dxs, const int32_t* rows, int32_t T, void* dx,
                          void* stream);

/* y [T, d] bf16: y[t] = residual[t] + sum_j w[t, j] z[rows[t, j]], from the experts' rows
 * z [S, d] bf16.  w fp32 [T, k] or NULL (1); residual bf16 [T, d] or NULL (0), which may be
 * y's buffer. */
int moe_combine_forward(const moe_exchange_cfg_t* cfg, const void* z, const int32_t* rows, const float* w,
                        const void* residual, int32_t T, void* y, void* stream);

/* Gradients of moe_combine_forward from dy [T, d] bf16 (the residual's is dy itself):
 *   dz  bf16 [S, d] or NULL: dz[rows[t, j]] = w[t, j] dy[t]
 *   dw  fp32 [T, k] or NULL: dw[t, j] = sum_i dy[t, i] z[rows[t, j], i]  (z is read only here)
 * One of them at least is given.  w is needed: where the forward pass went without, ones. */
int moe_combine_backward(const moe_exchange_cfg_t* cfg, const void* dy, const void* z, const int32_t* rows,
                         const float* w, int32_t T, void* dz, float* dw, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_EXCHANGE_H_ */
