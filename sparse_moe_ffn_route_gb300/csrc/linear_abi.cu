// C-ABI host layer of the linear layer and of the norm with an output in 8 bits
// (include/moe_linear.h): argument validation, workspace carving and launches.
#include <cmath>

#include "abi_check.h"
#include "block.h"
#include "linear_act.cuh"

using namespace moe;

namespace {

#define LINEAR_CUDA(call)                           \
  do {                                              \
    if ((call) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

int check_linear(const moe_linear_cfg_t* c) {
  if (!c || c->n_in <= 0 || c->n_out <= 0 || c->glu < 0 || c->glu > 1) return MOE_ERR_INVALID_ARG;
  if (c->format != MOE_LINEAR_BF16 && c->format != MOE_LINEAR_E4M3) return MOE_ERR_INVALID_ARG;
  if (c->act < 0 || c->act > (c->glu ? (int)MOE_ACT_CLAMPED_GLU : (int)MOE_LINEAR_GELU_TANH)) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->glu_limit) || !std::isfinite(c->glu_alpha) || c->glu_limit < 0.f) return MOE_ERR_INVALID_ARG;
  for (int r : c->reserved)
    if (r) return MOE_ERR_INVALID_ARG;
  if (c->n_in % (c->format == MOE_LINEAR_E4M3 ? 16 : 8) || c->n_out % 8) return MOE_ERR_UNSUPPORTED;
  return c->n_in > kMaxInputs || c->n_out > (c->glu ? kMaxInputs / 2 : kMaxInputs) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Status word | backward pass (bf16, no glu): dv | partial sums of the bias's gradient | the
// counts and partial sums of a split weight gradient.
struct Layout {
  size_t dv, bias, arrived, partial, total;
};

Layout layout(const moe_linear_cfg_t& c, int T) {
  Layout L{256, 256, 256, 256, 256};
  if (T == 0 || c.glu || c.format != MOE_LINEAR_BF16) return L;
  L.bias = L.dv + (c.act == MOE_LINEAR_NONE ? 0 : align_up((size_t)T * c.n_out * 2));
  L.arrived = L.bias + align_up((size_t)linear_bias_parts(c.n_out, T) * c.n_out * 4);
  const size_t split = (size_t)linear_split_tiles(c.n_in, c.n_out, T);
  L.partial = L.arrived + (split ? align_up(kGluArrivedBytes) : 0);
  L.total = L.partial + split * kGluSplitBytes;
  return L;
}

LinearShape shape(const moe_linear_cfg_t& c) { return LinearShape{c.n_in, c.n_out, c.format == MOE_LINEAR_E4M3}; }

}  // namespace

extern "C" {

int moe_block_norm_quant(const moe_norm_cfg_t* c, const moe_norm_inputs_t* in, int32_t T, void* y, void* q,
                         float* scale, void* stream) {
  if (!c || c->d_model <= 0) return MOE_ERR_INVALID_ARG;
  for (int r : c->reserved)
    if (r) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->eps) || c->eps < 0.f || !std::isfinite(c->residual_scale) || !std::isfinite(c->branch_scale))
    return MOE_ERR_INVALID_ARG;
  if (c->d_model % 8 || c->d_model > 16384) return MOE_ERR_UNSUPPORTED;
  const int st = check_tokens(T);
  if (st != MOE_OK || T == 0) return st;
  if (!in || !in->x || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (!in->branch && (in->post_w || in->gate)) return MOE_ERR_INVALID_ARG;
  if ((in->branch != nullptr) != (y != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(in->x, in->branch, in->post_w, in->gate, in->pre_w, y, q, scale)) return MOE_ERR_ALIGNMENT;
  const size_t row = (size_t)c->d_model, rows = (size_t)T * row;
  // A row's codes are written while other rows are still read.
  const Span out[] = {{q, rows}, {scale, (size_t)T * 4}, {y, rows * 2}};
  const Span ins[] = {{y == in->x ? nullptr : in->x, rows * 2}, {in->branch, rows * 2}, {in->post_w, row * 2},
                      {in->gate, (size_t)T * 4},                {in->pre_w, row * 2}};
  if (overlap(out, ins)) return MOE_ERR_INVALID_ARG;
  LINEAR_CUDA(launch_block_norm_quant(*c, *in, T, static_cast<uint16_t*>(y), static_cast<uint8_t*>(q), scale,
                                      static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

size_t moe_linear_workspace_bytes(const moe_linear_cfg_t* cfg, int32_t T) {
  return check_linear(cfg) != MOE_OK || check_tokens(T) != MOE_OK ? 0 : layout(*cfg, T).total;
}

int moe_linear_forward(const moe_linear_cfg_t* cfg, const void* x, const float* x_scale, int32_t T,
                       const moe_linear_weights_t* w, const void* residual, void* y, void* pre, void* ws,
                       size_t ws_bytes, void* stream) {
  int st = check_linear(cfg);
  if (st != MOE_OK || (st = check_tokens(T)) != MOE_OK || T == 0) return st;
  const bool eight = cfg->format == MOE_LINEAR_E4M3;
  if (!x || !w || !w->w || !y || !ws || (eight != (x_scale != nullptr)) || (eight != (w->scale != nullptr)) || (pre && cfg->glu))
    return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(x_scale) & 3u) return MOE_ERR_ALIGNMENT;
  if (!aligned16(x, w->w, w->scale, w->bias, residual, y, pre, ws)) return MOE_ERR_ALIGNMENT;
  if (ws_bytes < 256) return MOE_ERR_WORKSPACE;
  const size_t rows = (size_t)cfg->n_out * (cfg->glu ? 2 : 1), each = eight ? 1 : 2, outs = (size_t)T * cfg->n_out * 2;
  const Span out[] = {{y, outs}, {pre, outs}, {ws, 256}};
  const Span in[] = {{x, (size_t)T * cfg->n_in * each}, {x_scale, (size_t)T * 4}, {w->w, rows * cfg->n_in * each},
                     {w->scale, rows * 4}, {w->bias, rows * 2}, {residual == y ? nullptr : residual, outs}};
  if (overlap(out, in)) return MOE_ERR_INVALID_ARG;
  LinearEpi e{};
  e.act = cfg->act;
  e.glu = cfg->glu;
  e.gated = GluAct{cfg->act, cfg->glu_limit, cfg->glu_alpha};
  e.bias = static_cast<const uint16_t*>(w->bias);
  e.residual = static_cast<const uint16_t*>(residual);
  e.pre = static_cast<uint16_t*>(pre);
  e.x_scale = x_scale;
  e.w_scale = w->scale;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t* status = static_cast<uint32_t*>(ws);
  if (linear_streams(shape(*cfg), T, cfg->glu))
    LINEAR_CUDA(launch_linear_stream(shape(*cfg), x, T, w->w, static_cast<uint16_t*>(y), e, status, s));
  else
    LINEAR_CUDA(launch_linear_gemm(shape(*cfg), x, T, w->w, static_cast<uint16_t*>(y), e, status, s));
  return MOE_OK;
}

int moe_linear_backward(const moe_linear_cfg_t* cfg, const void* x, int32_t T, const moe_linear_weights_t* w,
                        const void* pre, const void* dy, void* dx, const moe_linear_grads_t* grads, void* ws,
                        size_t ws_bytes, void* stream) {
  int st = check_linear(cfg);
  if (st != MOE_OK || (st = check_tokens(T)) != MOE_OK) return st;
  if (cfg->glu || cfg->format != MOE_LINEAR_BF16) return MOE_ERR_UNSUPPORTED;
  const moe_linear_grads_t none{nullptr, nullptr};
  const moe_linear_grads_t& g = grads ? *grads : none;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!aligned16(g.w, g.bias)) return MOE_ERR_ALIGNMENT;
  const size_t matrix = (size_t)cfg->n_in * cfg->n_out * 2, bias = (size_t)cfg->n_out * 2;
  if (T == 0) {
    if (g.w) LINEAR_CUDA(cudaMemsetAsync(g.w, 0, matrix, s));
    if (g.bias) LINEAR_CUDA(cudaMemsetAsync(g.bias, 0, bias, s));
    return MOE_OK;
  }
  const bool act = cfg->act != MOE_LINEAR_NONE;
  if (!x || !w || !w->w || !dy || !ws || (act && !pre)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x, w->w, pre, dy, dx, ws)) return MOE_ERR_ALIGNMENT;
  const Layout L = layout(*cfg, T);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  // The products run side by side in one launch: what one of them writes another still reads.
  const size_t ins = (size_t)T * cfg->n_in * 2, outs = (size_t)T * cfg->n_out * 2;
  const Span out[] = {{dx, ins}, {g.w, matrix}, {g.bias, bias}, {ws, L.total}};
  const Span in[] = {{x, ins}, {w->w, matrix}, {act ? pre : nullptr, outs}, {dy, outs}};
  if (overlap(out, in)) return MOE_ERR_INVALID_ARG;
  char* base = static_cast<char*>(ws);
  uint32_t *status = reinterpret_cast<uint32_t*>(base), *arrived = reinterpret_cast<uint32_t*>(base + L.arrived);
  const bool products = dx || g.w;
  const LinearPlan plan = products ? plan_linear_backward(shape(*cfg), T, dx, g.w) : LinearPlan{};
  const int zeros = plan.parts > 1 ? (int)(kGluArrivedBytes / 4) : 0;
  const uint16_t* dv = static_cast<const uint16_t*>(dy);
  float* parts = reinterpret_cast<float*>(base + L.bias);
  const BiasParts sums{g.bias ? parts : nullptr, linear_bias_parts(cfg->n_out, T), cfg->n_out, static_cast<uint16_t*>(g.bias)};
  if (g.bias || (act && products)) {
    uint16_t* out_dv = act && products ? reinterpret_cast<uint16_t*>(base + L.dv) : nullptr;
    LINEAR_CUDA(launch_linear_dv(cfg->act, dv, static_cast<const uint16_t*>(pre), T, cfg->n_out, out_dv,
                                 g.bias ? parts : nullptr, status, arrived, zeros, s));
    if (out_dv) dv = out_dv;
  } else if (zeros) {
    LINEAR_CUDA(cudaMemsetAsync(arrived, 0, kGluArrivedBytes, s));
  }
  if (products)
    LINEAR_CUDA(launch_linear_backward(shape(*cfg), plan, static_cast<const uint16_t*>(x), T, static_cast<const uint16_t*>(w->w), dv,
                                       static_cast<uint16_t*>(dx), static_cast<uint16_t*>(g.w),
                                       GluSplit{reinterpret_cast<float*>(base + L.partial), arrived}, sums, status, s));
  else if (g.bias)
    LINEAR_CUDA(launch_linear_dbias(sums, s));
  return MOE_OK;
}

}  // extern "C"
