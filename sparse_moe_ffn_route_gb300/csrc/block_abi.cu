// C-ABI host layer of the dense block (include/moe_block.h): argument validation,
// workspace carving and the launch sequence of each entry point.
#include <cmath>

#include "block.h"

using namespace moe;

namespace {

// Tokens up to which a forward pass that keeps nothing streams the weights through warp
// MMAs (16 tokens a pass) instead of tcgen05 tiles of 128 token rows.
constexpr int kSkinnyTokens = 16;

// The kernels count rows and columns in 32 bits and step a whole grid's rows (norms: 3 rows
// ahead of up to 2432 groups of threads) or a row's bytes (skinny.cu: 2 per input) past the
// last one before they compare.  These bounds keep every such sum below 2^31.
constexpr int kMaxTokens = 1 << 30, kMaxInputs = 1 << 29, kMaxOutputs = 1 << 30;

size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }

// Null or 16-byte aligned.
template <typename... P>
bool aligned16(const P*... p) {
  return (((reinterpret_cast<uintptr_t>(p) & 15u) == 0) && ...);
}

// A buffer of a call.
struct Span {
  const void* at;
  size_t bytes;
};

// Whether any of `out` shares a byte with any of `in` or with another of `out`.
template <int NO, int NI>
bool overlap(const Span (&out)[NO], const Span (&in)[NI]) {
  auto share = [](const Span& a, const Span& b) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
    return p && q && p < q + b.bytes && q < p + a.bytes;
  };
  for (int i = 0; i < NO; ++i) {
    for (const Span& b : in)
      if (share(out[i], b)) return true;
    for (int j = i + 1; j < NO; ++j)
      if (share(out[i], out[j])) return true;
  }
  return false;
}

#define BLOCK_CUDA(call)                            \
  do {                                              \
    if ((call) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

int check_act(int act, float limit, float alpha) {
  if (act != MOE_ACT_SWIGLU && act != MOE_ACT_CLAMPED_GLU) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(limit) || !std::isfinite(alpha) || limit < 0.f) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int check_tokens(int T) { return T < 0 ? MOE_ERR_INVALID_ARG : T > kMaxTokens ? MOE_ERR_UNSUPPORTED : MOE_OK; }

int check_glu(const moe_glu_cfg_t* c) {
  if (!c || c->d_model <= 0 || c->ff <= 0) return MOE_ERR_INVALID_ARG;
  for (int r : c->reserved)
    if (r) return MOE_ERR_INVALID_ARG;
  const int st = check_act(c->act, c->glu_limit, c->glu_alpha);
  if (st != MOE_OK) return st;
  return c->d_model % 8 || c->ff % 8 || c->d_model > kMaxInputs || c->ff > kMaxInputs ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Workspace: status word | h [T, ff] (forward that keeps nothing), norms (forward that keeps,
// clamped) or dg, du [T, ff] | the backward pass's counts and partial sums of split products.
struct GluLayout {
  size_t status, h, norms, dg, du, arrived, partial, total;
};

GluLayout glu_layout(const moe_glu_cfg_t& c, int T) {
  const size_t a = align_up((size_t)T * c.ff * 2);
  GluLayout L;
  L.status = 0;
  L.h = L.norms = L.dg = 256;
  L.du = L.dg + a;
  L.arrived = L.du + a;
  const size_t split = (size_t)glu_split_tiles(c.d_model, c.ff, T);
  L.partial = L.arrived + (split ? align_up(kGluArrivedBytes) : 0);
  L.total = L.partial + split * kGluSplitBytes;
  const size_t norms = c.act == MOE_ACT_CLAMPED_GLU ? align_up(((size_t)T + 2 * (size_t)c.ff) * 4) : 0;
  if (L.total < L.norms + norms) L.total = L.norms + norms;
  return L;
}

// Saved: h bf16 [T, ff] | g | u, fp32 in blocks of 128 tokens.
struct SavedLayout {
  size_t g, u, total;
};

SavedLayout saved_layout(const moe_glu_cfg_t& c, int T) {
  const size_t blk = ((size_t)T + 127) / 128 * 128 * c.ff * 4;
  SavedLayout L;
  L.g = align_up((size_t)T * c.ff * 2);
  L.u = L.g + blk;
  L.total = L.u + blk;
  return L;
}

GluSaved saved_at(void* base, const SavedLayout& L) {
  char* p = static_cast<char*>(base);
  return GluSaved{reinterpret_cast<uint16_t*>(p), reinterpret_cast<float*>(p + L.g), reinterpret_cast<float*>(p + L.u)};
}

GluParams glu_params(const moe_glu_cfg_t& c, const moe_glu_weights_t& w) {
  return GluParams{static_cast<const uint16_t*>(w.gate), static_cast<const uint16_t*>(w.up),
                   static_cast<const uint16_t*>(w.down), c.d_model, c.ff, c.act, c.glu_limit, c.glu_alpha};
}

int check_glu_weights(const moe_glu_weights_t* w) {
  if (!w || !w->gate || !w->up || !w->down) return MOE_ERR_INVALID_ARG;
  return aligned16(w->gate, w->up, w->down) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

int check_norm(const moe_norm_cfg_t* c) {
  if (!c || c->d_model <= 0) return MOE_ERR_INVALID_ARG;
  for (int r : c->reserved)
    if (r) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->eps) || c->eps < 0.f || !std::isfinite(c->residual_scale) || !std::isfinite(c->branch_scale))
    return MOE_ERR_INVALID_ARG;
  return c->d_model % 8 || c->d_model > 16384 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_norm_inputs(const moe_norm_inputs_t* in) {
  if (!in || !in->x) return MOE_ERR_INVALID_ARG;
  if (!in->branch && (in->post_w || in->gate || !in->pre_w)) return MOE_ERR_INVALID_ARG;
  return aligned16(in->x, in->branch, in->post_w, in->gate, in->pre_w) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

}  // namespace

extern "C" {

size_t moe_glu_workspace_bytes(const moe_glu_cfg_t* cfg, int32_t T) {
  return check_glu(cfg) != MOE_OK || check_tokens(T) != MOE_OK ? 0 : glu_layout(*cfg, T).total;
}

size_t moe_glu_saved_bytes(const moe_glu_cfg_t* cfg, int32_t T) {
  return check_glu(cfg) != MOE_OK || check_tokens(T) != MOE_OK ? 0 : align_up(saved_layout(*cfg, T).total) + 256;
}

int moe_glu_forward(const moe_glu_cfg_t* cfg, const void* x, int32_t T, const moe_glu_weights_t* w, void* y,
                    void* saved, size_t saved_bytes, void* ws, size_t ws_bytes, void* stream) {
  int st = check_glu(cfg);
  if (st != MOE_OK || (st = check_tokens(T)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!x || !y || !ws) return MOE_ERR_INVALID_ARG;
  if ((st = check_glu_weights(w)) != MOE_OK) return st;
  if (!aligned16(x, y, saved, ws)) return MOE_ERR_ALIGNMENT;
  const GluLayout L = glu_layout(*cfg, T);
  if (ws_bytes < L.total || (saved && saved_bytes < moe_glu_saved_bytes(cfg, T))) return MOE_ERR_WORKSPACE;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const GluParams p = glu_params(*cfg, *w);
  char* base = static_cast<char*>(ws);
  uint32_t* status = reinterpret_cast<uint32_t*>(base + L.status);
  const uint16_t* xi = static_cast<const uint16_t*>(x);
  uint16_t* yo = static_cast<uint16_t*>(y);
  if (!saved && T <= kSkinnyTokens) {
    uint16_t* h = reinterpret_cast<uint16_t*>(base + L.h);
    // Few products per output leave h's rounding to bf16 visible beside y's own (1.6 times
    // y's error alone at one token and ff 512), so h then keeps its low half as well; over
    // more the roundings average out to 1.4 times, as on the path of the large batches.
    uint16_t* lo = T <= 8 && p.ff <= 4096 ? reinterpret_cast<uint16_t*>(base + L.du) : nullptr;
    BLOCK_CUDA(launch_skinny_bf16(p.gate, p.up, p.ff, p.d, xi, nullptr, T, &p, h, lo, status, false, s));
    BLOCK_CUDA(launch_skinny_bf16(p.down, nullptr, p.d, p.ff, h, lo, T, nullptr, yo, nullptr, nullptr, true, s));
    return MOE_OK;
  }
  GluSaved sv{reinterpret_cast<uint16_t*>(base + L.h), nullptr, nullptr};
  if (saved) sv = saved_at(saved, saved_layout(*cfg, T));
  BLOCK_CUDA(launch_glu_gate_up(p, xi, T, sv.h, sv.g, sv.u, reinterpret_cast<float*>(base + L.norms), status, s));
  BLOCK_CUDA(launch_glu_down(p, sv.h, T, yo, status, s));
  return MOE_OK;
}

int moe_glu_backward(const moe_glu_cfg_t* cfg, const void* x, int32_t T, const moe_glu_weights_t* w,
                     const void* saved, size_t saved_bytes, const void* dy, void* dx,
                     const moe_glu_grads_t* grads, void* ws, size_t ws_bytes, void* stream) {
  int st = check_glu(cfg);
  if (st != MOE_OK || (st = check_tokens(T)) != MOE_OK) return st;
  const moe_glu_grads_t none{nullptr, nullptr, nullptr};
  const moe_glu_grads_t& dw = grads ? *grads : none;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!aligned16(dw.gate, dw.up, dw.down)) return MOE_ERR_ALIGNMENT;
  if (T == 0) {
    const size_t n = (size_t)cfg->d_model * cfg->ff * 2;
    for (void* p : {dw.gate, dw.up, dw.down})
      if (p) BLOCK_CUDA(cudaMemsetAsync(p, 0, n, s));
    return MOE_OK;
  }
  if (!x || !saved || !dy || !ws) return MOE_ERR_INVALID_ARG;
  if ((st = check_glu_weights(w)) != MOE_OK) return st;
  if (!aligned16(x, saved, dy, dx, ws)) return MOE_ERR_ALIGNMENT;
  const GluLayout L = glu_layout(*cfg, T);
  if (ws_bytes < L.total || saved_bytes < moe_glu_saved_bytes(cfg, T)) return MOE_ERR_WORKSPACE;
  // The products run side by side in one launch: what one of them writes another still reads.
  const size_t rows = (size_t)T * cfg->d_model * 2, matrix = (size_t)cfg->d_model * cfg->ff * 2;
  const Span out[] = {{dx, rows}, {dw.gate, matrix}, {dw.up, matrix}, {dw.down, matrix}, {ws, L.total}};
  const Span in[] = {{x, rows},          {dy, rows},         {w->gate, matrix},
                     {w->up, matrix},    {w->down, matrix},  {saved, moe_glu_saved_bytes(cfg, T)}};
  if (overlap(out, in)) return MOE_ERR_INVALID_ARG;
  const GluParams p = glu_params(*cfg, *w);
  char* base = static_cast<char*>(ws);
  uint32_t* status = reinterpret_cast<uint32_t*>(base + L.status);
  uint16_t* dg = reinterpret_cast<uint16_t*>(base + L.dg);
  uint16_t* du = reinterpret_cast<uint16_t*>(base + L.du);
  const GluSaved sv = saved_at(const_cast<void*>(saved), saved_layout(*cfg, T));
  const uint16_t* dyi = static_cast<const uint16_t*>(dy);
  const GluSplit split{reinterpret_cast<float*>(base + L.partial), reinterpret_cast<uint32_t*>(base + L.arrived)};
  BLOCK_CUDA(launch_glu_backward(p, static_cast<const uint16_t*>(x), dyi, T, sv, dg, du, static_cast<uint16_t*>(dx),
                                 static_cast<uint16_t*>(dw.gate), static_cast<uint16_t*>(dw.up),
                                 static_cast<uint16_t*>(dw.down), split, status, s));
  return MOE_OK;
}

int moe_block_norm_forward(const moe_norm_cfg_t* cfg, const moe_norm_inputs_t* in, int32_t T, void* y, void* a,
                           void* stream) {
  int st = check_norm(cfg);
  if (st != MOE_OK || (st = check_tokens(T)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if ((st = check_norm_inputs(in)) != MOE_OK) return st;
  if ((in->branch != nullptr) != (y != nullptr) || (in->pre_w != nullptr) != (a != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y, a)) return MOE_ERR_ALIGNMENT;
  BLOCK_CUDA(launch_block_norm_fwd(*cfg, *in, T, static_cast<uint16_t*>(y), static_cast<uint16_t*>(a),
                                   static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

size_t moe_block_norm_workspace_bytes(const moe_norm_cfg_t* cfg, int32_t T) {
  if (check_norm(cfg) != MOE_OK || check_tokens(T) != MOE_OK) return 0;
  return 256 + (size_t)block_norm_parts(T) * 2 * cfg->d_model * 4;
}

int moe_block_norm_backward(const moe_norm_cfg_t* cfg, const moe_norm_inputs_t* in, int32_t T, const void* dy,
                            const void* da, const moe_norm_grads_t* grads, void* ws, size_t ws_bytes,
                            void* stream) {
  int st = check_norm(cfg);
  if (st != MOE_OK || (st = check_tokens(T)) != MOE_OK) return st;
  if (!grads) return MOE_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const moe_norm_grads_t& o = *grads;
  if (!aligned16(dy, da, o.dx, o.dbranch, o.dgate, o.dpost_w, o.dpre_w)) return MOE_ERR_ALIGNMENT;
  if (T == 0) {
    for (float* p : {o.dpost_w, o.dpre_w})
      if (p) BLOCK_CUDA(cudaMemsetAsync(p, 0, (size_t)cfg->d_model * 4, s));
    return MOE_OK;
  }
  if ((st = check_norm_inputs(in)) != MOE_OK) return st;
  if ((!dy && !da) || (dy && !in->branch) || (da && !in->pre_w)) return MOE_ERR_INVALID_ARG;
  if ((o.dbranch && !in->branch) || (o.dgate && !in->gate) || (o.dpost_w && !in->post_w) || (o.dpre_w && !in->pre_w))
    return MOE_ERR_INVALID_ARG;
  if (o.dpost_w || o.dpre_w) {
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned16(ws)) return MOE_ERR_ALIGNMENT;
    if (ws_bytes < moe_block_norm_workspace_bytes(cfg, T)) return MOE_ERR_WORKSPACE;
  }
  BLOCK_CUDA(launch_block_norm_bwd(*cfg, *in, T, static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(da), o,
                                   static_cast<float*>(ws), s));
  return MOE_OK;
}

int moe_w4_linear(const moe_w4_cfg_t* c, const void* x, int32_t T, const moe_w4_weights_t* w, void* y, void* stream) {
  if (!c || c->n_in <= 0 || c->n_out <= 0 || c->glu < 0 || c->glu > 1 || c->reserved[0]) return MOE_ERR_INVALID_ARG;
  const int st = check_act(c->act, c->glu_limit, c->glu_alpha);
  if (st != MOE_OK) return st;
  if (c->group != 32 && c->group != 64 && c->group != 128) return MOE_ERR_UNSUPPORTED;
  if (c->n_in % c->group || c->n_in > kMaxInputs || c->n_out > kMaxOutputs) return MOE_ERR_UNSUPPORTED;
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !y || !w || !w->codes || !w->scales) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x, y, w->codes, w->scales, w->zeros)) return MOE_ERR_ALIGNMENT;
  // Every CTA reads all of x and writes its columns of y.
  const Span out[] = {{y, (size_t)T * c->n_out * 2}}, in[] = {{x, (size_t)T * c->n_in * 2}};
  if (overlap(out, in)) return MOE_ERR_INVALID_ARG;
  BLOCK_CUDA(launch_skinny_w4(*c, *w, static_cast<const uint16_t*>(x), T, static_cast<uint16_t*>(y),
                              static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

}  // extern "C"
