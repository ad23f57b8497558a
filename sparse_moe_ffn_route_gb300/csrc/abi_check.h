// Checks of arguments that the entry points of the dense block, the linear layer and the
// exchange share.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {

// The kernels count rows and columns in 32 bits and step a whole grid's rows (norms: 3 rows
// ahead of up to 2432 groups of threads) or a row's bytes (skinny.cu: 2 per input) past the
// last one before they compare.  These bounds keep every such sum below 2^31.  (What a tensor
// takes in bytes is counted in 64 bits.)
constexpr int kMaxTokens = 1 << 30, kMaxInputs = 1 << 29, kMaxOutputs = 1 << 30;

inline size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }

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

inline int check_tokens(int T) { return T < 0 ? MOE_ERR_INVALID_ARG : T > kMaxTokens ? MOE_ERR_UNSUPPORTED : MOE_OK; }

}  // namespace moe
