// How linear_stream.cu cuts a product among the warps of a CTA.  Plain host code: the sums of
// bytes that have to fit in shared memory are formed in 64 bits, since x alone passes 2^31 bytes
// within the sizes that the linear layer takes.
#pragma once

#include <algorithm>

namespace moe {

constexpr int kStreamWarps = 16, kStepBytes = 128, kSlotBytes = 16 * kStepBytes, kMostDepth = 12;
constexpr int kStreamSpace = 227 * 1024;
constexpr int kXPad = 64;        // x's rows are a multiple of 128 bytes and this apart
constexpr int kRedPitch = 17;    // floats of a token in a warp's partial sums

// What of a product a CTA does at one time.  Sizes in bytes of k.
struct Cut {
  int slots, ws;               // tiles at one time, warps to a tile
  int depth;                   // steps ahead
  int steps, phase_steps;      // of k in all, and of x in shared memory at one time
};

// Bytes of a run of steps of x's T (1 to 16) rows.
inline long long stream_x_bytes(int T, long long steps) { return T * (steps * kStepBytes + kXPad); }

// The cut for T tokens, rows of `row` bytes, a CTA's share of `share` features in tiles of
// `features`, and shared memory for it, with partial sums of tok tokens (8 or 16).
inline Cut stream_cut(int T, int row, int share, int features, int tok, int& smem) {
  Cut c;
  c.steps = (row + kStepBytes - 1) / kStepBytes;
  c.slots = std::min((share + features - 1) / features, kStreamWarps);
  c.ws = std::min(kStreamWarps / c.slots, c.steps);
  const int warps = c.slots * c.ws, per = warps * kSlotBytes;
  c.phase_steps = (c.steps + c.ws - 1) / c.ws * c.ws;
  // as many steps ahead as there is room for beside x; where that is less than two, x comes in
  // phases of k beside four
  const int most = std::min(kMostDepth, c.phase_steps / c.ws), least = std::min(2, c.phase_steps / c.ws);
  const long long room = kStreamSpace - stream_x_bytes(T, c.phase_steps);
  c.depth = room < (long long)least * per ? 0 : (int)std::min<long long>(most, room / per);
  if (c.depth < least) {
    c.depth = 4;
    c.phase_steps = ((kStreamSpace - c.depth * per) / T - kXPad) / kStepBytes / c.ws * c.ws;
  }
  smem = (int)std::max<long long>((long long)c.depth * per + stream_x_bytes(T, c.phase_steps), warps * tok * kRedPitch * 4);
  return c;
}

}  // namespace moe
