"""How the linear layer's kernel for few tokens cuts a product: what it keeps in shared memory fits there,
at every size that the entry point takes.  The header that makes the cut is compiled and run here."""
import os
import subprocess

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include "stream_cut.h"
using namespace moe;

static long long bad = 0, seen = 0, phased = 0;

static void look(int T, int row, int share, int features) {
  const int tok = T > 8 ? 16 : 8;
  int smem = -1;
  const Cut c = stream_cut(T, row, share, features, tok, smem);
  const long long warps = (long long)c.slots * c.ws, rings = warps * c.depth * kSlotBytes;
  const long long x = (long long)T * ((long long)c.phase_steps * kStepBytes + kXPad);
  const long long sums = warps * tok * kRedPitch * 4;
  const long long phases = c.phase_steps > 0 ? ((long long)c.steps + c.phase_steps - 1) / c.phase_steps : 0;
  const bool ok = c.slots >= 1 && c.ws >= 1 && warps <= kStreamWarps && c.depth >= 1 && c.depth <= kMostDepth && c.phase_steps >= c.ws &&
                  c.phase_steps % c.ws == 0 && rings + x <= smem && sums <= smem && smem <= kStreamSpace &&
                  (long long)c.steps * kStepBytes >= row && phases * c.phase_steps >= c.steps &&
                  // what the kernel counts in 32 bits: bytes of k past the last phase, steps ahead of it
                  (phases * c.phase_steps + kMostDepth) * kStepBytes <= 0x7fffffffLL;
  ++seen;
  phased += phases > 1;
  if (!ok && bad++ < 5)
    std::printf("T %d row %d share %d: slots %d ws %d depth %d steps %d phase %d smem %d\n", T, row, share, c.slots, c.ws, c.depth, c.steps,
                c.phase_steps, smem);
}

int main() {
  const int shares[] = {1, 4, 7, 8, 9, 16, 27, 64, 100, 127, 128, 129, 255, 256, 1000, 1 << 22};
  for (int T = 1; T <= 16; ++T)
    for (int features = 8; features <= 16; features += 8)
      for (int share : shares) {
        for (int row = 16; row <= 1 << 16; row += row < 4096 ? 16 : 496) look(T, row, share, features);
        // up to 2^29 inputs of 2 bytes: around the powers of two, and where T rows pass 2^31
        for (int e = 16; e <= 30; ++e)
          for (long long by : {-4096LL, -128LL, -16LL, 0LL, 16LL, 128LL, 1LL << (e - 1)})
            if ((1LL << e) + by <= 1LL << 30) look(T, (int)((1LL << e) + by), share, features);
        for (int i = 1; i <= 4; ++i)
          for (int by = -256; by <= 256; by += 16) {
            const long long row = (long long)i * (1LL << 31) / T / 16 * 16 + by;
            if (row <= 1LL << 30) look(T, (int)row, share, features);
          }
      }
  std::printf("%lld cuts, %lld in phases, %lld wrong\n", seen, phased, bad);
  return bad != 0 || phased == 0;
}
"""


def test_what_a_cta_keeps_fits_its_shared_memory(tmp_path):
    src, exe = tmp_path / "cut.cpp", tmp_path / "cut"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error", "-I" + os.path.join(
        ROOT, "sparse_moe_ffn_route_gb300", "csrc"), str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
