"""A process whose first calls of the dense block come from several threads at once."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PROGRAM = r"""
import threading
import torch
import sparse_moe_ffn_route_gb300 as moe

N, T, D, FF = 8, 64, 256, 512
gen = torch.Generator(device="cuda").manual_seed(1)
rnd = lambda *s: (torch.randn(s, generator=gen, device="cuda") * s[-1] ** -0.5).bfloat16()
w = moe.GluWeights(rnd(FF, D), rnd(FF, D), rnd(D, FF))
x, dy = rnd(T, D), rnd(T, D)
cfg = moe.glu_cfg(D, FF)
streams = [torch.cuda.Stream() for _ in range(N)]
saved = [moe.glu_saved(cfg, T) for _ in range(N)]
torch.cuda.synchronize()
gate, out, failed = threading.Barrier(N), [None] * N, []

def work(i):
    try:
        with torch.cuda.stream(streams[i]):
            gate.wait()
            y = moe.moe_glu_forward(cfg, x, w, saved=saved[i])
            dx, g = moe.moe_glu_backward(cfg, x, w, saved[i], dy)
            out[i] = [y, dx, g.gate, g.up, g.down]
    except Exception as e:
        failed.append(repr(e))

threads = [threading.Thread(target=work, args=(i,)) for i in range(N)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not failed, failed
for o in out:
    assert all(torch.equal(a, b) for a, b in zip(o, out[0]))
y = moe.moe_glu_forward(cfg, x, w, saved=saved[0])
assert torch.equal(y, out[0][0])
print("ok")
"""


@pytest.mark.parametrize("attempt", range(4))
def test_first_calls_from_many_threads(attempt):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=200,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-3000:]
