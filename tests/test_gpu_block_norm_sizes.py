"""Rows for which the backward norm's groups of threads are 288 to 512 wide, and their edges."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_gpu_block import EPS, PARTS, close, norm64, norm_inputs, rnd  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["all", "post", "pre"])
@pytest.mark.parametrize("T,d", [(1, 4608), (155, 5128), (9, 6152), (310, 7680), (1, 8192), (153, 8192), (4, 8200)])
def test_block_norm_wide_rows(T, d, which):
    parts = PARTS[which]
    i, gen = norm_inputs(T, d, parts, seed=3)
    cfg = moe.norm_cfg(d, eps=EPS, residual_scale=0.9, branch_scale=-0.7)
    dy = rnd(gen, T, d) if parts[0] else None
    da = rnd(gen, T, d) if parts[3] else None
    want = norm64(i["x"], i["branch"], i["post_w"], i["gate"], i["pre_w"], dy, da, 0.9, -0.7)
    y, a = moe.moe_block_norm_forward(cfg, **i)
    g = moe.moe_block_norm_backward(cfg, i["x"], dy=dy, da=da, **{k: v for k, v in i.items() if k != "x"})
    got = {"y": y, "a": a, "dx": g.dx, "dbranch": g.dbranch, "dgate": g.dgate, "dpost_w": g.dpost_w, "dpre_w": g.dpre_w}
    assert {k for k, v in got.items() if v is not None} == set(want)
    for name, (v, tol) in want.items():
        close(got[name], v, tol, name)
