"""Activations and their slopes far from zero, where powers of v leave fp32's range: their limits."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_gpu_block import H, R, close  # noqa: E402
from test_gpu_linear import ACTS, lin64, slope64  # noqa: E402

pytestmark = pytest.mark.gpu


def far():
    """+-17 to +-3e38, in bf16."""
    v = torch.tensor([17.0, 60.0, 100.0, 1e3, 1e6, 1e9, 1e12, 1e13, 2e13, 1e15, 1.5e19, 3e19, 1e25, 1e30, 1e37, 2e37, 2e38, 3e38])
    return torch.cat((v, -v)).cuda().bfloat16()


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes(act):
    """pre is the caller's; W = 1, so that dx is dv, rounded once to bf16 (H), off by R of itself and of dy
    before (as in test_backward)."""
    v = far()
    T = v.numel()
    pre, one = v[:, None].expand(-1, 8).contiguous(), torch.ones(T, 8, dtype=torch.bfloat16, device="cuda")
    w = moe.LinearWeights(torch.eye(8, device="cuda").bfloat16(), torch.zeros(8, dtype=torch.bfloat16, device="cuda"))
    dx, g = moe.moe_linear_backward(moe.linear_cfg(8, 8, act=act), one, w, one, pre=pre)
    want = slope64(pre.double(), act)
    assert torch.isfinite(want).all()
    close(dx, want, H * want.abs() + 1.01 * R * (want.abs() + 1.0), "dx")
    total = want.sum(0)
    close(g.bias, total, H * total.abs() + 1.01 * R * (want.abs() + 1.0).sum(0), "dbias")
    # what is not finite stays so
    for bad in (float("nan"), float("inf")):
        pre[3, 2] = bad
        dx, _ = moe.moe_linear_backward(moe.linear_cfg(8, 8, act=act), one, w, one, pre=pre)
        assert torch.isnan(dx[3]).all() and not torch.isnan(dx[[0, 1, 2, 4]]).any()


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("act", ACTS[1:])
def test_values(act, T):
    """x = 0, so that v is the bias exactly; y is off by R of itself and rounded once.  A logistic function
    below 2^-126 may become 0 (1 / (1 + e^-v) is then not a normal number): that is so for v below
    -126 ln 2 = -87.33 alone, and |v| e^v falls from there on, so that y loses 87.4 2^-126 at most."""
    b = torch.cat((far(), torch.zeros(4, device="cuda").bfloat16()))
    x, w = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(b.numel(), 8, dtype=torch.bfloat16, device="cuda")
    y = moe.moe_linear_forward(moe.linear_cfg(8, b.numel(), act=act), x, moe.LinearWeights(w, b))
    want = lin64(b.double(), act)[None].expand(T, -1)
    close(y, want, (H + 1.01 * R) * want.abs() + 87.4 * 2.0 ** -126, "y")
