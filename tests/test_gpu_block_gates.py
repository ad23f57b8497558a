"""The gate's gradient over the gate's whole range: sigmoid(v) sigmoid(-v) is small at both
ends, and keeps its relative accuracy there."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")

pytestmark = pytest.mark.gpu

F, R = 2.0 ** -23, 2.0 ** -18
GATES = [0.0, 0.25, -0.25, 3.0, -3.0, 8.0, -8.0, 12.0, -12.0, 16.0, -16.0, 17.5, -17.5, 20.0, -20.0, 35.0, -35.0,
         60.0, -60.0, 80.0, -80.0]


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("d", [8, 64, 520, 4104])
def test_gate_gradient_of_far_gates(d, post):
    """dgate = branch_scale s (1 - s) sum dy p, from dy alone.  The sum is off by d 2^-23 of its
    terms' magnitudes, p (its norm) by R, the gate's factor by R: relative to the factor itself,
    however small it is."""
    gen = torch.Generator(device="cuda").manual_seed(d + post)
    T = len(GATES)
    x = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    z = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    dy = (torch.randn(T, d, generator=gen, device="cuda").abs() * z.float().sign()).bfloat16()   # no cancelling sum
    w = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).bfloat16() if post else None
    gate = torch.tensor(GATES, device="cuda")
    bs = -0.7
    g = moe.moe_block_norm_backward(moe.norm_cfg(d, eps=1e-6, branch_scale=bs), x, dy=dy, branch=z, post_w=w, gate=gate)
    p = z.double()
    if post:
        p = p * (p.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.double()
    k = bs * torch.sigmoid(gate.double()) * torch.sigmoid(-gate.double())
    terms = dy.double() * p
    want = k * terms.sum(1)
    tol = 1.01 * k.abs() * (d * F + 2 * R) * terms.abs().sum(1)
    bad = ~((g.dgate.double() - want).abs() <= tol)
    assert not bad.any(), [(GATES[i], float(g.dgate[i]), float(want[i])) for i in bad.nonzero().flatten().tolist()]


def test_gate_gradient_of_infinite_gates():
    d = 64
    x = torch.ones(3, d, device="cuda").bfloat16()
    gate = torch.tensor([float("inf"), float("-inf"), float("nan")], device="cuda")
    g = moe.moe_block_norm_backward(moe.norm_cfg(d), x, dy=x, branch=x, gate=gate)
    assert (g.dgate[:2] == 0).all() and torch.isnan(g.dgate[2])
    assert torch.equal(g.dbranch[0], x[0]) and (g.dbranch[1] == 0).all() and torch.isnan(g.dbranch[2]).all()
