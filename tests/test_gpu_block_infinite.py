"""Infinite weights of the dense block: the results are infinite or NaN where the formulas,
computed in 64 bits, make them so, and nowhere else."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")

pytestmark = pytest.mark.gpu

INF = float("inf")


def rnd(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()


def ffn(T, d, ff, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 31 * T + d + 7 * ff)
    return rnd(gen, T, d), moe.GluWeights(rnd(gen, ff, d, scale=d ** -0.5), rnd(gen, ff, d, scale=d ** -0.5),
                                          rnd(gen, d, ff, scale=ff ** -0.5))


def formula(x, w):
    x, g, u, d = (t.double() for t in (x, w.gate, w.up, w.down))

    def product(a, b):   # term by term, so that infinities meet what the formula says they meet
        return torch.stack([(row * b).sum(1) for row in a])

    g, u = product(x, g), product(x, u)
    return product(g * torch.sigmoid(g) * u, d)


def same_classes(got, want, name):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), (name, "NaN")
    assert torch.equal(torch.isinf(got), torch.isinf(want)), (name, "infinite")
    inf = torch.isinf(want)
    assert torch.equal(got[inf].sign(), want[inf].sign()), (name, "sign")


@pytest.mark.parametrize("back", [1, 3, 8])
@pytest.mark.parametrize("T,d,ff", [(1, 40, 64), (5, 72, 96), (8, 136, 32), (12, 104, 128), (16, 40, 64)])
def test_infinite_gate_and_up_at_the_end_of_a_row(T, d, ff, back):
    """d is no multiple of the 32 inputs that a step of the few-token kernel takes."""
    x, w = ffn(T, d, ff, back)
    x[:, d - back] = x[:, d - back].abs() + 0.5
    w.gate[3, d - back] = INF
    w.up[ff - 2, d - back] = -INF
    want = formula(x, w)
    assert torch.isinf(want).any()
    same_classes(moe.moe_glu_forward(moe.glu_cfg(d, ff), x, w), want, "y")


@pytest.mark.parametrize("back", [1, 8])
@pytest.mark.parametrize("T,d,ff", [(9, 64, 72), (16, 32, 40), (12, 96, 4104)])
def test_infinite_down_at_the_end_of_a_row(T, d, ff, back):
    x, w = ffn(T, d, ff, back)
    w.down[5, ff - back] = INF
    w.down[d - 1, ff - back] = -INF
    want = formula(x, w)
    assert torch.isinf(want[:, 5]).all() and torch.isfinite(want[:, 6:-1]).all()
    same_classes(moe.moe_glu_forward(moe.glu_cfg(d, ff), x, w), want, "y")

@pytest.mark.parametrize("T,d,ff,at", [(1, 64, 64, 7), (4, 96, 512, 300), (8, 64, 4096, 4000), (7, 32, 40, 39)])
def test_infinite_down_weight_meets_a_two_part_h(T, d, ff, at):
    """Few tokens, narrow FFN: h goes into the product as two bf16 numbers, of which the second
    one's sign, or a zero, must not decide what an infinite weight gives."""
    x, w = ffn(T, d, ff, at)
    w.down[5, at] = INF
    w.down[d - 1, at] = -INF
    w.down[9, at] = float("nan")
    want = formula(x, w)
    assert torch.isinf(want[:, 5]).all() and torch.isnan(want[:, 9]).all()
    same_classes(moe.moe_glu_forward(moe.glu_cfg(d, ff), x, w), want, "y")

@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,k,n,group", [(1, 32, 5, 32), (5, 96, 40, 32), (16, 224, 33, 32), (3, 64, 17, 64),
                                         (12, 192, 40, 64), (16, 8256, 20, 64)])
def test_infinite_last_group_scale(T, k, n, group, zeros):
    """n_in is no multiple of the 128 inputs that a step of the kernel takes.  The last group's
    codes lie above its zero and its inputs are positive, so every term is +inf."""
    gen = torch.Generator(device="cuda").manual_seed(T + k + n)
    x = rnd(gen, T, k)
    x[:, -group:] = x[:, -group:].abs() + 0.5
    codes = torch.randint(0, 256, (n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    codes[2, -group // 2:] = 0xCB
    scales = rnd(gen, n, k // group, scale=0.1)
    scales[2, -1] = INF
    z = torch.randint(0, 8, (n, k // group), generator=gen, device="cuda", dtype=torch.uint8) if zeros else None
    y = moe.moe_w4_linear(moe.w4_cfg(k, n, group), x, moe.W4Weights(codes, scales, z))
    assert (y[:, 2] == INF).all() and torch.isfinite(y[:, [i for i in range(n) if i != 2]]).all()
