"""The linear layer where its tiles are many: pairs of CTAs, widths that are no multiple of 32, several tiles
to a CTA; sums that are split or come in phases; and long rows.

Sums of whole numbers are exact in fp32 below 2^24, in whatever order and parts they are added up, and
so are products with scales that are powers of two: without an activation every output has to be the
exact value rounded once to bf16, bit for bit."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_gpu_block import ALPHA, H, LIMIT, Guarded, close, gen_for  # noqa: E402
from test_gpu_linear import inputs, sums64, y64  # noqa: E402

pytestmark = pytest.mark.gpu

# pairs and single CTAs, 144 to 256 columns, 2 to 6 tiles to a unit; rows of 6 KB and of 16 bytes
MANY = [(3000, 2048, 2048), (4096, 2048, 2048), (3000, 1024, 4000), (4000, 1024, 2000), (3000, 3008, 3000), (1001, 2880, 5120),
        (2000, 1040, 8200), (5000, 640, 904), (9000, 256, 2600), (20000, 16, 200), (1100, 4096, 2200)]
# few tokens with long rows (x in phases up to 8 tokens), split sums, one row of tiles
LONG = [(1, 262144, 24), (3, 98320, 40), (5, 50000, 1000), (8, 40000, 72), (8, 20000, 2600), (16, 20000, 264), (40, 30000, 256),
        (128, 16384, 512), (130, 20000, 72), (777, 8208, 640)]


def whole(gen, *shape, most=3):
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").bfloat16()


def powers(gen, n):
    return torch.exp2(torch.randint(-3, 4, (n,), generator=gen, device="cuda").float())


@pytest.mark.parametrize("fmt", [moe.LINEAR_BF16, moe.LINEAR_E4M3])
@pytest.mark.parametrize("T,k,n", MANY + LONG)
def test_forward_to_the_bit(T, k, n, fmt):
    gen = gen_for(T, k, n, fmt)
    x, w, b, r = whole(gen, T, k), whole(gen, n, k), whole(gen, n, most=40), whole(gen, T, n, most=100)
    v = x.float().double() @ w.double().T
    assert v.abs().max() < 2 ** 18            # with scales, bias and residual: below 2^24 of their least step
    xs = ws = None
    if fmt == moe.LINEAR_E4M3:
        xs, ws = powers(gen, T), powers(gen, n)
        v = v * xs.double()[:, None] * ws.double()
        x, w = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
    v = v + b.double()
    cfg = moe.linear_cfg(k, n, fmt=fmt)
    y, pre, room = Guarded((T, n)), Guarded((T, n)), moe.linear_workspace(cfg, T)
    moe.moe_linear_forward(cfg, x, moe.LinearWeights(w, b, ws), x_scale=xs, residual=r, pre=pre.t, y=y.t, ws=room)
    assert moe.moe_device_status(room)[0] == moe.MOE_OK
    exact = v.float().double() == v           # all but sums of wide scales that pass 24 bits
    assert exact.float().mean() > 0.99
    assert torch.equal(pre.t[exact], v.bfloat16()[exact])
    v = v + r.double()
    exact &= v.float().double() == v
    assert torch.equal(y.t[exact], v.bfloat16()[exact])
    y.check()
    pre.check()
    # in the residual's place, without pre
    moe.moe_linear_forward(cfg, x, moe.LinearWeights(w, b, ws), x_scale=xs, residual=r, y=r)
    assert torch.equal(r, y.t)


@pytest.mark.parametrize("fmt", [moe.LINEAR_BF16, moe.LINEAR_E4M3])
@pytest.mark.parametrize("T,k,n", [(3000, 1024, 4000), (4000, 1024, 2000), (1001, 2880, 5120), (2500, 4096, 1608), (5000, 640, 904)])
@pytest.mark.parametrize("form", ["silu", "gelu", "swiglu", "clamped"])
def test_activations(T, k, n, fmt, form):
    glu = form in ("swiglu", "clamped")
    act = {"silu": moe.LINEAR_SILU, "gelu": moe.LINEAR_GELU, "swiglu": moe.ACT_SWIGLU, "clamped": moe.ACT_CLAMPED_GLU}[form]
    x, xs, w, r, _ = inputs(T, k, n, fmt, glu, seed=act)
    cfg = moe.linear_cfg(k, n, act=act, glu=glu, fmt=fmt, glu_limit=LIMIT, glu_alpha=ALPHA)
    y, pre = Guarded((T, n)), None if glu else Guarded((T, n))
    moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r, pre=None if glu else pre.t, y=y.t)
    v, e = sums64(x, w.w, xs, w.scale, w.bias)
    if pre is not None:
        close(pre.t, v, H * v.abs() + 1.01 * e, "pre")
        pre.check()
    close(y.t, *y64(v, e, dict(glu=glu, act=act), r), "y")
    y.check()


@pytest.mark.parametrize("T,k,n", [(3000, 2048, 2048), (777, 640, 2880), (2500, 4096, 1608), (8192, 256, 512), (16384, 512, 264), (60, 8200, 4000),
                                   (20000, 16, 200)])
def test_backward_to_the_bit(T, k, n):
    gen = gen_for(T, k, n)
    x, w, dy = whole(gen, T, k), whole(gen, n, k), whole(gen, T, n)
    dx, dw, db = Guarded((T, k)), Guarded((n, k)), Guarded((n,))
    moe.moe_linear_backward(moe.linear_cfg(k, n), x, moe.LinearWeights(w, dy[0].clone()), dy, dx=dx.t, grads=moe.LinearGrads(dw.t, db.t))
    X, W, g = x.double(), w.double(), dy.double()
    for got, want, name in ((dx, g @ W, "dx"), (dw, g.T @ X, "dw"), (db, g.sum(0), "dbias")):
        assert want.abs().max() < 2 ** 24
        assert torch.equal(got.t, want.bfloat16()), name
        got.check()


# the weights' gradient cut over the tokens: its counts are cleared by a memset of its own where no launch
# comes before the products; dx in a launch of its own; one launch for all
@pytest.mark.parametrize("T,k,n", [(8192, 256, 512), (60, 8200, 4000), (3000, 2048, 2048)])
def test_backward_captured(T, k, n):
    gen = gen_for(T, n, 3)
    x, w, dy = whole(gen, T, k), moe.LinearWeights(whole(gen, n, k)), whole(gen, T, n)
    cfg = moe.linear_cfg(k, n)

    def step():
        dx, g = moe.moe_linear_backward(cfg, x, w, dy)
        _, only = moe.moe_linear_backward(cfg, x, w, dy, need_dx=False)
        return dx, g.w, only.w

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        x.copy_(whole(gen, T, k))
        dy.copy_(whole(gen, T, n))
        graph.replay()
        dx, dw = dy.double() @ w.w.double(), dy.double().T @ x.double()
        assert torch.equal(out[0], dx.bfloat16()) and torch.equal(out[1], dw.bfloat16()) and torch.equal(out[2], dw.bfloat16())
