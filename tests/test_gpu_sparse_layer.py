"""The exchange, the 8-bit norm and the linear layer run together, as the example uses them: a sparse
layer's training step against automatic differentiation in 64 bits, and its 8-bit form; and their
calls on streams other than the current one."""
import importlib.util
import os

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
pytestmark = pytest.mark.gpu


def example():
    spec = importlib.util.spec_from_file_location("sparse_layer", os.path.join(ROOT, "examples", "sparse_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_runs():
    losses, full, small = example().main()
    assert all(v == v for v in losses) and torch.isfinite(small).all() and torch.isfinite(full).all()


def reference(layer, x, ids, weights, leaves):
    """The layer in 64 bits, expert by expert."""
    y = x.clone()
    for e in range(layer.experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        h = torch.nn.functional.silu(x[t] @ leaves["w1"][e].T + leaves["b1"][e])
        y = y.index_add(0, t, weights[t, j][:, None] * (h @ leaves["w2"][e].T + leaves["b2"][e]))
    return y


@pytest.mark.parametrize("tokens,d,ff,experts,top_k", [(300, 136, 264, 8, 2), (5, 64, 72, 16, 4), (700, 64, 128, 3, 3)])
def test_training_step_against_autograd(tokens, d, ff, experts, top_k):
    ex = example()
    layer = ex.Layer(d, ff, experts, top_k, seed=tokens)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(tokens, d, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(tokens, d, generator=gen, device="cuda").bfloat16()
    ids, weights = ex.routing(layer, tokens)
    y, kept = layer.forward(x, ids, weights)
    g, dx, dweights = layer.backward(kept, weights, dy)
    leaves = {k: v.double().requires_grad_() for k, v in layer.w.items()}
    x64, w64 = x.double().requires_grad_(), weights.double().requires_grad_()
    want = reference(layer, x64, ids, w64, leaves)
    want.backward(dy.double())
    # every tensor on the way is rounded to bf16, 2^-9 of it in the root mean square at most: seven
    # of them (h, z, y; dz, dh, dv, dxs) and the kept pre, whose rounding acts through silu'' <
    # 1, lie before any one result
    bound = 2.0 ** -9 * 10 ** 0.5
    off = lambda a, b: (a.double() - b).norm() / b.norm()  # noqa: E731
    assert off(y, want.detach()) < bound
    assert off(dx, x64.grad - dy.double()) < bound
    assert off(dweights, w64.grad) < bound
    for k in leaves:
        assert off(g[k], leaves[k].grad) < bound, k


def test_eight_bits_against_the_formula():
    """Values in e4m3 with a scale per row are off by 2^-4 of themselves at most, 2^-5 in the mean
    square; four such tensors (rows, h, both weights) stand before z, each product averages the
    errors of its terms: 2^-5 sqrt(4), and silu' is below 1.1."""
    ex = example()
    layer = ex.Layer(256, 384, 8, 2, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(400, 256, generator=gen, device="cuda").bfloat16()
    norm_w = (1 + 0.2 * torch.randn(256, generator=gen, device="cuda")).bfloat16()
    ids, weights = ex.routing(layer, 400)
    got = (ex.serve(layer, x, norm_w, ids, weights) - x).double()
    v = x.double()
    v = v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * norm_w.double()
    want = reference(layer, v, ids, weights.double(), {k: t.double() for k, t in layer.w.items()}) - v
    # (got was rounded to bf16 on the residual, of size 1: 2^-9 beside a layer of size about 0.6)
    assert (got - want).norm() < 1.1 * (2.0 ** -5 * 2 + 2.0 ** -8) * want.norm()


def flat(out):
    if out is None:
        return []
    if torch.is_tensor(out):
        return [out]
    return [t for o in (out if isinstance(out, (tuple, list)) else vars(out).values()) for t in flat(o)]


@pytest.mark.parametrize("T", [4, 300, 5000])
def test_buffers_of_a_call_on_a_given_stream(T):
    """What a call allocates belongs to its stream until that is done, whatever the caller allocates
    meanwhile."""
    d, n, E, k = 256, 512, 16, 4
    gen = torch.Generator(device="cuda").manual_seed(T)

    def rnd(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    x, dy, w = rnd(T, d), rnd(T, n), moe.LinearWeights(rnd(n, d), rnd(n))
    ids = torch.rand(T, E, generator=gen, device="cuda").topk(k, 1).indices.int()
    weights = torch.rand(T, k, generator=gen, device="cuda")
    ex, lin, norm = moe.exchange_cfg(d, E, k), moe.linear_cfg(d, n, act=moe.LINEAR_GELU), moe.norm_cfg(d)
    pre = moe.linear_pre(lin, T)
    moe.moe_linear_forward(lin, x, w, pre=pre)
    sent = moe.moe_dispatch_forward(ex, x, ids)
    pre_w = rnd(d)
    calls = {"dispatch": lambda s: moe.moe_dispatch_forward(ex, x, ids, stream=s),
             "dispatch backward": lambda s: moe.moe_dispatch_backward(ex, sent.xs, sent.rows, stream=s),
             "combine": lambda s: moe.moe_combine_forward(ex, sent.xs, sent.rows, weights, x, stream=s),
             "combine backward": lambda s: moe.moe_combine_backward(ex, x, sent.xs, sent.rows, weights, stream=s),
             "norm": lambda s: moe.moe_block_norm_quant(norm, x, pre_w=pre_w, stream=s),
             "linear": lambda s: moe.moe_linear_forward(lin, x, w, stream=s),
             "linear backward": lambda s: moe.moe_linear_backward(lin, x, w, dy, pre=pre, stream=s)}
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    sizes = {moe.moe_linear_workspace_bytes(lin, T), moe.moe_dispatch_workspace_bytes(ex, T), 2 * T * d, 2 * T * n, 2 * T * k * d,
             4 * T * k, T * d, 4 * T, 2 * d * n, 4 * (E + 1)}
    for name, call in calls.items():
        want = [t.clone() for t in flat(call(None))]
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):     # some milliseconds of ordinary work before the call's
            hold = big
            for _ in range(40):
                hold = (hold @ big).clamp_(-1, 1)
        got = call(side)
        junk = [torch.full((m,), 0x55, dtype=torch.uint8, device="cuda") for m in sizes for _ in range(4)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(flat(got), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
        assert all((j == 0x55).all() for j in junk), name
