"""The dense block's operators run together: the example's training steps and its 4-bit decode,
and one step's gradients against automatic differentiation of the whole stack in 64 bits."""
import importlib.util
import os

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
pytestmark = pytest.mark.gpu


def example():
    spec = importlib.util.spec_from_file_location("dense_block", os.path.join(ROOT, "examples", "dense_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_learns_and_serves():
    losses, full, small = example().main()
    assert losses[-1] < 0.95 * losses[0] and all(b < a + 1e-3 for a, b in zip(losses, losses[1:]))
    # 4-bit codes with group scales: a weight is off by at most half a code of about 15 across
    # its group's range (some 4 sigma), 1/12 of its size in the mean square; three layers of
    # three products each, halved by the branch scale, stay well under 0.3
    assert torch.isfinite(small).all() and (small - full).norm() < 0.3 * full.norm()


def test_stack_gradients_against_autograd():
    ex = example()
    st = ex.Stack(d=136, ff=264, layers=2, tokens=48, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(48, 136, generator=gen, device="cuda").bfloat16()
    da = torch.randn(48, 136, generator=gen, device="cuda").bfloat16()
    kept, a = st.forward(x)
    grads = st.backward(kept, da)
    leaves = [{k: v.double().requires_grad_() for k, v in w.items()} for w in st.w]

    def norm(v, w):
        return v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w

    y = x.double()
    b = norm(y, st.first.double())
    for w in leaves:
        g = b @ w["gate"].T
        z = (g * torch.sigmoid(g) * (b @ w["up"].T)) @ w["down"].T
        y = y + 0.5 * torch.sigmoid(w["logit"])[:, None] * norm(z, w["post"])
        b = norm(y, w["pre"])
    b.backward(da.double())
    # every tensor between the operators is rounded to bf16 (2^-9 in the root mean square at
    # most, some ten of them in turn on the way to and from the first layer): 2^-9 sqrt(20)
    assert (a.double() - b).norm() < 2.0 ** -9 * 20 ** 0.5 * b.norm()
    for got, want in zip(grads, leaves):
        for k, v in got.items():
            ref = want[k].grad
            assert (v.double() - ref).norm() < 2.0 ** -9 * 20 ** 0.5 * ref.norm(), k
