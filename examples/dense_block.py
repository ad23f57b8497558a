"""A stack of dense blocks, trained and then served in 4 bits, on the library's block operators.

    a_0 = norm(y_0);  z_l = FFN_l(a_l);  y_{l+1} = y_l + 0.5 sigmoid(gate_l) norm(z_l),  a_{l+1} = norm(y_{l+1})

``train`` fits a_L to a target: forward and backward passes of the gated FFN
(moe_glu_forward, moe_glu_backward) and of the fused norm, gate and residual between the
blocks (moe_block_norm_forward, moe_block_norm_backward), with plain gradient steps on fp32
copies of the weights.  ``serve`` rounds the trained weights to 4-bit codes and runs a few
tokens through moe_w4_linear and the same norms, captured once as a CUDA graph.

    python examples/dense_block.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sparse_moe_ffn_route_gb300 as moe  # noqa: E402


class Stack:
    def __init__(self, d=512, ff=1024, layers=3, tokens=256, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=gen, device="cuda") * scale

        self.d, self.ff, self.tokens = d, ff, tokens
        self.ffn = moe.glu_cfg(d, ff)
        self.norm = moe.norm_cfg(d, residual_scale=1.0, branch_scale=0.5)
        # fp32 weights, which the steps change, and the bf16 ones that the kernels read
        self.master = [{"gate": normal(ff, d, scale=d ** -0.5), "up": normal(ff, d, scale=d ** -0.5),
                        "down": normal(d, ff, scale=ff ** -0.5), "post": torch.ones(d, device="cuda"),
                        "pre": torch.ones(d, device="cuda"), "logit": torch.zeros(tokens, device="cuda")}
                       for _ in range(layers)]
        self.first = torch.ones(d, dtype=torch.bfloat16, device="cuda")   # norm of the input
        self.ws = moe.glu_workspace(self.ffn, tokens)
        self.saved = [moe.glu_saved(self.ffn, tokens) for _ in range(layers)]
        self.round()

    def round(self):
        self.w = [{k: v if k == "logit" else v.bfloat16() for k, v in m.items()} for m in self.master]

    def weights(self, layer):
        return moe.GluWeights(layer["gate"], layer["up"], layer["down"])

    def forward(self, x):
        """Per layer its inputs (y, a) and its branch z; and the last a."""
        kept, y = [], x
        _, a = moe.moe_block_norm_forward(self.norm, x, pre_w=self.first)
        for w, saved in zip(self.w, self.saved):
            z = moe.moe_glu_forward(self.ffn, a, self.weights(w), saved=saved, ws=self.ws)
            kept.append((y, a, z))
            y, a = moe.moe_block_norm_forward(self.norm, y, branch=z, post_w=w["post"], gate=w["logit"],
                                              pre_w=w["pre"])
        return kept, a

    def backward(self, kept, da):
        grads, dy = [], None
        for w, saved, (y, a, z) in zip(reversed(self.w), reversed(self.saved), reversed(kept)):
            n = moe.moe_block_norm_backward(self.norm, y, dy=dy, da=da, branch=z, post_w=w["post"], gate=w["logit"],
                                            pre_w=w["pre"])
            dy = n.dx
            da, g = moe.moe_glu_backward(self.ffn, a, self.weights(w), saved, n.dbranch, ws=self.ws)
            grads.append({"gate": g.gate, "up": g.up, "down": g.down, "post": n.dpost_w, "pre": n.dpre_w,
                          "logit": n.dgate})
        return grads[::-1]


def train(stack: Stack, x, target, steps=20, rate=2.0):
    """Loss of every step."""
    losses = []
    for _ in range(steps):
        kept, a = stack.forward(x)
        off = a.float() - target
        losses.append(off.square().mean().item())
        grads = stack.backward(kept, (2.0 / off.numel() * off).bfloat16())
        for m, g in zip(stack.master, grads):
            for k in m:
                m[k] -= rate * g[k].float()
        stack.round()
    return losses


def serve(stack: Stack, x, group=64):
    """a of a few tokens with the weights in 4 bits: one captured graph per step."""
    T = x.shape[0]
    up_cfg = moe.w4_cfg(stack.d, stack.ff, group, glu=True)
    down_cfg = moe.w4_cfg(stack.ff, stack.d, group)
    packed = [(moe.w4_quantize(torch.cat((m["gate"], m["up"])), group), moe.w4_quantize(m["down"], group))
              for m in stack.master]

    def step():
        y, (_, a) = x, moe.moe_block_norm_forward(stack.norm, x, pre_w=stack.first)
        for w, (up, down) in zip(stack.w, packed):
            z = moe.moe_w4_linear(down_cfg, moe.moe_w4_linear(up_cfg, a, up), down)
            y, a = moe.moe_block_norm_forward(stack.norm, y, branch=z, post_w=w["post"], gate=w["logit"][:T],
                                              pre_w=w["pre"])
        return a

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = step()
    graph.replay()
    torch.cuda.synchronize()
    return a


def main():
    stack = Stack()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(stack.tokens, stack.d, generator=gen, device="cuda").bfloat16()
    target = torch.randn(stack.tokens, stack.d, generator=gen, device="cuda")
    losses = train(stack, x, target)
    print("loss", " ".join(f"{v:.4f}" for v in losses[::4] + losses[-1:]))
    full = stack.forward(x)[1][:4].float()
    small = serve(stack, x[:4]).float()
    print(f"4-bit weights: {((small - full).norm() / full.norm()).item():.3f} of the bf16 output's norm off")
    return losses, full, small


if __name__ == "__main__":
    main()
