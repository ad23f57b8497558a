"""A sparse layer whose experts are linear layers of the library: trained in bf16, served in 8 bits.

    xs, rows = tokens sorted by expert (moe_dispatch_forward);  per expert e, on its rows:
    h = silu(xs W1_e^T + b1_e);  z = h W2_e^T + b2_e;  y = x + sum_j w_j z[rows_j]  (moe_combine_forward)

``train`` fits y to a target with plain gradient steps on fp32 copies of the experts' weights (the
routing is given).  ``serve`` runs the same layer in 8 bits: the norm writes the rows in e4m3, they
are dispatched as they are, and both products take e4m3 operands.

    python examples/sparse_layer.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sparse_moe_ffn_route_gb300 as moe  # noqa: E402


class Layer:
    def __init__(self, d=256, ff=384, experts=8, top_k=2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=gen, device="cuda") * scale

        self.d, self.ff, self.experts = d, ff, experts
        self.exchange = moe.exchange_cfg(d, experts, top_k)
        self.up, self.down = moe.linear_cfg(d, ff, act=moe.LINEAR_SILU), moe.linear_cfg(ff, d)
        # fp32 weights, which the steps change, and the bf16 ones that the kernels read
        self.master = {"w1": normal(experts, ff, d, scale=d ** -0.5), "b1": normal(experts, ff, scale=0.1),
                       "w2": normal(experts, d, ff, scale=ff ** -0.5), "b2": normal(experts, d, scale=0.1)}
        self.round()

    def round(self):
        self.w = {k: v.bfloat16() for k, v in self.master.items()}

    def forward(self, x, ids, weights):
        """y, and what backward needs.  The experts' shares are read back to cut the rows."""
        sent = moe.moe_dispatch_forward(self.exchange, x, ids)
        ends = sent.offsets.tolist()
        h, pre, z = (torch.empty(sent.xs.shape[0], n, dtype=torch.bfloat16, device=x.device) for n in (self.ff, self.ff, self.d))
        for e in range(self.experts):
            r = slice(ends[e], ends[e + 1])
            moe.moe_linear_forward(self.up, sent.xs[r], moe.LinearWeights(self.w["w1"][e], self.w["b1"][e]), pre=pre[r], y=h[r])
            moe.moe_linear_forward(self.down, h[r], moe.LinearWeights(self.w["w2"][e], self.w["b2"][e]), y=z[r])
        y = moe.moe_combine_forward(self.exchange, z, sent.rows, w=weights, residual=x)
        return y, (sent, ends, h, pre, z)

    def backward(self, kept, weights, dy):
        """Gradients of the experts' weights (bf16), of x (without the residual's, which is dy) and
        of the routing weights."""
        sent, ends, h, pre, z = kept
        dz, dweights = moe.moe_combine_backward(self.exchange, dy, z, sent.rows, weights)
        g = {k: torch.empty_like(v) for k, v in self.w.items()}
        dxs = torch.empty_like(sent.xs)
        for e in range(self.experts):
            r = slice(ends[e], ends[e + 1])
            dh, _ = moe.moe_linear_backward(self.down, h[r], moe.LinearWeights(self.w["w2"][e], self.w["b2"][e]), dz[r],
                                            grads=moe.LinearGrads(g["w2"][e], g["b2"][e]))
            moe.moe_linear_backward(self.up, sent.xs[r], moe.LinearWeights(self.w["w1"][e], self.w["b1"][e]), dh, pre=pre[r],
                                    dx=dxs[r], grads=moe.LinearGrads(g["w1"][e], g["b1"][e]))
        return g, moe.moe_dispatch_backward(self.exchange, dxs, sent.rows), dweights


def train(layer, x, ids, weights, target, steps=20, rate=20.0):
    """Loss of every step."""
    losses = []
    for _ in range(steps):
        y, kept = layer.forward(x, ids, weights)
        off = y.float() - target
        losses.append(off.square().mean().item())
        g, _, _ = layer.backward(kept, weights, (2.0 / off.numel() * off).bfloat16())
        for k in layer.master:
            layer.master[k] -= rate * g[k].float()
        layer.round()
    return losses


def serve(layer, x, norm_w, ids, weights):
    """y = x + the layer of norm(x), rows, weights and both products' operands in e4m3."""
    up = moe.linear_cfg(layer.d, layer.ff, act=moe.LINEAR_SILU, fmt=moe.LINEAR_E4M3)
    down = moe.linear_cfg(layer.ff, layer.d, fmt=moe.LINEAR_E4M3)
    packed = []
    for e in range(layer.experts):
        (w1, s1), (w2, s2) = moe.w8_quantize(layer.w["w1"][e]), moe.w8_quantize(layer.w["w2"][e])
        packed.append((moe.LinearWeights(w1, layer.w["b1"][e], s1), moe.LinearWeights(w2, layer.w["b2"][e], s2)))
    _, q, scale = moe.moe_block_norm_quant(moe.norm_cfg(layer.d), x, pre_w=norm_w)
    cfg = moe.exchange_cfg(layer.d, layer.experts, ids.shape[1], fmt=moe.ROWS_E4M3)
    sent = moe.moe_dispatch_forward(cfg, q, ids, x_scale=scale)
    ends = sent.offsets.tolist()
    z = torch.empty(sent.xs.shape[0], layer.d, dtype=torch.bfloat16, device=x.device)
    for e in range(layer.experts):
        r = slice(ends[e], ends[e + 1])
        h = moe.moe_linear_forward(up, sent.xs[r], packed[e][0], x_scale=sent.xs_scale[r])
        _, hq, hs = moe.moe_block_norm_quant(moe.norm_cfg(layer.ff), h)
        moe.moe_linear_forward(down, hq, packed[e][1], x_scale=hs, y=z[r])
    return moe.moe_combine_forward(layer.exchange, z, sent.rows, w=weights, residual=x)


def routing(layer, tokens, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    top = torch.randn(tokens, layer.experts, generator=gen, device="cuda").topk(layer.exchange.top_k, 1)
    return top.indices.int(), torch.softmax(top.values, 1)


def main():
    layer = Layer()
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(512, layer.d, generator=gen, device="cuda").bfloat16()
    target = torch.randn(512, layer.d, generator=gen, device="cuda")
    ids, weights = routing(layer, 512)
    losses = train(layer, x, ids, weights, target)
    print("loss", " ".join(f"{v:.4f}" for v in losses[::4] + losses[-1:]))
    ones = torch.ones(layer.d, dtype=torch.bfloat16, device="cuda")
    normed = moe.moe_block_norm_forward(moe.norm_cfg(layer.d), x, pre_w=ones)[1]
    full = (layer.forward(normed, ids, weights)[0] - normed).float()
    small = (serve(layer, x, ones, ids, weights) - x).float()
    print(f"8 bits: {((small - full).norm() / full.norm()).item():.3f} of the bf16 layer's norm off")
    return losses, full, small


if __name__ == "__main__":
    main()
