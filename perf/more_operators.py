"""The measured cases of three groups of operators around the sparse layer: tokens sorted by expert
and back with their weights (forward and backward), the block's norm with an output in 8 bits, and
the linear layer with bias, activation and residual in its epilogue (bf16 forward and training
step, 8-bit operands forward).

`run` computes them in plain torch operations in 32 bits, or, where `own` is set, through the
library's entry points.  `exact` is their definition in 64 bits, with the gradients from automatic
differentiation."""
import math

import torch

own = False

NONE, SILU, GELU, GELU_TANH = 0, 1, 2, 3     # activations of the linear layer
SWIGLU, CLAMPED = 0, 1                       # and of its gated form
LIMIT, ALPHA, EPS = 7.0, 1.702, 1e-6
RESIDUAL, BRANCH = 0.9, 0.7
E4M3_MAX, LEAST_SCALE = 448.0, 2.0 ** -126


def listed():
    return [
        # a decode step's few tokens to the rows of their experts: latency
        {"name": "dispatch batch 8 2048", "op": "dispatch", "T": 8, "d": 2048, "E": 256, "k": 8, "bits": 16},
        # a prefill batch whose rows the norm has left in 8 bits
        {"name": "dispatch 8-bit 8192 2880", "op": "dispatch", "T": 8192, "d": 2880, "E": 32, "k": 4, "bits": 8},
        # the experts' rows of a decode batch back to their tokens, onto the residual stream
        {"name": "combine batch 32 2880", "op": "combine", "T": 32, "d": 2880, "E": 32, "k": 4},
        # training: out, back, and both gradients, for a full batch and for a ragged one
        {"name": "exchange train 4096 2048", "op": "exchange", "T": 4096, "d": 2048, "E": 256, "k": 8},
        {"name": "exchange train 1001 2880", "op": "exchange", "T": 1001, "d": 2880, "E": 32, "k": 4},
        # between two blocks, decoding and over a prefill batch, for a layer that takes 8 bits
        {"name": "norm 8-bit batch 8 2048", "op": "norm8", "T": 8, "d": 2048},
        {"name": "norm 8-bit 8192 2880", "op": "norm8", "T": 8192, "d": 2880},
        # a projection of one token: the stream of its weights
        {"name": "linear token 2048x4096", "op": "linear", "T": 1, "k": 2048, "n": 4096, "act": NONE,
         "residual": True},
        # a ragged piece of a prompt with an activation, sizes that are no power of two
        {"name": "linear prompt 777 2880x5120", "op": "linear", "T": 777, "k": 2880, "n": 5120, "act": GELU,
         "residual": False},
        # a training step of a square layer
        {"name": "linear train 4096 2048x2048", "op": "train", "T": 4096, "k": 2048, "n": 2048, "act": SILU,
         "residual": True},
        # gated layers of 8-bit operands: a decode batch, and a full prefill batch (the largest case)
        {"name": "linear 8-bit 16 4096x12288 glu", "op": "linear8", "T": 16, "k": 4096, "n": 12288, "glu": True,
         "act": SWIGLU},
        {"name": "linear 8-bit 8192 2880x8192 glu", "op": "linear8", "T": 8192, "k": 2880, "n": 8192, "glu": True,
         "act": CLAMPED},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "exchange", "exchange", "norm8", "linear", "linear", "train", "linear8",
                     "linear8"])
    if op in ("dispatch", "combine", "exchange"):
        E = _log(rng, 4, 512)
        k = rng.randint(1, min(E, 8))
        d = _log(rng, 256, 8192, 16)
        c = {"op": op, "T": min(_log(rng, 1, 16384), 8192 * 8 * 2048 // (d * k)), "d": d, "E": E, "k": k}
        if op == "dispatch":
            c["bits"] = rng.choice([8, 16])
        return c
    if op == "norm8":
        return {"op": op, "T": _log(rng, 1, 16384), "d": _log(rng, 256, 8192, 8)}
    k, n = _log(rng, 256, 8192, 16 if op == "linear8" else 8), _log(rng, 256, 8192, 8)
    glu = op == "linear8" and rng.random() < 0.5
    most = 8192 * 2880 * 8192 // (k * n) // (3 if op == "train" else 1)
    c = {"op": op, "T": min(_log(rng, 16 if op == "train" else 1, 8192), most), "k": k, "n": n}
    if op == "linear8":
        return {**c, "glu": glu, "act": rng.choice([SWIGLU, CLAMPED] if glu else [NONE, SILU, GELU, GELU_TANH])}
    return {**c, "act": rng.choice([NONE, SILU, GELU, GELU_TANH]), "residual": rng.random() < 0.5}


def work(case):
    op, T = case["op"], case["T"]
    if op in ("dispatch", "combine", "exchange"):
        d, k = case["d"], case["k"]
        S = T * k
        routing = 4 * S + 4 * (case["E"] + 1)      # ids in, or rows; offsets
        if op == "dispatch":                       # ids, x -> rows, offsets, xs (8 bits: and the scales)
            per = 2 * d if case["bits"] == 16 else d + 4
            return {"bytes": (T + S) * per + 4 * S + routing, "flops": 0}
        if op == "combine":                        # z, rows, w, residual -> y
            return {"bytes": 2 * d * (S + 2 * T) + 8 * S, "flops": 2 * S * d}
        # out: x -> xs; back: z -> y; gradients: dy, z -> dz, dw and dxs -> dx, each tensor once
        return {"bytes": 2 * d * (4 * S + 4 * T) + 4 * S * 4 + routing, "flops": 6 * S * d}
    if op == "norm8":
        # x, branch -> y, q; the gates, the scales and both weights
        return {"bytes": 7 * T * case["d"] + 8 * T + 4 * case["d"], "flops": 14 * T * case["d"]}
    k, n = case["k"], case["n"]
    if op == "linear8":
        rows = n * (2 if case["glu"] else 1)
        return {"bytes": T * k + rows * k + 2 * T * n + 4 * (T + rows) + 2 * rows, "flops": 2 * T * rows * k}
    nbytes = 2 * (T * k + n * k + n + T * n * (2 if case["residual"] else 1))
    if op == "linear":
        return {"bytes": nbytes, "flops": 2 * T * n * k}
    # training: also dy in, dx and the gradients of the weights and the bias out
    return {"bytes": nbytes + 2 * (T * n + T * k + n * k + n), "flops": 6 * T * n * k}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    def bf16(t):
        return t.to(torch.bfloat16)

    def eight(t):
        """t in e4m3 with a scale per row, as the weights of a checkpoint or the norm leave it."""
        scale = (t.abs().amax(1) / E4M3_MAX).clamp(min=LEAST_SCALE)
        return (t / scale[:, None]).to(torch.float8_e4m3fn), scale

    s = {"case": dict(case)}
    op, T = case["op"], case["T"]
    if op in ("dispatch", "combine", "exchange"):
        d, E, k = case["d"], case["E"], case["k"]
        # routing as a router leaves it: some experts more popular than others
        logits = normal(T, E) + normal(E, scale=0.5)
        top = logits.topk(k, dim=1)
        s["ids"] = top.indices.to(torch.int32)
        if op != "dispatch":
            s["w"] = torch.softmax(top.values, 1)
            s["residual"] = bf16(normal(T, d, scale=4.0))
            s["z"] = bf16(normal(T * k, d))                     # the experts' outputs
        if op == "combine":
            s["rows"] = _sort(s["ids"], E)[1]                   # the dispatch has left them
        elif op == "dispatch" and case["bits"] == 8:
            s["x"], s["x_scale"] = eight(normal(T, d) * torch.exp(normal(T, 1)))
        else:
            s["x"] = bf16(normal(T, d))
        if op == "exchange":
            s["dy"] = bf16(normal(T, d, scale=1.0 / math.sqrt(T)))
            s["dxs"] = bf16(normal(T * k, d, scale=1.0 / math.sqrt(T)))
    elif op == "norm8":
        d = case["d"]
        s["x"] = bf16(normal(T, d, scale=4.0))                  # the residual stream
        s["branch"] = bf16(normal(T, d) * torch.exp(normal(T, 1)))
        s["gate"] = normal(T)
        s["post_w"] = bf16(1.0 + normal(d, scale=0.2))
        s["pre_w"] = bf16(1.0 + normal(d, scale=0.2))
    elif op == "linear8":
        k, rows = case["k"], case["n"] * (2 if case["glu"] else 1)
        s["x"], s["x_scale"] = eight(normal(T, k))
        # the clamped activation meets gates past its limit (2 in 100)
        spread = 3.0 if case["glu"] and case["act"] == CLAMPED else 1.0
        s["w"], s["w_scale"] = eight(normal(rows, k, scale=spread / math.sqrt(k)))
        s["bias"] = bf16(normal(rows, scale=0.2))
    else:
        k, n = case["k"], case["n"]
        s["x"] = bf16(normal(T, k))
        s["w"] = bf16(normal(n, k, scale=1.0 / math.sqrt(k)))
        s["bias"] = bf16(normal(n, scale=0.2))
        s["residual"] = bf16(normal(T, n)) if case["residual"] else None
        if op == "train":
            s["dy"] = bf16(normal(T, n, scale=1.0 / math.sqrt(T)))
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import sparse_moe_ffn_route_gb300 as moe
    case = s["case"]
    op = case["op"]
    if "call" not in s:
        # what a program sets up once for its buffers: the configuration, workspace and outputs
        if op in ("dispatch", "combine", "exchange"):
            cfg = moe.exchange_cfg(case["d"], case["E"], case["k"],
                                   fmt=moe.ROWS_E4M3 if case.get("bits") == 8 else moe.ROWS_BF16)
            if op == "combine":
                s["call"] = moe.bind_combine_forward(cfg, s["z"], s["rows"], w=s["w"], residual=s["residual"])
            else:
                s["call"] = moe.bind_dispatch_forward(cfg, s["x"], s["ids"], x_scale=s.get("x_scale"))
            if op == "exchange":
                rows = s["call"].out.rows
                s["back"] = moe.bind_combine_forward(cfg, s["z"], rows, w=s["w"], residual=s["residual"])
                s["grad"] = moe.bind_combine_backward(cfg, s["dy"], s["z"], rows, s["w"])
                s["grad_x"] = moe.bind_dispatch_backward(cfg, s["dxs"], rows)
        elif op == "norm8":
            cfg = moe.norm_cfg(case["d"], eps=EPS, residual_scale=RESIDUAL, branch_scale=BRANCH)
            s["call"] = moe.bind_block_norm_quant(cfg, s["x"], branch=s["branch"], post_w=s["post_w"], gate=s["gate"],
                                                  pre_w=s["pre_w"])
        elif op == "linear8":
            cfg = moe.linear_cfg(case["k"], case["n"], act=case["act"], glu=case["glu"], fmt=moe.LINEAR_E4M3,
                                 glu_limit=LIMIT, glu_alpha=ALPHA)
            w = moe.LinearWeights(s["w"], bias=s["bias"], scale=s["w_scale"])
            s["call"] = moe.bind_linear_forward(cfg, s["x"], w, x_scale=s["x_scale"])
        else:
            cfg = moe.linear_cfg(case["k"], case["n"], act=case["act"])
            w = moe.LinearWeights(s["w"], bias=s["bias"])
            if op == "linear":
                s["call"] = moe.bind_linear_forward(cfg, s["x"], w, residual=s["residual"])
            else:
                pre = None if case["act"] == NONE else moe.linear_pre(cfg, case["T"])
                s["call"] = moe.bind_linear_forward(cfg, s["x"], w, residual=s["residual"], pre=pre)
                s["back"] = moe.bind_linear_backward(cfg, s["x"], w, s["dy"], pre=pre)
    if op in ("dispatch", "exchange"):
        sent = s["call"]()
        out = {"offsets": sent.offsets, "rows": sent.rows, "xs": sent.xs}
        if op == "dispatch":
            return {**out, "xs_scale": sent.xs_scale} if case["bits"] == 8 else out
        y = s["back"]()
        dz, dw = s["grad"]()
        return {**out, "y": y, "dz": dz, "dw": dw, "dx": s["grad_x"]()}
    if op == "norm8":
        y, q, scale = s["call"]()
        return {"y": y, "q": q, "scale": scale}
    if op == "train":
        y = s["call"]()
        dx, grads = s["back"]()
        return {"y": y, "dx": dx, "dw": grads.w, "dbias": grads.bias}
    return {"y": s["call"]()}


# ------------------------------------------------------------------ plain forms, 32 bits
def _sort(ids, E):
    """offsets [E + 1] and rows [T, k]: the slots in the order of their experts, equal ones in their own."""
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(flat.numel(), device=flat.device)
    counts = torch.zeros(E, dtype=torch.long, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    return offsets.to(torch.int32), rows.to(torch.int32).reshape(ids.shape)


def _scatter(x, rows, n):
    """out[rows[t, j]] = x[t] (or x[t, j])."""
    if x.dim() == 2:
        x = x[:, None].expand(-1, rows.shape[1], -1)
    out = torch.empty(n, x.shape[-1], dtype=x.dtype, device=x.device)
    out[rows.reshape(-1).long()] = x.reshape(n, -1)
    return out


def _act(z, act):
    if act == NONE:
        return z
    if act == SILU:
        return z / (1.0 + torch.exp(-z))
    if act == GELU:
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_slope(z, act):
    if act == NONE:
        return torch.ones_like(z)
    if act == SILU:
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == GELU:
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    c = 2.0 * math.sqrt(2.0 / math.pi)
    p = 1.0 / (1.0 + torch.exp(-c * (z + 0.044715 * z * z * z)))
    return p + z * p * (1.0 - p) * c * (1.0 + 3.0 * 0.044715 * z * z)


def _gated(g, u, act):
    if act == SWIGLU:
        return g / (1.0 + torch.exp(-g)) * u
    g = torch.clamp(g, max=LIMIT)
    return (torch.clamp(u, -LIMIT, LIMIT) + 1.0) * g / (1.0 + torch.exp(-ALPHA * g))


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    bf16 = torch.bfloat16
    if op in ("dispatch", "combine", "exchange"):
        out = {}
        rows = s.get("rows")
        if op != "combine":
            offsets, rows = _sort(s["ids"], case["E"])
            x = s["x"].view(torch.uint8) if s["x"].dtype == torch.float8_e4m3fn else s["x"]
            out = {"offsets": offsets, "rows": rows, "xs": _scatter(x, rows, rows.numel()).view(s["x"].dtype)}
            if "x_scale" in s:
                out["xs_scale"] = _scatter(s["x_scale"][:, None], rows, rows.numel())[:, 0]
        if op == "dispatch":
            return out
        at = rows.long()
        z = s["z"].float()[at]                                      # [T, k, d]
        out["y"] = (s["residual"].float() + (s["w"][:, :, None] * z).sum(1)).to(bf16)
        if op == "combine":
            return out
        dy = s["dy"].float()[:, None]
        out["dz"] = _scatter((s["w"][:, :, None] * dy).to(bf16), rows, rows.numel())
        out["dw"] = (dy * z).sum(2)
        out["dx"] = s["dxs"].float()[at].sum(1).to(bf16)
        return out
    if op == "norm8":
        x, z = s["x"].float(), s["branch"].float()
        p = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * s["post_w"].float()
        y = RESIDUAL * x + (BRANCH / (1.0 + torch.exp(-s["gate"])))[:, None] * p
        a = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * s["pre_w"].float()
        scale = (a.abs().amax(1) / E4M3_MAX).clamp(min=LEAST_SCALE)
        return {"y": y.to(bf16), "q": (a / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale}
    x, w = s["x"].float(), s["w"].float()
    if op == "linear8":
        # the products of the codes first: a scale multiplies whole sums
        v = (x @ w.T) * s["x_scale"][:, None] * s["w_scale"] + s["bias"].float()
        return {"y": (_gated(*v.split(case["n"], 1), case["act"]) if case["glu"] else _act(v, case["act"])).to(bf16)}
    v = x @ w.T + s["bias"].float()
    y = _act(v, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if op == "linear":
        return {"y": y.to(bf16)}
    dv = s["dy"].float() * _act_slope(v, case["act"])
    return {"y": y.to(bf16), "dx": (dv @ w).to(bf16), "dw": (dv.T @ x).to(bf16), "dbias": dv.sum(0).to(bf16)}


# ------------------------------------------------------------------ the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def leaf(name, grad):
        return s[name].double().requires_grad_(grad)

    if op in ("dispatch", "combine", "exchange"):
        E, k = case["E"], case["k"]
        flat = s["ids"].reshape(-1)
        hot = flat[:, None] == torch.arange(E, device=flat.device)
        seen = hot.cumsum(0)                                         # slots of each expert so far
        first = torch.cat((seen.new_zeros(1), seen[-1].cumsum(0)))
        row = first[:-1][flat.long()] + seen[torch.arange(flat.numel(), device=flat.device), flat.long()] - 1
        back = torch.argsort(row)                                    # the slot of each row
        token = back.div(k, rounding_mode="floor")
        out = {}
        if op != "combine":
            out = {"offsets": first, "rows": row.reshape(-1, k), "xs": s["x"].double()[token]}
        if op == "dispatch":
            return {**out, "xs_scale": s["x_scale"].double()[token]} if case["bits"] == 8 else out
        grad = op == "exchange"
        z, w, x = leaf("z", grad), leaf("w", grad), torch.zeros_like(s["residual"], dtype=torch.float64)
        # each row to its token, weighted
        y = x.index_add(0, token, w.reshape(-1)[back][:, None] * z) + s["residual"].double()
        out["y"] = y.detach()
        if grad:
            out["dz"], out["dw"] = torch.autograd.grad(y, (z, w), s["dy"].double())
            out["dx"] = x.index_add(0, token, s["dxs"].double())     # of a row's copies, their sum
        return out
    if op == "norm8":
        x, z, gate, post, pre = (s[n].double() for n in ("x", "branch", "gate", "post_w", "pre_w"))

        def norm(v, w):
            return v / (v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt() * w

        y = RESIDUAL * x + BRANCH * torch.sigmoid(gate).unsqueeze(1) * norm(z, post)
        a = norm(y, pre)
        scale = torch.maximum(a.abs().max(1).values / E4M3_MAX, torch.full_like(a[:, 0], LEAST_SCALE))
        # to the nearest value with three bits behind the first (steps of 2^-9 at least), ties to even
        v = a / scale[:, None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
        return {"y": y, "q": torch.round(v / step) * step, "scale": scale}
    if op == "linear8":
        w = s["w"].double() * s["w_scale"].double()[:, None]
        v = torch.einsum("tk,ok->to", s["x"].double() * s["x_scale"].double()[:, None], w) + s["bias"].double()
        if not case["glu"]:
            return {"y": _exact_act(v, case["act"])}
        g, u = v[:, :case["n"]], v[:, case["n"]:]
        if case["act"] == SWIGLU:
            return {"y": torch.nn.functional.silu(g) * u}
        g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
        return {"y": (u + 1.0) * g * torch.sigmoid(ALPHA * g)}
    train = op == "train"
    x, w, bias = leaf("x", train), leaf("w", train), leaf("bias", train)
    y = _exact_act(torch.nn.functional.linear(x, w, bias), case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].double()
    if not train:
        return {"y": y}
    dx, dw, db = torch.autograd.grad(y, (x, w, bias), s["dy"].double())
    return {"y": y.detach(), "dx": dx, "dw": dw, "dbias": db}


def _exact_act(z, act):
    if act == SILU:
        return torch.nn.functional.silu(z)
    if act in (GELU, GELU_TANH):
        return torch.nn.functional.gelu(z, approximate="tanh" if act == GELU_TANH else "none")
    return z
