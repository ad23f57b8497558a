"""The measured cases of the dense block's operators: the gated FFN (forward, and a training step
with its backward pass), the norms either side of a block with its gate and residual scale (forward
and backward), and the linear layer with 4-bit weights and group scales.

`run` computes them in plain torch operations in 32 bits, or, where `own` is set, through the
library's entry points.  `exact` is their definition in 64 bits, with the gradients from automatic
differentiation."""
import math

import torch

own = False

SWIGLU, CLAMPED = 0, 1
LIMIT, ALPHA, EPS = 7.0, 1.702, 1e-6


def listed():
    return [
        # the shared expert of a sparse layer on its own, one token of one sequence: latency
        {"name": "ffn token 2048x512", "op": "ffn", "T": 1, "d": 2048, "ff": 512, "act": SWIGLU},
        # a wide dense layer in a small decode batch: the weights' stream from memory
        {"name": "ffn batch 8 4096x12288", "op": "ffn", "T": 8, "d": 4096, "ff": 12288, "act": SWIGLU},
        # a ragged piece of a prompt, clamped activation, sizes that are no power of two
        {"name": "ffn prompt 777 2880x2880", "op": "ffn", "T": 777, "d": 2880, "ff": 2880, "act": CLAMPED},
        # a full prefill batch of a dense layer
        {"name": "ffn prefill 8192 2048x8192", "op": "ffn", "T": 8192, "d": 2048, "ff": 8192, "act": SWIGLU},
        # training steps: the narrow shared expert, a ragged batch with the clamped activation,
        # and a dense layer's full batch (the largest case)
        {"name": "train 4096 2048x512", "op": "train", "T": 4096, "d": 2048, "ff": 512, "act": SWIGLU},
        {"name": "train 1001 2880x2880", "op": "train", "T": 1001, "d": 2880, "ff": 2880, "act": CLAMPED},
        {"name": "train 8192 2048x8192", "op": "train", "T": 8192, "d": 2048, "ff": 8192, "act": SWIGLU},
        # between two blocks while decoding: post-norm, gate, residual and the next pre-norm
        {"name": "norm batch 8 2048", "op": "norm", "T": 8, "d": 2048},
        # the same over a prefill batch, and its backward pass in training
        {"name": "norm prefill 8192 2880", "op": "norm", "T": 8192, "d": 2880},
        {"name": "norm backward 8192 2048", "op": "norm_bwd", "T": 8192, "d": 2048},
        # 4-bit weights: gate and up with the activation for one token, and the largest matrix of a
        # decode step (an output projection) for sixteen sequences
        {"name": "w4 token 2048x512 glu", "op": "w4", "T": 1, "k": 2048, "n": 512, "group": 128, "zeros": False,
         "glu": True},
        {"name": "w4 batch 16 4096x32768", "op": "w4", "T": 16, "k": 4096, "n": 32768, "group": 64, "zeros": True,
         "glu": False},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "train", "norm", "norm_bwd", "w4"])
    if op in ("ffn", "train"):
        d, ff = _log(rng, 256, 4096, 8), _log(rng, 256, 8192, 8)
        most = 8192 * 2048 * 8192 // (d * ff)
        return {"op": op, "T": min(_log(rng, 1 if op == "ffn" else 16, 8192), most), "d": d, "ff": ff,
                "act": rng.choice([SWIGLU, CLAMPED])}
    if op in ("norm", "norm_bwd"):
        return {"op": op, "T": _log(rng, 1, 16384), "d": _log(rng, 256, 8192, 8)}
    group = rng.choice([32, 64, 128])
    glu = rng.random() < 0.5
    return {"op": op, "T": _log(rng, 1, 16), "k": _log(rng, 512, 8192, group), "n": _log(rng, 256, 16384),
            "group": group, "zeros": rng.random() < 0.5, "glu": glu}


def work(case):
    T = case["T"]
    if case["op"] in ("ffn", "train"):
        d, ff = case["d"], case["ff"]
        passes = 1 if case["op"] == "ffn" else 3     # products: 3 forward, 6 backward
        # x, the weights, y; in training also dy, dx and the weights' gradients
        nbytes = 2 * (2 * T * d + 3 * d * ff) * (1 if case["op"] == "ffn" else 2)
        return {"bytes": nbytes, "flops": 6 * T * d * ff * passes}
    if case["op"] == "norm":
        # x, branch -> y, a; the gates and both weights
        return {"bytes": 8 * T * case["d"] + 4 * T + 4 * case["d"], "flops": 12 * T * case["d"]}
    if case["op"] == "norm_bwd":
        # x, branch, dy, da -> dx, dbranch; gates and their gradients; the weights and theirs (fp32)
        return {"bytes": 12 * T * case["d"] + 8 * T + 12 * case["d"], "flops": 30 * T * case["d"]}
    rows = case["n"] * (2 if case["glu"] else 1)
    per_group = 3 if case["zeros"] else 2
    return {"bytes": rows * case["k"] // 2 + rows * (case["k"] // case["group"]) * per_group
            + 2 * T * (case["k"] + case["n"]), "flops": 2 * T * rows * case["k"]}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    def bf16(t):
        return t.to(torch.bfloat16)

    s = {"case": dict(case)}
    T = case["T"]
    if case["op"] in ("ffn", "train"):
        d, ff = case["d"], case["ff"]
        # the clamped activation meets gates past its limit (2 in 100)
        spread = 3.0 if case["act"] == CLAMPED else 1.0
        s["x"] = bf16(normal(T, d))
        s["gate"] = bf16(normal(ff, d, scale=spread / math.sqrt(d)))
        s["up"] = bf16(normal(ff, d, scale=spread / math.sqrt(d)))
        s["down"] = bf16(normal(d, ff, scale=1.0 / math.sqrt(ff)))
        if case["op"] == "train":
            s["dy"] = bf16(normal(T, d, scale=1.0 / math.sqrt(T)))
    elif case["op"] in ("norm", "norm_bwd"):
        d = case["d"]
        s["x"] = bf16(normal(T, d, scale=4.0))           # the residual stream
        s["branch"] = bf16(normal(T, d) * torch.exp(normal(T, 1)))   # a block's output, rows of any size
        s["gate"] = normal(T)
        s["post_w"] = bf16(1.0 + normal(d, scale=0.2))
        s["pre_w"] = bf16(1.0 + normal(d, scale=0.2))
        if case["op"] == "norm_bwd":
            s["dy"] = bf16(normal(T, d))
            s["da"] = bf16(normal(T, d))
    else:
        k, rows = case["k"], case["n"] * (2 if case["glu"] else 1)
        s["x"] = bf16(normal(T, k))
        s["codes"] = torch.randint(0, 256, (rows, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
        s["scales"] = bf16(torch.exp(normal(rows, k // case["group"], scale=0.3)) / (5.0 * math.sqrt(k)))
        s["zeros"] = (torch.randint(4, 12, (rows, k // case["group"]), generator=gen, device="cuda",
                                    dtype=torch.uint8) if case["zeros"] else None)
    return s


RESIDUAL, BRANCH = 0.9, 0.7


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import sparse_moe_ffn_route_gb300 as moe
    case = s["case"]
    op = case["op"]
    if "call" not in s:
        # what a program sets up once for its buffers: the configuration, workspace and outputs
        if op in ("ffn", "train"):
            cfg = moe.glu_cfg(case["d"], case["ff"], act=case["act"], glu_limit=LIMIT, glu_alpha=ALPHA)
            w = moe.GluWeights(s["gate"], s["up"], s["down"])
            ws = moe.glu_workspace(cfg, case["T"])
            if op == "ffn":
                s["call"] = moe.bind_glu_forward(cfg, s["x"], w, ws=ws)
            else:
                saved = moe.glu_saved(cfg, case["T"])
                s["call"] = moe.bind_glu_forward(cfg, s["x"], w, saved=saved, ws=ws)
                s["back"] = moe.bind_glu_backward(cfg, s["x"], w, saved, s["dy"], ws=ws)
        elif op in ("norm", "norm_bwd"):
            cfg = moe.norm_cfg(case["d"], eps=EPS, residual_scale=RESIDUAL, branch_scale=BRANCH)
            parts = dict(branch=s["branch"], post_w=s["post_w"], gate=s["gate"], pre_w=s["pre_w"])
            if op == "norm":
                s["call"] = moe.bind_block_norm_forward(cfg, s["x"], **parts)
            else:
                s["call"] = moe.bind_block_norm_backward(cfg, s["x"], dy=s["dy"], da=s["da"], **parts)
        else:
            cfg = moe.w4_cfg(case["k"], case["n"], group=case["group"], glu=case["glu"])
            s["call"] = moe.bind_w4_linear(cfg, s["x"], moe.W4Weights(s["codes"], s["scales"], s["zeros"]))
    if op == "train":
        y = s["call"]()
        dx, grads = s["back"]()
        return {"y": y, "dx": dx, "dgate": grads.gate, "dup": grads.up, "ddown": grads.down}
    if op == "norm":
        y, a = s["call"]()
        return {"y": y, "a": a}
    if op == "norm_bwd":
        g = s["call"]()
        return {"dx": g.dx, "dbranch": g.dbranch, "dgate": g.dgate, "dpost_w": g.dpost_w, "dpre_w": g.dpre_w}
    return {"y": s["call"]()}


# ------------------------------------------------------------------ plain forms, 32 bits
def _act(g, u, act):
    """h, and its derivatives by g and by u."""
    if act == SWIGLU:
        e = 1.0 / (1.0 + torch.exp(-g))
        return g * e * u, u * (e + g * e * (1.0 - e)), g * e
    gc = torch.where(g > LIMIT, torch.full_like(g, LIMIT), g)
    uc = torch.where(u > LIMIT, torch.full_like(u, LIMIT), torch.where(u < -LIMIT, torch.full_like(u, -LIMIT), u))
    e = 1.0 / (1.0 + torch.exp(-ALPHA * gc))
    by_g = (uc + 1.0) * (e + ALPHA * gc * e * (1.0 - e)) * (g <= LIMIT)
    by_u = gc * e * (u.abs() <= LIMIT)
    return (uc + 1.0) * gc * e, by_g, by_u


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    x = s["x"].float()
    if op in ("ffn", "train"):
        wg, wu, wd = s["gate"].float(), s["up"].float(), s["down"].float()
        h, by_g, by_u = _act(x @ wg.T, x @ wu.T, case["act"])
        y = (h @ wd.T).bfloat16()
        if op == "ffn":
            return {"y": y}
        dy = s["dy"].float()
        dh = dy @ wd
        dg, du = dh * by_g, dh * by_u
        return {"y": y, "dx": (dg @ wg + du @ wu).bfloat16(), "dgate": (dg.T @ x).bfloat16(),
                "dup": (du.T @ x).bfloat16(), "ddown": (dy.T @ h).bfloat16()}
    if op in ("norm", "norm_bwd"):
        z, wpost, wpre = s["branch"].float(), s["post_w"].float(), s["pre_w"].float()
        rz = 1.0 / torch.sqrt((z * z).mean(1, keepdim=True) + EPS)
        p = z * rz * wpost
        gate = (1.0 / (1.0 + torch.exp(-s["gate"])))[:, None]
        y = RESIDUAL * x + BRANCH * gate * p
        ry = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
        if op == "norm":
            return {"y": y.bfloat16(), "a": (y * ry * wpre).bfloat16()}
        da = s["da"].float()
        q = da * wpre
        total = s["dy"].float() + ry * (q - y * ry * ry * (q * y).mean(1, keepdim=True))
        dp = BRANCH * gate * total
        v = dp * wpost
        return {"dx": (RESIDUAL * total).bfloat16(),
                "dbranch": (rz * (v - z * rz * rz * (v * z).mean(1, keepdim=True))).bfloat16(),
                "dgate": (BRANCH * gate * (1.0 - gate))[:, 0] * (total * p).sum(1),
                "dpost_w": (dp * z * rz).sum(0), "dpre_w": (da * y * ry).sum(0)}
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), 2).reshape(s["codes"].shape[0], -1, case["group"]).float()
    q = q - (8.0 if s["zeros"] is None else s["zeros"].float()[:, :, None])
    w = (q * s["scales"].float()[:, :, None]).reshape(q.shape[0], -1)
    y = x @ w.T
    if case["glu"]:
        y = _act(y[:, : case["n"]], y[:, case["n"]:], SWIGLU)[0]
    return {"y": y.bfloat16()}


# ------------------------------------------------------------------ the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def leaf(name, grad=True):
        return s[name].double().requires_grad_(grad)

    def activation(g, u, act):
        if act == SWIGLU:
            return g * torch.sigmoid(g) * u
        g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
        return (u + 1) * (g * torch.sigmoid(ALPHA * g))

    if op in ("ffn", "train"):
        x, wg, wu, wd = (leaf(n, op == "train") for n in ("x", "gate", "up", "down"))
        linear = torch.nn.functional.linear
        y = linear(activation(linear(x, wg), linear(x, wu), case["act"]), wd)
        if op == "ffn":
            return {"y": y}
        dx, dg, du, dd = torch.autograd.grad(y, (x, wg, wu, wd), s["dy"].double())
        return {"y": y.detach(), "dx": dx, "dgate": dg, "dup": du, "ddown": dd}
    if op in ("norm", "norm_bwd"):
        x, z, gate, post, pre = (leaf(n, op == "norm_bwd") for n in ("x", "branch", "gate", "post_w", "pre_w"))

        def norm(v, w):
            return v * (v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS).rsqrt() * w

        y = RESIDUAL * x + BRANCH * torch.sigmoid(gate).unsqueeze(1) * norm(z, post)
        a = norm(y, pre)
        if op == "norm":
            return {"y": y, "a": a}
        got = torch.autograd.grad((y, a), (x, z, gate, post, pre), (s["dy"].double(), s["da"].double()))
        return dict(zip(("dx", "dbranch", "dgate", "dpost_w", "dpre_w"), got))
    codes = s["codes"].to(torch.int32)
    q = torch.empty(codes.shape[0], case["k"], dtype=torch.float64, device=codes.device)
    q[:, 0::2] = codes.remainder(16).double()
    q[:, 1::2] = codes.div(16, rounding_mode="floor").double()
    groups = torch.arange(case["k"], device=codes.device).div(case["group"], rounding_mode="floor")
    zero = 8.0 if s["zeros"] is None else s["zeros"].double()[:, groups]
    y = torch.einsum("tk,ok->to", s["x"].double(), (q - zero) * s["scales"].double()[:, groups])
    if case["glu"]:
        y = activation(*y.split(case["n"], 1), SWIGLU)
    return {"y": y}
