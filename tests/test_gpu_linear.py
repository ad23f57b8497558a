"""The linear layer and the norm with an output in 8 bits against plain implementations in 64 bits.

Bounds are worst-case rounding bounds, element by element, as in test_gpu_block: an output rounded
to bf16 is off by at most half a step, 2^-8 of its value (H); a sum of n products in fp32 by n 2^-23
(F) of the sum of their magnitudes; activations and norms lose 2^-18 (R) in all; a value rounded to
e4m3 is off by half a step, 2^-4 of it (below 2^-6: 2^-10)."""
import math

import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_gpu_block import ALPHA, F, H, LIMIT, R, Guarded, act64, close, gen_for, norm64, rnd  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = [moe.LINEAR_NONE, moe.LINEAR_SILU, moe.LINEAR_GELU, moe.LINEAR_GELU_TANH]
# bounds of |act'| and |act''| (GELU: 1.129 and 0.798; its tanh form and SiLU stay below 1.13 and 0.85)
SLOPE, CURVE = 1.13, 0.85


def lin64(v, act):
    if act == moe.LINEAR_SILU:
        return v * torch.sigmoid(v)
    if act == moe.LINEAR_GELU:
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if act == moe.LINEAR_GELU_TANH:
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def slope64(v, act):
    with torch.enable_grad():
        v = v.detach().requires_grad_()
        return torch.autograd.grad(lin64(v, act).sum(), v)[0]


def sums64(x, w, xs, ws, bias):
    """v and its bound."""
    x, w = x.double(), w.double()
    k = x.shape[1]
    by = 1.0 if xs is None else xs.double()[:, None] * ws.double()
    v, e = (x @ w.T) * by, k * F * (x.abs() @ w.abs().T) * by
    e = e + 2 * F * v.abs()
    if bias is not None:
        v = v + bias.double()
        e = e + F * v.abs()
    return v, e


def y64(v, e, case, residual):
    """y and its bound, from v and its bound."""
    if case["glu"]:
        n = v.shape[1] // 2
        g, u, eg, eu = v[:, :n], v[:, n:], e[:, :n], e[:, n:]
        y, _, _ = act64(g, u, case["act"])
        ey = 1.1 * (u.abs() + 1 + eu) * eg + (g.abs() + eg) * eu + R * y.abs()
    else:
        y = lin64(v, case["act"])
        ey = SLOPE * e + (R * y.abs() if case["act"] else 0.0)
    if residual is not None:
        y = y + residual.double()
        ey = ey + F * y.abs()
    return y, H * y.abs() + 1.01 * ey


def inputs(T, k, n, fmt=0, glu=False, seed=0, bias=True, residual=True):
    gen = gen_for(T, k, n, fmt, glu, seed)
    rows = 2 * n if glu else n
    x, w = rnd(gen, T, k), rnd(gen, rows, k, scale=2.0 / k ** 0.5)
    b = rnd(gen, rows) if bias else None
    r = rnd(gen, T, n) if residual else None
    if fmt == moe.LINEAR_E4M3:
        x, xs = moe.w8_quantize(x.float() * torch.exp(rnd(gen, T, 1).float()))
        w, ws = moe.w8_quantize(w)
        return x, xs, moe.LinearWeights(w, b, ws), r, gen
    return x, None, moe.LinearWeights(w, b), r, gen


# one token to several tiles, single CTAs, pairs and split sums, ragged on every side
SIZES = [(1, 16, 8), (1, 2048, 512), (2, 80, 1000), (5, 4096, 72), (16, 8208, 40), (16, 2880, 2880), (17, 64, 128),
         (40, 2048, 256), (64, 8192, 1024), (100, 3008, 3000), (127, 256, 264), (129, 272, 136), (300, 512, 4096),
         (777, 2880, 640), (1500, 1024, 1000)]


@pytest.mark.parametrize("fmt", [moe.LINEAR_BF16, moe.LINEAR_E4M3])
@pytest.mark.parametrize("T,k,n", SIZES)
def test_forward(T, k, n, fmt):
    for i, (act, bias, residual) in enumerate([(0, False, False), (1, True, False), (2, False, True), (3, True, True), (0, True, True)]):
        x, xs, w, r, _ = inputs(T, k, n, fmt, seed=i, bias=bias, residual=residual)
        cfg = moe.linear_cfg(k, n, act=act, fmt=fmt)
        y, pre, ws = Guarded((T, n)), Guarded((T, n)), moe.linear_workspace(cfg, T)
        moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r, pre=pre.t, y=y.t, ws=ws)
        assert moe.moe_device_status(ws)[0] == moe.MOE_OK
        v, e = sums64(x, w.w, xs, w.scale, w.bias)
        close(pre.t, v, H * v.abs() + 1.01 * e, ("pre", act))
        close(y.t, *y64(v, e, dict(glu=False, act=act), r), ("y", act))
        y.check()
        pre.check()
        assert torch.equal(moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r), y.t)
        if r is not None:   # in place
            moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r, y=r)
            assert torch.equal(r, y.t)


@pytest.mark.parametrize("fmt", [moe.LINEAR_BF16, moe.LINEAR_E4M3])
@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_CLAMPED_GLU])
@pytest.mark.parametrize("T,k,n", SIZES)
def test_forward_gated(T, k, n, act, fmt):
    for i, (bias, residual) in enumerate([(False, False), (True, True)]):
        x, xs, w, r, _ = inputs(T, k, n, fmt, True, seed=i + 2 * act, bias=bias, residual=residual)
        cfg = moe.linear_cfg(k, n, act=act, glu=True, fmt=fmt, glu_limit=LIMIT, glu_alpha=ALPHA)
        y = Guarded((T, n))
        moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r, y=y.t)
        v, e = sums64(x, w.w, xs, w.scale, w.bias)
        close(y.t, *y64(v, e, dict(glu=True, act=act), r), "y")
        y.check()


BACK = [(1, 64, 8), (16, 80, 264), (17, 256, 72), (100, 1000, 520), (129, 136, 1032), (777, 640, 2880), (1500, 1024, 512),
        (2206, 456, 1000), (8192, 256, 512), (3000, 2048, 2048)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,k,n", BACK)
def test_backward(T, k, n, act):
    x, _, w, _, gen = inputs(T, k, n, seed=act + 10, residual=False)
    dy = rnd(gen, T, n, scale=1.0 / T ** 0.5)
    cfg = moe.linear_cfg(k, n, act=act)
    ws = Guarded((moe.moe_linear_workspace_bytes(cfg, T),), torch.uint8)     # rubbish in it
    pre = moe.linear_pre(cfg, T)
    moe.moe_linear_forward(cfg, x, w, pre=pre, ws=ws.t)
    dx, dw, db = Guarded((T, k)), Guarded((n, k)), Guarded((n,))
    kept = None if act == moe.LINEAR_NONE else pre
    moe.moe_linear_backward(cfg, x, w, dy, pre=kept, dx=dx.t, grads=moe.LinearGrads(dw.t, db.t), ws=ws.t)
    assert moe.moe_device_status(ws.t)[0] == moe.MOE_OK
    # from the kept pre, whose own rounding test_forward bounds
    g = dy.double()
    s = slope64(pre.double(), act)
    dv = g * s
    edv = R * (dv.abs() + g.abs()) if act else 0 * dv
    rdv = edv + (H * (dv.abs() + edv) if act else 0.0)      # rounded for the products
    W, X = w.w.double(), x.double()
    want = dv @ W
    close(dx.t, want, H * want.abs() + 1.01 * (rdv @ W.abs() + n * F * (dv.abs() @ W.abs())), "dx")
    want = dv.T @ X
    close(dw.t, want, H * want.abs() + 1.01 * (rdv.T @ X.abs() + T * F * (dv.abs().T @ X.abs())), "dw")
    want = dv.sum(0)
    close(db.t, want, H * want.abs() + 1.01 * (edv.sum(0) + T * F * dv.abs().sum(0)), "dbias")
    for b in (dx, dw, db, ws):
        b.check()
    # parts of the outputs alone: the same to within how the sums over the tokens are cut
    only = moe.moe_linear_backward(cfg, x, w, dy, pre=kept, grads=moe.LinearGrads(None, None))[0]
    want = dv @ W
    close(only, want, H * want.abs() + 1.01 * (rdv @ W.abs() + n * F * (dv.abs() @ W.abs())), "dx alone")
    ws.t.fill_(0xA5)
    none, grads = moe.moe_linear_backward(cfg, x, w, dy, pre=kept, need_dx=False, grads=moe.LinearGrads(None, torch.empty_like(db.t)), ws=ws.t)
    assert none is None and grads.w is None and torch.equal(grads.bias, db.t)
    assert moe.moe_device_status(ws.t)[0] == moe.MOE_OK
    _, grads = moe.moe_linear_backward(cfg, x, w, dy, pre=kept, need_dx=False, grads=moe.LinearGrads(torch.empty_like(dw.t), None))
    want = dv.T @ X
    close(grads.w, want, H * want.abs() + 1.01 * (rdv.T @ X.abs() + T * F * (dv.abs().T @ X.abs())), "dw alone")
    # twice the same bits
    again = moe.moe_linear_backward(cfg, x, w, dy, pre=kept)
    assert torch.equal(again[0], dx.t) and torch.equal(again[1].w, dw.t) and torch.equal(again[1].bias, db.t)


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_formula_and_differences(act):
    """The whole pass, pre kept in bf16, against automatic differentiation in 64 bits, and that against
    central differences."""
    T, k, n = 50, 136, 72
    x, _, w, r, gen = inputs(T, k, n, seed=30 + act)
    dy = rnd(gen, T, n)
    cfg, pre = moe.linear_cfg(k, n, act=act), moe.linear_pre(moe.linear_cfg(k, n), T)
    moe.moe_linear_forward(cfg, x, w, residual=r, pre=pre)
    dx, g = moe.moe_linear_backward(cfg, x, w, dy, pre=None if act == 0 else pre)
    leaves = [t.double().requires_grad_() for t in (x, w.w, w.bias)]

    def loss(a, b, c):
        return (dy.double() * (lin64(a @ b.T + c, act) + r.double())).sum()

    want = torch.autograd.grad(loss(*leaves), leaves)
    with torch.no_grad():
        along = [rnd(gen, *t.shape).double() for t in leaves]
        h = 1e-5
        num = (loss(*(t + h * u for t, u in zip(leaves, along))) - loss(*(t - h * u for t, u in zip(leaves, along)))) / (2 * h)
        dot = sum((a * b).sum() for a, b in zip(want, along))
        assert abs(num - dot) <= 1e-6 * sum((a * b).abs().sum() for a, b in zip(want, along))
        v, e = sums64(x, w.w, None, None, w.bias)
        ev = (H * v.abs() + 1.01 * e) if act else 0 * v                 # of the kept pre
        dv = dy.double() * slope64(v, act)
        edv = dy.double().abs() * (CURVE * ev + (2 * R if act else 0.0))
        rdv = edv + (H * (dv.abs() + edv) if act else 0.0)
        W, X = w.w.double(), x.double()
        close(dx, want[0], H * want[0].abs() + 1.01 * (rdv @ W.abs() + n * F * (dv.abs() @ W.abs())), "dx")
        close(g.w, want[1], H * want[1].abs() + 1.01 * (rdv.T @ X.abs() + T * F * (dv.abs().T @ X.abs())), "dw")
        close(g.bias, want[2], H * want[2].abs() + 1.01 * (edv.sum(0) + T * F * dv.abs().sum(0)), "dbias")


@pytest.mark.parametrize("fmt", [moe.LINEAR_BF16, moe.LINEAR_E4M3])
@pytest.mark.parametrize("T", [7, 16, 200])
def test_rows_do_not_mix(T, fmt):
    """NaN and infinities of a token's row, a weight's row, a scale or a bias stay in their row or
    column; far activations take their limits."""
    k, n = 144, 96
    x, xs, w, r, _ = inputs(T, k, n, fmt, seed=4)
    cfg = moe.linear_cfg(k, n, act=moe.LINEAR_SILU, fmt=fmt)
    clean = moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r)

    def changed(t, at, v):
        c = (t.float() if t.dtype == torch.float8_e4m3fn else t).clone()
        c[at] = v
        return c.to(t.dtype)

    nan = float("nan")
    y = moe.moe_linear_forward(cfg, changed(x, (3, 5), nan), w, x_scale=xs, residual=r)
    rows = [i for i in range(T) if i != 3]
    assert torch.isnan(y[3]).all() and torch.equal(y[rows], clean[rows])
    y = moe.moe_linear_forward(cfg, x, moe.LinearWeights(changed(w.w, (10, 5), nan), w.bias, w.scale), x_scale=xs, residual=r)
    cols = [i for i in range(n) if i != 10]
    assert torch.isnan(y[:, 10]).all() and torch.equal(y[:, cols], clean[:, cols])
    y = moe.moe_linear_forward(cfg, x, moe.LinearWeights(w.w, changed(w.bias, 7, float("inf")), w.scale), x_scale=xs, residual=r)
    cols = [i for i in range(n) if i != 7]
    assert torch.isinf(y[:, 7]).all() and torch.equal(y[:, cols], clean[:, cols])
    if fmt == moe.LINEAR_E4M3:
        y = moe.moe_linear_forward(cfg, x, w, x_scale=changed(xs, 2, nan), residual=r)
        rows = [i for i in range(T) if i != 2]
        assert torch.isnan(y[2]).all() and torch.equal(y[rows], clean[rows])
    for act in ACTS[1:]:    # +-300, where exp leaves fp32's range
        b = torch.where(torch.arange(n, device="cuda") % 2 == 0, 300.0, -300.0).bfloat16()
        y = moe.moe_linear_forward(moe.linear_cfg(k, n, act=act, fmt=fmt), x, moe.LinearWeights(w.w, b, w.scale), x_scale=xs)
        v, e = sums64(x, w.w, xs, w.scale, b)
        close(y, *y64(v, e, dict(glu=False, act=act), None), "far")


def test_scales_at_the_ends_of_their_range():
    """A product of scales alone would leave fp32's range."""
    T, k, n = 20, 64, 16
    x, xs, w, _, _ = inputs(T, k, n, moe.LINEAR_E4M3, bias=False, residual=False)
    xs = torch.full_like(xs, 2.0 ** -100)
    xs[::2] = 2.0 ** 100
    s = torch.full_like(w.scale, 2.0 ** 90)
    for few in (False, True):
        t = slice(0, 5 if few else T)
        y = moe.moe_linear_forward(moe.linear_cfg(k, n, fmt=moe.LINEAR_E4M3), x[t].contiguous(),
                                   moe.LinearWeights(w.w, None, s), x_scale=xs[t].contiguous())
        v, e = sums64(x[t], w.w, xs[t], s, None)
        small = torch.arange(v.shape[0], device="cuda") % 2 == 1
        close(y[small], v[small], (H * v.abs() + 1.01 * e)[small], "small")
        assert torch.isinf(y[~small]).all() or (v[~small].abs() < 2.0 ** 128).any()


@pytest.mark.parametrize("T", [3, 16, 40, 300])
def test_scales_of_a_run_of_rows(T):
    """x_scale may start on any fp32."""
    x, xs, w, r, _ = inputs(T, 128, 96, moe.LINEAR_E4M3, seed=60)
    cfg = moe.linear_cfg(128, 96, fmt=moe.LINEAR_E4M3)
    want = moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r)
    for shift in (1, 2, 3):
        room = torch.full((T + 8,), float("nan"), device="cuda")
        room[shift:shift + T] = xs
        assert torch.equal(moe.moe_linear_forward(cfg, x, w, x_scale=room[shift:shift + T], residual=r), want)


def test_no_tokens():
    x, _, w, _, _ = inputs(4, 64, 48)
    cfg = moe.linear_cfg(64, 48)
    assert moe.moe_linear_forward(cfg, x[:0], w).shape == (0, 48)
    dx, g = moe.moe_linear_backward(cfg, x[:0], w, torch.empty(0, 48, dtype=torch.bfloat16, device="cuda"))
    assert dx.shape == (0, 64) and (g.w == 0).all() and (g.bias == 0).all()
    y, q, s = moe.moe_block_norm_quant(moe.norm_cfg(64), x[:0], pre_w=x[0])
    assert y is None and q.shape == (0, 64) and s.shape == (0,)


@pytest.mark.parametrize("T,k,n,glu", [(64, 2048, 256, False), (300, 256, 2048, True), (700, 512, 1024, False)])
@pytest.mark.parametrize("fmt", [moe.LINEAR_BF16, moe.LINEAR_E4M3])
def test_wait_gives_up_reports_timeout_and_recovers(T, k, n, glu, fmt):
    x, xs, w, r, _ = inputs(T, k, n, fmt, glu)
    cfg = moe.linear_cfg(k, n, act=1, glu=glu, fmt=fmt)
    ws = moe.linear_workspace(cfg, T)
    want = moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r, ws=ws)
    assert moe.moe_device_status(ws)[0] == moe.MOE_OK
    try:
        moe.moe_test_set_wait_limit(1 << 14, True)
        moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r, ws=ws)
        status, bits = moe.moe_device_status(ws)
    finally:
        moe.moe_test_set_wait_limit(moe.DEFAULT_WAIT_POLLS, False)
    assert status == -7 and bits & (1 << 8), (status, bits)
    assert torch.equal(moe.moe_linear_forward(cfg, x, w, x_scale=xs, residual=r, ws=ws), want)
    assert moe.moe_device_status(ws)[0] == moe.MOE_OK


# ----------------------------------------------------------------------------- norm in 8 bits
NORMS = [(1, 8), (3, 64), (8, 2048), (5, 2056), (33, 2880), (300, 520), (7, 8192), (4, 8200), (2, 16384), (2000, 256)]


def quant_close(q, scale, a, ea):
    """scale and codes of a, given a's bound."""
    top = a.abs().amax(1)
    etop = ea.amax(1)
    want = (top / 448).clamp(min=2.0 ** -126)
    assert ((scale.double() - want).abs() <= 1.01 * etop / 448 + 4 * F * want).all()
    v = a / scale.double()[:, None]
    tol = torch.maximum(2.0 ** -4 * v.abs(), torch.full_like(v, 2.0 ** -10)) * 1.01 + 1.1 * ea / scale.double()[:, None] + 4 * F * v.abs()
    close(q.float(), v, tol, "q")
    assert (q.float().abs().amax(1)[top > 0] == 448).all()      # the largest takes the largest code


@pytest.mark.parametrize("parts", ["all", "plain", "no pre", "no post", "x norm", "x", "gate"])
@pytest.mark.parametrize("T,d", NORMS)
def test_norm_quant(T, d, parts):
    gen = gen_for(T, d, len(parts))
    x, z = rnd(gen, T, d, scale=3.0), rnd(gen, T, d) * torch.exp(rnd(gen, T, 1).float()).bfloat16()
    post, gate, pre = 1 + rnd(gen, d, scale=0.2), rnd(gen, T, dtype=torch.float32), 1 + rnd(gen, d, scale=0.2)
    kw = {"all": dict(branch=z, post_w=post, gate=gate, pre_w=pre), "plain": dict(branch=z), "no pre": dict(branch=z, post_w=post),
          "no post": dict(branch=z, gate=gate, pre_w=pre), "x norm": dict(pre_w=pre), "x": {}, "gate": dict(branch=z, gate=gate)}[parts]
    cfg = moe.norm_cfg(d, residual_scale=0.9, branch_scale=0.7)
    y, q, s = Guarded((T, d)) if "branch" in kw else None, Guarded((T, d), torch.float8_e4m3fn), Guarded((T,), torch.float32)
    moe.moe_block_norm_quant(cfg, x, y=y and y.t, q=q.t, scale=s.t, **kw)
    full = {k: kw.get(k) for k in ("branch", "post_w", "gate", "pre_w")}
    out = norm64(x, full["branch"], full["post_w"], full["gate"], full["pre_w"], None, None, 0.9, 0.7)
    if y is not None:
        close(y.t, *out["y"], "y")
        y.check()
        # moe_block_norm_forward's y: a row's squares may be added in another order there (a thread has
        # other elements), so that both are within the bound of the exact value, and of each other by
        # twice that
        close(moe.moe_block_norm_forward(cfg, x, **kw)[0], y.t.double(), 2 * out["y"][1], "y of the bf16 form")
    if full["pre_w"] is not None:
        a, ea = out["a"]
        ea = ea - H * a.abs()        # a is not rounded to bf16
    elif y is not None:
        a, ea = out["y"]
        ea = ea - H * a.abs()
    else:
        a, ea = x.double(), 0 * x.double()
    quant_close(q.t, s.t, a, ea)
    q.check()
    s.check()


def test_norm_quant_rows_of_zeros_nan_and_infinities():
    d = 64
    x = rnd(gen_for(2), 6, d)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 2.0 ** -133          # a subnormal of bf16: the scale's least value holds
    cfg = moe.norm_cfg(d)
    _, q, s = moe.moe_block_norm_quant(cfg, x)
    assert s[1] == 2.0 ** -126 and (q[1].float() == 0).all()
    assert torch.isnan(q[2].float()).tolist() == [i == 5 for i in range(d)]
    assert s[2].item() == pytest.approx(x[2].float().nan_to_num(0).abs().max().item() / 448, rel=1e-6)
    assert torch.isinf(s[3]) and torch.isnan(q[3].float())[7] and (q[3].float()[[i for i in range(d) if i != 7]] == 0).all()
    assert s[4] == 2.0 ** -126 and (q[4].float() == 2.0 ** -7).all()
    _, qc, sc = moe.moe_block_norm_quant(cfg, x[[0, 5]].contiguous())
    assert torch.equal(q.view(torch.uint8)[[0, 5]], qc.view(torch.uint8)) and torch.equal(s[[0, 5]], sc)
    # with the norm a row of zeros stays one
    _, q, s = moe.moe_block_norm_quant(cfg, x, pre_w=torch.ones(d, dtype=torch.bfloat16, device="cuda"))
    assert s[1] == 2.0 ** -126 and (q[1].float() == 0).all() and torch.isnan(q[2].float()).all()


def test_quantisers_agree():
    """The norm's kernel on x alone and the weights' quantiser: the same scales to a step of fp32, and
    codes that differ at most where a value lies on a border."""
    x = rnd(gen_for(8), 200, 1032)
    _, q, s = moe.moe_block_norm_quant(moe.norm_cfg(1032), x)
    p, t = moe.w8_quantize(x)
    assert ((s - t).abs() <= F * t).all()
    assert (q.view(torch.uint8) != p.view(torch.uint8)).float().mean() < 1e-3


def test_norm_quant_in_place_y():
    gen = gen_for(6)
    x, z, pre = rnd(gen, 50, 264), rnd(gen, 50, 264), rnd(gen, 264)
    cfg = moe.norm_cfg(264)
    y, q, s = moe.moe_block_norm_quant(cfg, x, branch=z, pre_w=pre)
    y2, q2, s2 = moe.moe_block_norm_quant(cfg, x, branch=z, pre_w=pre, y=x)
    assert y2 is x and torch.equal(x, y) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


# ----------------------------------------------------------------------------- calls
@pytest.mark.parametrize("T,k,n", [(5, 136, 96), (100, 136, 96), (300, 264, 304), (1200, 128, 512)])
def test_tensors_on_odd_multiples_of_16_bytes(T, k, n):
    """Tensors that begin 16 bytes past a multiple of 32 give the bits that aligned ones give."""
    gen = gen_for(T, n, 16)

    def off(t):
        flat = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
        step = 16 // t.element_size()
        start = step if flat.data_ptr() % 32 == 0 else 0
        v = flat[start:start + t.numel()].view(t.shape)
        assert v.data_ptr() % 32 == 16
        return v.copy_(t)

    x, w, b, r, dy = rnd(gen, T, k), rnd(gen, n, k, scale=k ** -0.5), rnd(gen, n), rnd(gen, T, n), rnd(gen, T, n)
    cfg = moe.linear_cfg(k, n, act=moe.LINEAR_GELU)
    pre, pre2, y2 = moe.linear_pre(cfg, T), off(moe.linear_pre(cfg, T)), off(dy)
    y = moe.moe_linear_forward(cfg, x, moe.LinearWeights(w, b), residual=r, pre=pre)
    moe.moe_linear_forward(cfg, off(x), moe.LinearWeights(off(w), off(b)), residual=off(r), pre=pre2, y=y2)
    assert torch.equal(y, y2) and torch.equal(pre, pre2)
    dx, g = moe.moe_linear_backward(cfg, x, moe.LinearWeights(w, b), dy, pre=pre)
    dx2, g2 = moe.moe_linear_backward(cfg, off(x), moe.LinearWeights(off(w), off(b)), off(dy), pre=off(pre), dx=off(dx),
                                      grads=moe.LinearGrads(off(g.w), off(g.bias)))
    assert torch.equal(dx, dx2) and torch.equal(g.w, g2.w) and torch.equal(g.bias, g2.bias)


def test_captured_and_replayed_beside_eager_calls():
    T, k, n = 200, 264, 520
    x, _, w, r, gen = inputs(T, k, n, seed=40)
    dy = rnd(gen, T, n)
    cfg = moe.linear_cfg(k, n, act=moe.LINEAR_GELU)

    def step():
        pre = moe.linear_pre(cfg, T)
        y = moe.moe_linear_forward(cfg, x, w, residual=r, pre=pre)
        dx, g = moe.moe_linear_backward(cfg, x, w, dy, pre=pre)
        return y, dx, g.w, g.bias

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for turn in range(4):
        x.copy_(rnd(gen, T, k))
        dy.copy_(rnd(gen, T, n))
        graphs[turn % 2].replay()
        for a, b in zip(outs[turn % 2], step()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [4, 600])
def test_two_calls_at_once_on_streams_of_their_own(T):
    x, _, w, r, _ = inputs(T, 512, 1024, seed=50)
    x8, xs, w8, r8, _ = inputs(T, 512, 1024, moe.LINEAR_E4M3, True, seed=51)
    cfg, cfg8 = moe.linear_cfg(512, 1024, act=2), moe.linear_cfg(512, 1024, glu=True, fmt=moe.LINEAR_E4M3)
    want = moe.moe_linear_forward(cfg, x, w, residual=r), moe.moe_linear_forward(cfg8, x8, w8, x_scale=xs, residual=r8)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    got = [(moe.moe_linear_forward(cfg, x, w, residual=r, stream=a),
            moe.moe_linear_forward(cfg8, x8, w8, x_scale=xs, residual=r8, stream=b)) for _ in range(20)]
    for s in (a, b):
        torch.cuda.current_stream().wait_stream(s)
    for p, q in got:
        assert torch.equal(p, want[0]) and torch.equal(q, want[1])
