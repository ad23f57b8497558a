"""The dense block's kernels against plain implementations in 64 bits.

Bounds are worst-case rounding bounds, element by element.  An output rounded to bf16 is
off by at most half a step, 2^-8 of its value (H); so is every operand rounded to bf16 on
the way (h, dg, du).  A sum of n products in fp32 is off by at most n 2^-23 of the sum of
their magnitudes (each addition rounds or truncates once); activations and norms lose a few
2^-24 per step, taken as 2^-18 (R) in all.
"""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")

pytestmark = pytest.mark.gpu

H, F, R = 2.0 ** -8, 2.0 ** -23, 2.0 ** -18
LIMIT, ALPHA = 7.0, 1.702


def rnd(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def gen_for(*key):
    return torch.Generator(device="cuda").manual_seed(sum((i + 1) * 7919 * int(k) for i, k in enumerate(key)))


def close(got, want, tol, name):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (name, int(bad.sum()), float((got - want)[bad].abs().max()), float(tol[bad].min()),
                           bad.nonzero()[:4].tolist())


class Guarded:
    """An output in the middle of a larger buffer whose other bytes must not change."""

    def __init__(self, shape, dtype=torch.bfloat16):
        n = 1
        for s in shape:
            n *= s
        self.pad = 4096
        size = n * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((size + 2 * self.pad,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.raw[self.pad:self.pad + size].view(dtype).view(shape)

    def check(self):
        assert (self.raw[:self.pad] == 0xA5).all() and (self.raw[-self.pad:] == 0xA5).all()


# ----------------------------------------------------------------------------- gated FFN
def act64(g, u, act):
    """h, dh/dg, dh/du."""
    if act == moe.ACT_SWIGLU:
        s = torch.sigmoid(g)
        return g * s * u, u * (s + g * s * (1 - s)), g * s
    gc, uc = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    s = torch.sigmoid(ALPHA * gc)
    return ((uc + 1) * gc * s, (uc + 1) * (s + ALPHA * gc * s * (1 - s)) * (g <= LIMIT),
            gc * s * (u.abs() <= LIMIT))


def glu64(x, wg, wu, wd, dy, act):
    """Results and bounds: {name: (value, tolerance)}."""
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    T, d = x.shape
    ff = wg.shape[0]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = d * F * (x.abs() @ wg.abs().T), d * F * (x.abs() @ wu.abs().T)
    h, by_g, by_u = act64(g, u, act)
    # |dh/dg| <= 1.1 (|u| + 1), |dh/du| <= |g|, second derivatives of the gate at most
    # max(1, alpha) / 2, to first order in eg, eu
    eh = 1.1 * (u.abs() + 1 + eu) * eg + (g.abs() + eg) * eu + R * h.abs()
    near = ((g.abs() - LIMIT).abs() <= eg) | ((u.abs() - LIMIT).abs() <= eu)   # may clamp either way
    y = h @ wd.T
    eh = eh + H * (h.abs() + eh)
    out = {"y": (y, H * y.abs() + 1.01 * (eh @ wd.abs().T + ff * F * (h.abs() @ wd.abs().T)))}
    if dy is None:
        return out
    dy = dy.double()
    dh = dy @ wd
    edh = d * F * (dy.abs() @ wd.abs())
    top = max(1.0, ALPHA) / 2
    dg, du = dh * by_g, dh * by_u
    edg = by_g.abs() * edh + (dh.abs() + edh) * (top * (u.abs() + 1 + eu) * eg + 1.1 * eu) + R * (
        dh.abs() * (u.abs() + 1) * 1.1)
    edu = by_u.abs() * edh + (dh.abs() + edh) * 1.1 * eg + R * du.abs()
    if act == moe.ACT_CLAMPED_GLU:
        edg = edg + near * dh.abs() * (LIMIT + 1) * 1.1
        edu = edu + near * dh.abs() * LIMIT
    edg, edu = edg + H * (dg.abs() + edg), edu + H * (du.abs() + edu)

    def product(a, ea, b, n):   # a b^T-like sums: a (error ea) against exact b
        v = a @ b
        return v, H * v.abs() + 1.01 * (ea @ b.abs() + n * F * (a.abs() @ b.abs()))

    dx = dg @ wg + du @ wu
    out["dx"] = (dx, H * dx.abs() + 1.01 * (edg @ wg.abs() + edu @ wu.abs() + 2 * ff * F * (
        dg.abs() @ wg.abs() + du.abs() @ wu.abs())))
    out["gate"] = product(dg.T, edg.T, x, T)
    out["up"] = product(du.T, edu.T, x, T)
    v = dy.T @ h
    out["down"] = (v, H * v.abs() + 1.01 * (dy.abs().T @ eh + T * F * (dy.abs().T @ h.abs())))
    return out


def glu_inputs(T, d, ff, act, seed=1):
    gen = gen_for(T, d, ff, act, seed)
    spread = 3.0 if act == moe.ACT_CLAMPED_GLU else 1.0
    x = rnd(gen, T, d)
    w = moe.GluWeights(rnd(gen, ff, d, scale=spread * d ** -0.5), rnd(gen, ff, d, scale=spread * d ** -0.5),
                       rnd(gen, d, ff, scale=ff ** -0.5))
    return x, w, rnd(gen, T, d)


SHAPES = [(1, 8, 8), (8, 96, 12288), (10, 13544, 72), (16, 72, 8000), (3, 6152, 4864), (1, 2048, 512), (2, 40, 24), (7, 64, 64), (8, 264, 136), (16, 2880, 328), (17, 64, 2880),
          (33, 136, 520), (64, 512, 72), (128, 256, 256), (129, 264, 1000), (300, 520, 392), (777, 1024, 512),
          (1500, 72, 2056), (20, 4096, 2048), (100, 2056, 4096), (250, 4104, 264)]


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_CLAMPED_GLU])
@pytest.mark.parametrize("T,d,ff", SHAPES)
def test_glu_forward(T, d, ff, act):
    x, w, _ = glu_inputs(T, d, ff, act)
    want, tol = glu64(x, w.gate, w.up, w.down, None, act)["y"]
    cfg = moe.glu_cfg(d, ff, act=act)
    for keep in (False, True):
        y = Guarded((T, d))
        ws = moe.glu_workspace(cfg, T)
        saved = moe.glu_saved(cfg, T) if keep else None
        got = moe.moe_glu_forward(cfg, x, w, saved=saved, y=y.t, ws=ws)
        assert moe.moe_device_status(ws)[0] == moe.MOE_OK
        close(got, want, tol, "y")
        y.check()


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_CLAMPED_GLU])
@pytest.mark.parametrize("T,d,ff", SHAPES)
def test_glu_backward(T, d, ff, act):
    x, w, dy = glu_inputs(T, d, ff, act)
    want = glu64(x, w.gate, w.up, w.down, dy, act)
    cfg = moe.glu_cfg(d, ff, act=act)
    ws, saved = moe.glu_workspace(cfg, T), moe.glu_saved(cfg, T)
    y = moe.moe_glu_forward(cfg, x, w, saved=saved, ws=ws)
    out = {"dx": Guarded((T, d)), "gate": Guarded((ff, d)), "up": Guarded((ff, d)), "down": Guarded((d, ff))}
    grads = moe.GluGrads(out["gate"].t, out["up"].t, out["down"].t)
    dx, got = moe.moe_glu_backward(cfg, x, w, saved, dy, dx=out["dx"].t, grads=grads, ws=ws)
    assert moe.moe_device_status(ws)[0] == moe.MOE_OK
    close(y, *want["y"], "y")
    for name, t in (("dx", dx), ("gate", got.gate), ("up", got.up), ("down", got.down)):
        close(t, *want[name], name)
        out[name].check()


@pytest.mark.parametrize("T,d,ff,act", [(8192, 256, 512, 0), (2060, 624, 344, 1), (2708, 632, 592, 0),
                                        (5000, 264, 136, 1), (4100, 520, 1032, 0)])
def test_glu_backward_of_many_tokens_on_few_weights(T, d, ff, act):
    """Weights of few tiles: units share the tokens of a tile's gradient.  The workspace
    starts as rubbish, is not left, and a second run gives the same bits."""
    x, w, dy = glu_inputs(T, d, ff, act)
    want = glu64(x, w.gate, w.up, w.down, dy, act)
    cfg = moe.glu_cfg(d, ff, act=act)
    saved = moe.glu_saved(cfg, T)
    moe.moe_glu_forward(cfg, x, w, saved=saved)
    ws = Guarded((moe.moe_glu_workspace_bytes(cfg, T),), torch.uint8)
    first = None
    for names in (("gate", "up", "down"), ("gate", "up", "down"), ("up",), ("down",)):
        ws.t.fill_(0xFF)
        grads = moe.GluGrads(*(torch.empty_like(getattr(w, n)) if n in names else None for n in ("gate", "up", "down")))
        dx, got = moe.moe_glu_backward(cfg, x, w, saved, dy, grads=grads, ws=ws.t)
        assert moe.moe_device_status(ws.t)[0] == moe.MOE_OK
        close(dx, *want["dx"], "dx")
        for n in names:
            close(getattr(got, n), *want[n], n)
        ws.check()
        if len(names) == 3:
            if first is not None:
                assert all(torch.equal(getattr(first, n), getattr(got, n)) for n in names)
            first = got


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_CLAMPED_GLU])
def test_glu_gradient_against_differences(act):
    """Directional derivatives of sum(dy * FFN) by central differences in 64 bits."""
    T, d, ff = 37, 72, 136
    x, w, dy = glu_inputs(T, d, ff, act, seed=5)
    want = glu64(x, w.gate, w.up, w.down, dy, act)
    cfg = moe.glu_cfg(d, ff, act=act)
    saved = moe.glu_saved(cfg, T)
    moe.moe_glu_forward(cfg, x, w, saved=saved)
    dx, g = moe.moe_glu_backward(cfg, x, w, saved, dy)
    args = [t.double() for t in (x, w.gate, w.up, w.down)]

    def loss(v):
        h, _, _ = act64(v[0] @ v[1].T, v[0] @ v[2].T, act)
        return ((h @ v[3].T) * dy.double()).sum()

    gen = gen_for(act, 77)
    for i, (name, got) in enumerate((("dx", dx), ("gate", g.gate), ("up", g.up), ("down", g.down))):
        v = torch.randn(args[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        eps = 1e-6
        plus, minus = list(args), list(args)
        plus[i], minus[i] = args[i] + eps * v, args[i] - eps * v
        diff = (loss(plus) - loss(minus)) / (2 * eps)
        along = (got.double() * v).sum()
        # the kernel's own bound along v, and the difference quotient's (the clamp's kink
        # within eps of a value, and cancellation 2^-52 / eps): 1e-5 of the terms
        tol = (want[name][1] * v.abs()).sum() + 1e-5 * (want[name][0] * v).abs().sum()
        assert abs(along - diff) <= tol, (name, float(along), float(diff), float(tol))


def test_glu_partial_gradients_and_empty_batch():
    T, d, ff = 50, 64, 136
    x, w, dy = glu_inputs(T, d, ff, 0)
    cfg = moe.glu_cfg(d, ff)
    saved = moe.glu_saved(cfg, T)
    moe.moe_glu_forward(cfg, x, w, saved=saved)
    dx, full = moe.moe_glu_backward(cfg, x, w, saved, dy)
    for names in (("gate",), ("up", "down"), ("down",), ()):
        part = moe.GluGrads(*(torch.empty_like(getattr(full, n)) if n in names else None
                              for n in ("gate", "up", "down")))
        dx2, got = moe.moe_glu_backward(cfg, x, w, saved, dy, grads=part)
        assert torch.equal(dx, dx2)
        for n in names:
            assert torch.equal(getattr(got, n), getattr(full, n))
    none, got = moe.moe_glu_backward(cfg, x, w, saved, dy, need_dx=False)
    assert none is None and torch.equal(got.up, full.up)
    e = x[:0]
    saved0 = moe.glu_saved(cfg, 0)
    assert moe.moe_glu_forward(cfg, e, w, saved=saved0).shape == (0, d)
    got = moe.GluGrads(*(torch.full_like(t, 3.0) for t in (w.gate, w.up, w.down)))
    moe.moe_glu_backward(cfg, e, w, saved0, e, grads=got)
    assert all((t == 0).all() for t in (got.gate, got.up, got.down))


@pytest.mark.parametrize("T", [5, 200])
def test_glu_rows_do_not_mix(T):
    """A row of infinities and one of NaN spoil themselves and, through the sums over the
    tokens, the weights' gradients, but no other row."""
    d, ff = 136, 264
    x, w, dy = glu_inputs(T, d, ff, 0, seed=3)
    cfg = moe.glu_cfg(d, ff)
    y0 = moe.moe_glu_forward(cfg, x, w)
    bad = x.clone()
    bad[1, 3] = float("inf")
    bad[3, 5] = float("nan")
    saved = moe.glu_saved(cfg, T)
    for sv in (None, saved):
        y1 = moe.moe_glu_forward(cfg, bad, w, saved=sv)
        keep = [i for i in range(T) if i not in (1, 3)]
        if sv is None:
            assert torch.equal(y1[keep], y0[keep])
        assert torch.isfinite(y1[keep]).all() and torch.isnan(y1[3]).all() and not torch.isfinite(y1[1]).any()
    dx, g = moe.moe_glu_backward(cfg, bad, w, saved, dy)
    assert torch.isfinite(dx[keep]).all() and torch.isnan(dx[3]).all()
    assert torch.isnan(g.gate).any()


def test_glu_clamped_nan_passes():
    d, ff = 64, 64
    x, w, _ = glu_inputs(4, d, ff, 1)
    x[2, 0] = float("nan")
    for sv in (None, moe.glu_saved(moe.glu_cfg(d, ff, act=1), 4)):
        y = moe.moe_glu_forward(moe.glu_cfg(d, ff, act=1), x, w, saved=sv)
        assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3]]).all()


@pytest.mark.parametrize("T,d", [(1, 2880), (130, 2880), (64, 8192)])
def test_glu_clamp_border_takes_the_exact_side(T, d):
    """Gate and up values within 1e-7 .. 1e-4 of the clamp's border, nearer than a truncating
    sum of d products resolves: the gradient passes exactly where the 64-bit value is inside."""
    gen = gen_for(T, d, 11)
    ff = 128
    x = rnd(gen, T, d)
    t = T // 2                      # the token whose values are placed
    x[t, :4] = torch.tensor([2.0 ** -4, 2.0 ** -11, 2.0 ** -18, 2.0 ** -25])
    w = {n: rnd(gen, ff, d, scale=0.3 * d ** -0.5) for n in ("gate", "up")}
    off = torch.logspace(-7, -4, ff // 2, dtype=torch.float64, device="cuda")
    target = LIMIT + torch.cat((off, -off))
    for n in w:
        m = w[n]
        # a first part of the sum close to the target, then ever finer corrections
        m[:, 4:] = (m[:, 4:].double() + (target - x[t, 4:].double() @ m[:, 4:].double().T)[:, None] * x[t, 4:].double()
                    / x[t, 4:].double().square().sum()).bfloat16()
        m[:, :4] = 0
        for j in range(4):
            m[:, j] = ((target - m.double() @ x[t].double()) / x[t, j].double()).bfloat16()
    value = {n: w[n].double() @ x[t].double() for n in w}
    assert all(((v - LIMIT).abs() < 2e-4).all() for v in value.values())
    inside = {n: value[n].float().double() <= LIMIT for n in w}
    assert all(i.any() and not i.all() for i in inside.values())
    cfg = moe.glu_cfg(d, ff, act=moe.ACT_CLAMPED_GLU)
    weights = moe.GluWeights(w["gate"], w["up"], rnd(gen, d, ff, scale=ff ** -0.5))
    saved = moe.glu_saved(cfg, T)
    moe.moe_glu_forward(cfg, x, weights, saved=saved)
    dy = torch.zeros_like(x)        # only the placed token has a gradient
    dy[t] = rnd(gen, d)
    _, g = moe.moe_glu_backward(cfg, x, weights, saved, dy)
    assert torch.equal(g.gate.abs().amax(1) > 0, inside["gate"])
    assert torch.equal(g.up.abs().amax(1) > 0, inside["up"])


def test_glu_repeats_bit_for_bit_and_in_a_graph():
    T, d, ff = 333, 520, 264
    x, w, dy = glu_inputs(T, d, ff, 0, seed=9)
    cfg = moe.glu_cfg(d, ff)
    ws, saved = moe.glu_workspace(cfg, T), moe.glu_saved(cfg, T)
    fwd = moe.bind_glu_forward(cfg, x, w, saved=saved, ws=ws)
    bwd = moe.bind_glu_backward(cfg, x, w, saved, dy, ws=ws)
    y = fwd().clone()
    dx, g = bwd()
    first = [t.clone() for t in (dx, g.gate, g.up, g.down)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        fwd(), bwd()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        yg = fwd()
        dxg, gg = bwd()
    for t in (yg, dxg, gg.gate, gg.up, gg.down):
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(yg, y)
    for a, b in zip((dxg, gg.gate, gg.up, gg.down), first):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,d,ff", [(64, 2048, 256), (300, 256, 2048), (700, 512, 1024)])
def test_glu_wait_gives_up_reports_timeout_and_recovers(T, d, ff):
    """A load that is never issued (the test hook) runs the bounded waits out: the call reports
    MOE_ERR_TIMEOUT, and the next one is right.  Split tiles, pairs and many tiles."""
    x, w, dy = glu_inputs(T, d, ff, 0)
    cfg = moe.glu_cfg(d, ff)
    ws, saved = moe.glu_workspace(cfg, T), moe.glu_saved(cfg, T)
    want = glu64(x, w.gate, w.up, w.down, dy, 0)
    for backward in (False, True):
        moe.moe_glu_forward(cfg, x, w, saved=saved, ws=ws)
        assert moe.moe_device_status(ws)[0] == moe.MOE_OK
        try:
            moe.moe_test_set_wait_limit(1 << 14, True)
            if backward:
                moe.moe_glu_backward(cfg, x, w, saved, dy, ws=ws)
            else:
                moe.moe_glu_forward(cfg, x, w, ws=ws)
            status, bits = moe.moe_device_status(ws)
        finally:
            moe.moe_test_set_wait_limit(moe.DEFAULT_WAIT_POLLS, False)
        assert status == -7 and bits & (1 << 8), (status, bits)
    y = moe.moe_glu_forward(cfg, x, w, saved=saved, ws=ws)
    dx, g = moe.moe_glu_backward(cfg, x, w, saved, dy, ws=ws)
    assert moe.moe_device_status(ws)[0] == moe.MOE_OK
    for name, t in (("y", y), ("dx", dx), ("gate", g.gate), ("up", g.up), ("down", g.down)):
        close(t, *want[name], name)


# ----------------------------------------------------------------------------- norms
EPS = 1e-6


def norm64(x, z, post, gate, pre, dy, da, rs, bs):
    """Plain formulas and bounds in 64 bits."""
    x = x.double()
    d = x.shape[1]
    sg = None if gate is None else torch.sigmoid(gate.double())[:, None]
    c = bs if sg is None else bs * sg
    rz = 1.0
    if z is not None:
        z = z.double()
        if post is not None:
            rz = (z.square().mean(1, keepdim=True) + EPS).rsqrt()
            p = z * rz * post.double()
        else:
            p = z
        y = rs * x + c * p
        ey = R * ((rs * x).abs() + (c * p).abs())
    else:
        y, ey = x, 0 * x
    out = {}
    if z is not None:
        out["y"] = (y, H * y.abs() + 1.01 * ey)
    ry = (y.square().mean(1, keepdim=True) + EPS).rsqrt()
    ery = ry ** 3 * (y.abs() * ey).mean(1, keepdim=True) * 1.1 + R * ry
    if pre is not None:
        pre = pre.double()
        a = y * ry * pre
        ea = (ey * ry + y.abs() * ery) * pre.abs() + R * a.abs()
        out["a"] = (a, H * a.abs() + 1.01 * ea)
    if dy is None and da is None:
        return out
    D = torch.zeros_like(x) if dy is None else dy.double()
    eD = R * D.abs()
    if pre is not None:
        v = torch.zeros_like(x) if da is None else da.double()
        q = v * pre
        m = (q * y).mean(1, keepdim=True)
        em = (q.abs() * ey).mean(1, keepdim=True) + d * F * (q * y).abs().mean(1, keepdim=True)
        D = D + ry * (q - y * ry ** 2 * m)
        eD = eD + (ery + R * ry) * (q.abs() + 3 * y.abs() * ry ** 2 * m.abs()) + ry ** 3 * (ey * m.abs() + y.abs() * em)
        t = v * y * ry
        et = v.abs() * (ey * ry + y.abs() * ery)
        out["dpre_w"] = (t.sum(0), 1.01 * (et.sum(0) + x.shape[0] * F * t.abs().sum(0)) + R * t.abs().sum(0))
    f = rs if z is not None else 1.0
    out["dx"] = (f * D, H * (f * D).abs() + 1.01 * abs(f) * eD)
    if z is not None:
        dp, edp = c * D, abs(bs) * eD + R * (c * D).abs()
        if gate is not None:
            k = bs * (sg * (1 - sg))[:, 0]
            s = (D * p).sum(1)
            out["dgate"] = (k * s, 1.01 * (k.abs() + 1e-7) * ((eD * p.abs()).sum(1) + (d * F + R) * (D * p).abs().sum(1)))
        if post is not None:
            w = post.double()
            t = dp * z * rz
            out["dpost_w"] = (t.sum(0), 1.01 * ((edp * (z * rz).abs()).sum(0) + (x.shape[0] * F + R) * t.abs().sum(0)))
            q = dp * w
            m = (q * z).mean(1, keepdim=True)
            em = (edp * (w * z).abs()).mean(1, keepdim=True) + (d * F + R) * (q * z).abs().mean(1, keepdim=True)
            dz = rz * (q - z * rz ** 2 * m)
            edz = rz * (edp * w.abs() + R * q.abs()) + z.abs() * rz ** 3 * (em + R * m.abs())
        else:
            dz, edz = dp, edp
        out["dbranch"] = (dz, H * dz.abs() + 1.01 * edz)
    return out


PARTS = {"pre": (0, 0, 0, 1), "post": (1, 1, 0, 0), "plain": (1, 0, 0, 0), "gated": (1, 0, 1, 0),
         "gated pre": (1, 0, 1, 1), "all": (1, 1, 1, 1), "post pre": (1, 1, 0, 1)}
NORM_SHAPES = [(1, 8), (1, 2048), (3, 40), (8, 2880), (33, 264), (2, 16384), (700, 2048), (400, 4104), (1000, 8200),
               (5000, 256)]


def norm_inputs(T, d, parts, seed=0):
    gen = gen_for(T, d, *parts, seed)
    z, post, gate, pre = parts
    return dict(x=rnd(gen, T, d, scale=4.0), branch=rnd(gen, T, d) if z else None,
                post_w=(1 + rnd(gen, d, scale=0.2).float()).bfloat16() if post else None,
                gate=rnd(gen, T, dtype=torch.float32) if gate else None,
                pre_w=(1 + rnd(gen, d, scale=0.2).float()).bfloat16() if pre else None), gen


@pytest.mark.parametrize("which", PARTS)
@pytest.mark.parametrize("T,d", NORM_SHAPES)
def test_block_norm(T, d, which):
    parts = PARTS[which]
    i, gen = norm_inputs(T, d, parts)
    rs, bs = 0.9, -0.7
    cfg = moe.norm_cfg(d, eps=EPS, residual_scale=rs, branch_scale=bs)
    dy = rnd(gen, T, d) if parts[0] else None
    da = rnd(gen, T, d) if parts[3] else None
    want = norm64(i["x"], i["branch"], i["post_w"], i["gate"], i["pre_w"], dy, da, rs, bs)
    y = Guarded((T, d)) if parts[0] else None
    a = Guarded((T, d)) if parts[3] else None
    gy, ga = moe.moe_block_norm_forward(cfg, **i, y=y and y.t, a=a and a.t)
    g = moe.moe_block_norm_backward(cfg, i["x"], dy=dy, da=da, **{k: v for k, v in i.items() if k != "x"})
    got = {"y": gy, "a": ga, "dx": g.dx, "dbranch": g.dbranch, "dgate": g.dgate, "dpost_w": g.dpost_w,
           "dpre_w": g.dpre_w}
    assert {k for k, v in got.items() if v is not None} == set(want)
    for name, (v, tol) in want.items():
        close(got[name], v, tol, name)
    for o in (y, a):
        if o:
            o.check()


@pytest.mark.parametrize("given", ["dy", "da"])
def test_block_norm_backward_one_gradient(given):
    T, d = 21, 520
    i, gen = norm_inputs(T, d, PARTS["all"], seed=4)
    v = rnd(gen, T, d)
    cfg = moe.norm_cfg(d, eps=EPS, residual_scale=0.5, branch_scale=2.0)
    want = norm64(i["x"], i["branch"], i["post_w"], i["gate"], i["pre_w"], v if given == "dy" else None,
                  v if given == "da" else None, 0.5, 2.0)
    g = moe.moe_block_norm_backward(cfg, i["x"], **{given: v}, **{k: t for k, t in i.items() if k != "x"})
    for name in ("dx", "dbranch", "dgate", "dpost_w", "dpre_w"):
        close(getattr(g, name), *want[name], name)


def test_block_norm_gradient_against_differences():
    T, d = 9, 136
    i, gen = norm_inputs(T, d, PARTS["all"], seed=6)
    dy, da = rnd(gen, T, d), rnd(gen, T, d)
    rs, bs = 0.8, 1.3
    cfg = moe.norm_cfg(d, eps=EPS, residual_scale=rs, branch_scale=bs)
    want = norm64(i["x"], i["branch"], i["post_w"], i["gate"], i["pre_w"], dy, da, rs, bs)
    g = moe.moe_block_norm_backward(cfg, i["x"], dy=dy, da=da, **{k: t for k, t in i.items() if k != "x"})
    names = ("x", "branch", "gate", "post_w", "pre_w")
    args = {n: i[n].double() for n in names}

    def loss(v):
        z = v["branch"]
        p = z * (z.square().mean(1, keepdim=True) + EPS).rsqrt() * v["post_w"]
        y = rs * v["x"] + bs * torch.sigmoid(v["gate"])[:, None] * p
        a = y * (y.square().mean(1, keepdim=True) + EPS).rsqrt() * v["pre_w"]
        return (y * dy.double()).sum() + (a * da.double()).sum()

    for n in names:
        v = torch.randn(args[n].shape, generator=gen, device="cuda", dtype=torch.float64)
        eps = 1e-6
        diff = (loss({**args, n: args[n] + eps * v}) - loss({**args, n: args[n] - eps * v})) / (2 * eps)
        value, bound = want["d" + n]
        along = (getattr(g, "d" + n).double() * v).sum()
        tol = (bound * v.abs()).sum() + 1e-5 * (value * v).abs().sum()
        assert abs(along - diff) <= tol, (n, float(along), float(diff))


def test_block_norm_edges():
    """Rows of zeros, a row of NaN among others, a gate of either infinity, in-place use and
    an empty batch."""
    T, d = 12, 264
    i, gen = norm_inputs(T, d, PARTS["all"], seed=8)
    cfg = moe.norm_cfg(d, eps=EPS)
    i["x"][2] = 0
    i["branch"][2] = 0
    i["branch"][4, 7] = float("nan")
    i["gate"][5], i["gate"][6] = float("inf"), float("-inf")
    y, a = moe.moe_block_norm_forward(cfg, **i)
    assert (y[2] == 0).all() and (a[2] == 0).all()
    assert torch.isnan(y[4]).all() and torch.isnan(a[4]).all()
    rest = [t for t in range(T) if t != 4]
    assert torch.isfinite(y[rest]).all() and torch.isfinite(a[rest]).all()
    assert torch.equal(y[6], i["x"][6])
    dy, da = rnd(gen, T, d), rnd(gen, T, d)
    g = moe.moe_block_norm_backward(cfg, i["x"], dy=dy, da=da, **{k: t for k, t in i.items() if k != "x"})
    assert torch.isfinite(g.dx[rest]).all() and torch.isfinite(g.dbranch[rest]).all()
    assert (g.dgate[[5, 6]] == 0).all() and torch.isnan(g.dx[4]).all() and torch.isnan(g.dpost_w).all()
    # in place
    x2, z2, dy2, da2 = (t.clone() for t in (i["x"], i["branch"], dy, da))
    parts = dict(post_w=i["post_w"], gate=i["gate"], pre_w=i["pre_w"])
    grads = moe.NormGrads(dy2, da2)
    moe.moe_block_norm_backward(cfg, x2, dy=dy2, da=da2, branch=z2, grads=grads, **parts)
    assert torch.equal(dy2[rest], g.dx[rest]) and torch.equal(da2[rest], g.dbranch[rest])
    moe.moe_block_norm_forward(cfg, x2, branch=z2, y=x2, a=z2, **parts)
    assert torch.equal(x2[rest], y[rest]) and torch.equal(z2[rest], a[rest])
    e = i["x"][:0]
    g = moe.NormGrads(dpre_w=torch.full((d,), 5.0, device="cuda"))
    moe.moe_block_norm_backward(cfg, e, da=e, pre_w=i["pre_w"], grads=g)
    assert (g.dpre_w == 0).all()


def test_block_norm_backward_repeats_bit_for_bit():
    T, d = 3000, 512
    i, gen = norm_inputs(T, d, PARTS["all"], seed=2)
    dy, da = rnd(gen, T, d), rnd(gen, T, d)
    call = moe.bind_block_norm_backward(moe.norm_cfg(d), i["x"], dy=dy, da=da,
                                        **{k: t for k, t in i.items() if k != "x"})
    first = [t.clone() for t in vars(call()).values()]
    assert all(torch.equal(a, b) for a, b in zip(first, vars(call()).values()))


# ----------------------------------------------------------------------------- 4-bit linear
def w4_inputs(T, k, rows, group, zeros, seed=0):
    gen = gen_for(T, k, rows, group, zeros, seed)
    w = moe.W4Weights(torch.randint(0, 256, (rows, k // 2), generator=gen, device="cuda", dtype=torch.uint8),
                      rnd(gen, rows, k // group, scale=0.2 * k ** -0.5),
                      torch.randint(0, 16, (rows, k // group), generator=gen, device="cuda",
                                    dtype=torch.uint8) if zeros else None)
    return rnd(gen, T, k), w


def w4_64(x, w, group):
    q = torch.stack((w.codes & 15, w.codes >> 4), 2).reshape(w.codes.shape[0], -1, group).double()
    q = q - (8.0 if w.zeros is None else w.zeros.double()[:, :, None])
    m = (q * w.scales.double()[:, :, None]).reshape(q.shape[0], -1)
    return x.double() @ m.T, x.shape[1] * F * (x.double().abs() @ m.abs().T)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,k,n,group", [
    (1, 128, 1, 128), (1, 32, 16, 32), (3, 96, 17, 32), (8, 192, 40, 64), (5, 2048, 1000, 128), (9, 4096, 77, 64),
    (16, 8192, 130, 32), (16, 128 * 9, 2500, 128), (17, 320, 33, 32), (40, 576, 50, 64), (7, 13824, 70, 64),
    (12, 14336, 40, 128), (16, 4096, 6000, 64)])
def test_w4_linear(T, k, n, group, zeros):
    x, w = w4_inputs(T, k, n, group, zeros)
    want, e = w4_64(x, w, group)
    y = Guarded((T, n))
    moe.moe_w4_linear(moe.w4_cfg(k, n, group), x, w, y=y.t)
    close(y.t, want, H * want.abs() + 1.01 * e, "y")
    y.check()


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_CLAMPED_GLU])
@pytest.mark.parametrize("T,k,n,group", [(1, 2048, 512, 128), (4, 64, 3, 32), (8, 448, 100, 64), (13, 1024, 300, 128)])
def test_w4_linear_glu(T, k, n, group, act):
    x, w = w4_inputs(T, k, 2 * n, group, True, seed=act)
    v, e = w4_64(x, w, group)
    g, u, eg, eu = v[:, :n], v[:, n:], e[:, :n], e[:, n:]
    want, _, _ = act64(g, u, act)
    tol = H * want.abs() + 1.01 * (1.1 * (u.abs() + 1 + eu) * eg + (g.abs() + eg) * eu + R * want.abs())
    y = moe.moe_w4_linear(moe.w4_cfg(k, n, group, glu=True, act=act), x, w)
    close(y, want, tol, "y")


def test_w4_rows_do_not_mix_and_high_zero_bits():
    x, w = w4_inputs(6, 256, 40, 64, True)
    cfg = moe.w4_cfg(256, 40, 64)
    y = moe.moe_w4_linear(cfg, x, w)
    bad = x.clone()
    bad[2, 0] = float("nan")
    z = moe.moe_w4_linear(cfg, bad, w)
    assert torch.isnan(z[2]).all() and torch.equal(z[[0, 1, 3, 4, 5]], y[[0, 1, 3, 4, 5]])
    high = moe.W4Weights(w.codes, w.scales, w.zeros | 0xF0)   # only the low four bits count
    assert torch.equal(moe.moe_w4_linear(cfg, x, high), y)
    assert moe.moe_w4_linear(cfg, x[:0], w).shape == (0, 40)


def test_other_streams():
    """Calls on a stream of their own, ordered by events, and a bound call that follows
    torch's current stream."""
    x, w = w4_inputs(4, 512, 96, 128, False)
    cfg = moe.w4_cfg(512, 96)
    want = moe.moe_w4_linear(cfg, x, w)
    call = moe.bind_w4_linear(cfg, x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    other = moe.moe_w4_linear(cfg, x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)


@pytest.mark.parametrize("change", ["cpu", "dtype", "shape", "stride", "bytes"])
def test_binding_refuses(change):
    x, w, dy = glu_inputs(4, 64, 128, 0)
    cfg = moe.glu_cfg(64, 128)
    kw = {}
    if change == "cpu":
        w = moe.GluWeights(w.gate.cpu(), w.up, w.down)
    elif change == "dtype":
        x = x.float()
    elif change == "shape":
        w = moe.GluWeights(w.gate, w.up[:64], w.down)
    elif change == "stride":
        w = moe.GluWeights(w.gate, w.up, w.gate.t())
    else:
        kw = dict(ws=torch.empty(1 << 20, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_glu_forward(cfg, x, w, **kw)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.moe_glu_forward(cfg, *glu_inputs(4, 64, 128, 0)[:2], ws=small)
    assert e.value.status == -3
