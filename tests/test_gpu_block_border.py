"""The clamp's border for limits and operands of any size: the gradient passes exactly where
the 64-bit value lies inside, however large the terms whose sum it is."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")

pytestmark = pytest.mark.gpu

FF = 128


def operands(T, d, limit, kind, gen):
    """x, and gate and up weights whose values for token T // 2 lie 1e-7 .. 1e-4 times the
    terms' size either side of the border."""
    def rnd(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()

    x = rnd(T, d, scale=64.0 if kind == "large" else 1.0)
    t = T // 2                      # the token whose values are placed
    x[t, :4] = torch.tensor([2.0 ** -4, 2.0 ** -11, 2.0 ** -18, 2.0 ** -25])
    size = 1.0
    if kind == "cancelling":        # +-512 early, taken back at the end: partial sums of 512
        x[t, 4] = x[t, d - 1] = 1.0
        size = 16.0
    if kind == "large":
        size = 16.0
    off = size * torch.logspace(-7, -4, FF // 2, dtype=torch.float64, device="cuda")
    target = limit + torch.cat((off, -off))
    free = slice(5, d - 1)
    w = []
    for _ in range(2):
        m = rnd(FF, d, scale=0.3 * d ** -0.5)
        m[:, 4] = m[:, d - 1] = 0
        if kind == "cancelling":
            m[:, 4], m[:, d - 1] = 512.0, -512.0
        m[:, :4] = 0
        # a first part of the sum close to the target, then ever finer corrections
        xf = x[t, free].double()
        m[:, free] = (m[:, free].double() + (target - m[:, 4:].double() @ x[t, 4:].double())[:, None] * xf
                      / xf.square().sum()).bfloat16()
        for j in range(4):
            m[:, j] = ((target - m.double() @ x[t].double()) / x[t, j].double()).bfloat16()
        w.append(m)
    return x, w, t, size


@pytest.mark.parametrize("kind", ["plain", "cancelling", "large"])
@pytest.mark.parametrize("limit", [0.0, 0.05, 1.0, 7.0])
@pytest.mark.parametrize("T,d", [(1, 2880), (130, 2880), (64, 8192), (20, 72)])
def test_border_takes_the_exact_side(T, d, limit, kind):
    gen = torch.Generator(device="cuda").manual_seed(1000 * T + d + int(100 * limit) + len(kind))
    x, w, t, size = operands(T, d, limit, kind, gen)
    value = [m.double() @ x[t].double() for m in w]
    assert all(((v - limit).abs() < 4e-4 * size).all() for v in value)
    # a value nearer than fp32 resolves (the border's own step, and 2^-32 of the terms, which
    # is what a sum that keeps its roundings may lose) may take either side
    sure = [((v.abs() - limit).abs() > 2.0 ** -22 * limit + 2.0 ** -32 * 64 * size) for v in value]
    assert all(s.sum() > FF // 2 for s in sure)
    cfg = moe.glu_cfg(d, FF, act=moe.ACT_CLAMPED_GLU, glu_limit=limit)
    down = (torch.randn(d, FF, generator=gen, device="cuda") * FF ** -0.5).bfloat16()
    weights = moe.GluWeights(*w, down)
    ws, saved = moe.glu_workspace(cfg, T), moe.glu_saved(cfg, T)
    moe.moe_glu_forward(cfg, x, weights, saved=saved, ws=ws)
    dy = torch.zeros_like(x)        # only the placed token has a gradient
    dy[t] = torch.randn(d, generator=gen, device="cuda").bfloat16()
    _, g = moe.moe_glu_backward(cfg, x, weights, saved, dy, ws=ws)
    assert moe.moe_device_status(ws)[0] == moe.MOE_OK
    passes = [g.gate.abs().amax(1) > 0, g.up.abs().amax(1) > 0]
    inside = [value[0] <= limit, value[1].abs() <= limit]
    for name, p, i, s in zip(("gate", "up"), passes, inside, sure):
        assert torch.equal(p[s], i[s]), (name, int((p != i)[s].sum()))


@pytest.mark.parametrize("T", [1, 130])
@pytest.mark.parametrize("case", ["far", "beside infinity", "beside nan", "beside huge"])
def test_border_beside_rows_of_any_size(T, case):
    """Norms whose squares leave fp32's range, and features beside ones whose sums are not
    finite; the workspace is exactly as large as the library asks for."""
    d, limit = 2880, 7.0
    gen = torch.Generator(device="cuda").manual_seed(T + len(case))
    x, w, t, size = operands(T, d, limit, "plain", gen)
    keep = torch.ones(FF, dtype=torch.bool, device="cuda")
    if case == "far":               # exact powers of two: the values stay what they are
        x[t] *= 2.0 ** 90
        w = [m * 2.0 ** -90 for m in w]
    else:
        for f in (3, 40, 100):
            keep[f] = False
            for m in w:
                m[f, 100] = {"beside infinity": float("inf"), "beside nan": float("nan"), "beside huge": 1e37}[case]
    value = [m.double() @ x[t].double() for m in w]
    assert all(((v - limit).abs() < 4e-4 * size)[keep].all() for v in value)
    sure = [((v.abs() - limit).abs() > 2.0 ** -22 * limit + 2.0 ** -26 * size) & keep for v in value]
    cfg = moe.glu_cfg(d, FF, act=moe.ACT_CLAMPED_GLU, glu_limit=limit)
    weights = moe.GluWeights(*w, torch.ones(d, FF, device="cuda").bfloat16())
    n, pad = moe.moe_glu_workspace_bytes(cfg, T), 4096
    raw = torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    ws, saved = raw[pad:pad + n], moe.glu_saved(cfg, T)
    moe.moe_glu_forward(cfg, x, weights, saved=saved, ws=ws)
    dy = torch.zeros_like(x)
    dy[t] = torch.randn(d, generator=gen, device="cuda").bfloat16()
    _, g = moe.moe_glu_backward(cfg, x, weights, saved, dy, ws=ws)
    assert moe.moe_device_status(ws)[0] == moe.MOE_OK
    assert (raw[:pad] == 0xA5).all() and (raw[-pad:] == 0xA5).all()
    for m, v, s, limit_of in zip((g.gate, g.up), value, sure, (lambda v: v <= limit, lambda v: v.abs() <= limit)):
        assert torch.equal((m.abs().amax(1) > 0)[s], limit_of(v)[s])


def test_rows_of_zeros_at_a_limit_of_zero():
    """Padding tokens lie on the border of a limit of 0 exactly; nothing is to be settled there."""
    T, d = 700, 520
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    x[100:] = 0
    r = lambda *s: (torch.randn(s, generator=gen, device="cuda") * s[1] ** -0.5).bfloat16()   # noqa: E731
    w = moe.GluWeights(r(FF, d), r(FF, d), r(d, FF))
    cfg = moe.glu_cfg(d, FF, act=moe.ACT_CLAMPED_GLU, glu_limit=0.0)
    ws, saved = moe.glu_workspace(cfg, T), moe.glu_saved(cfg, T)
    y = moe.moe_glu_forward(cfg, x, w, saved=saved, ws=ws)
    dx, g = moe.moe_glu_backward(cfg, x, w, saved, torch.ones_like(x), ws=ws)
    assert moe.moe_device_status(ws)[0] == moe.MOE_OK
    assert (y[100:] == 0).all() and torch.isfinite(dx).all() and torch.isfinite(g.gate).all()
