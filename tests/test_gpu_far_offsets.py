"""Tensors of more than 2^31 elements: rows on either side of what 32 bits address."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_gpu_block import F, H, R, close, gen_for, norm64, rnd  # noqa: E402
from test_gpu_exchange import sums64 as row_sums64  # noqa: E402
from test_gpu_linear import lin64, quant_close, slope64, sums64  # noqa: E402

pytestmark = pytest.mark.gpu


def some(T, gen, n=200):
    """Rows from all over, the first and the last ones among them."""
    t = torch.randint(0, T, (n,), generator=gen, device="cuda")
    return torch.cat((t, torch.tensor([0, T // 2, T - 2, T - 1], device="cuda")))


def test_exchange():
    T, d, E, k = 300000, 2048, 40, 4                     # 2.46e9 elements of sorted rows
    gen = gen_for(T)
    ids = torch.randint(-1, E, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    x, w = rnd(gen, T, d), rnd(gen, T, k, dtype=torch.float32)
    cfg = moe.exchange_cfg(d, E, k)
    sent = moe.moe_dispatch_forward(cfg, x, ids)
    live = ids >= 0
    assert int(sent.offsets[-1]) == int(live.sum()) and (sent.rows[~live] == -1).all()
    flat = ids.reshape(-1)
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)[:int(live.sum())]
    assert torch.equal(sent.rows.reshape(-1)[order], torch.arange(order.numel(), dtype=torch.int32, device="cuda"))
    t = some(T, gen)
    rows, at = sent.rows[t], sent.rows[t].long().clamp(min=0)
    assert torch.equal(sent.xs[at][live[t]], x[t][:, None].expand(-1, k, -1)[live[t]])
    y = moe.moe_combine_forward(cfg, sent.xs, sent.rows, w=w, residual=x)
    want, mag = row_sums64(sent.xs[at].reshape(-1, d), torch.where(rows < 0, -1, torch.arange(rows.numel(), device="cuda").reshape(rows.shape).int()),
                           w[t], x[t])
    close(y[t], want, H * want.abs() + 1.01 * (k + 1) * F * mag, "y")
    dz, dw = moe.moe_combine_backward(cfg, x, sent.xs, sent.rows, w)
    terms = x[t].double().square()
    close(dw[t], torch.where(live[t], terms.sum(1, keepdim=True), 0.0), d * F * terms.sum(1, keepdim=True).expand(-1, k), "dw")
    want = w[t].double()[:, :, None] * x[t].double()[:, None]
    close(dz[at][live[t]], want[live[t]], (H * (1 + H) * want.abs() + 1e-40)[live[t]], "dz")


def test_norm_in_8_bits():
    T, d = 600000, 4096                                  # 2.46e9 elements
    gen = gen_for(T, d)
    x, z, pre = rnd(gen, T, d), rnd(gen, T, d), rnd(gen, d)
    y, q, scale = moe.moe_block_norm_quant(moe.norm_cfg(d), x, branch=z, pre_w=pre)
    t = some(T, gen, 60)
    out = norm64(x[t], z[t], None, None, pre, None, None, 1.0, 1.0)
    close(y[t], *out["y"], "y")
    a, ea = out["a"]
    quant_close(q[t], scale[t], a, ea - H * a.abs())


def test_linear_layer():
    T, k, n = 1100000, 64, 2048                          # 2.25e9 elements of y, pre, dy
    gen = gen_for(T, n)
    x, w = rnd(gen, T, k), moe.LinearWeights(rnd(gen, n, k, scale=0.25), rnd(gen, n))
    cfg = moe.linear_cfg(k, n, act=moe.LINEAR_SILU)
    pre = moe.linear_pre(cfg, T)
    dy = rnd(gen, T, n)
    y = moe.moe_linear_forward(cfg, x, w, residual=dy, pre=pre)
    t = some(T, gen)
    v, e = sums64(x[t], w.w, None, None, w.bias)
    close(pre[t], v, H * v.abs() + 1.01 * e, "pre")
    want = lin64(v, moe.LINEAR_SILU) + dy[t].double()
    close(y[t], want, H * want.abs() + 1.01 * (1.13 * e + R * (want - dy[t].double()).abs() + F * want.abs()), "y")
    del y
    dx, g = moe.moe_linear_backward(cfg, x, w, dy, pre=pre)
    s, gy = slope64(pre[t].double(), moe.LINEAR_SILU), dy[t].double()
    dv = gy * s
    rdv = R * (dv.abs() + gy.abs())
    rdv = rdv + H * (dv.abs() + rdv)
    W = w.w.double()
    want = dv @ W
    close(dx[t], want, H * want.abs() + 1.01 * (rdv @ W.abs() + n * F * (dv.abs() @ W.abs())), "dx")
    total, mag, off, dw, edw = 0.0, 0.0, 0.0, 0.0, 0.0
    for a in range(0, T, 50000):
        gy = dy[a:a + 50000].double()
        dv = gy * slope64(pre[a:a + 50000].double(), moe.LINEAR_SILU)
        e = R * (dv.abs() + gy.abs())
        total, mag, off = total + dv.sum(0), mag + dv.abs().sum(0), off + e.sum(0)
        X = x[a:a + 50000].double()
        dw, edw = dw + dv.T @ X, edw + (e + H * (dv.abs() + e)).T @ X.abs()
    close(g.bias, total, H * total.abs() + 1.01 * (off + 4096 * F * mag), "dbias")
    close(g.w, dw, H * dw.abs() + 1.01 * (edw + 4096 * F * edw / H), "dw")
