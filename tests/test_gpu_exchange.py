"""The exchange (moe_exchange.h) against plain implementations in 64 bits.

The sort and the copies are exact.  A sum of k products in fp32 is off by at most (k + 1) 2^-23 of
the sum of their magnitudes, its rounding to bf16 by half a step, 2^-8 of its value (H); a product
in fp32 rounded to bf16 by H (1 + 2^-8)."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_gpu_block import F, H, Guarded, close, gen_for, rnd  # noqa: E402

pytestmark = pytest.mark.gpu


def routing(gen, T, E, k, bad=0.0):
    """topk ids (of a token distinct); `bad`: that share of them outside [0, E)."""
    ids = (torch.rand(T, E, generator=gen, device="cuda") ** (1 + torch.arange(E, device="cuda") % 3)).topk(k, 1).indices.int()
    if bad:
        out = torch.rand(T, k, generator=gen, device="cuda") < bad
        odd = torch.tensor([-1, E, -(1 << 31), (1 << 31) - 1], dtype=torch.int32, device="cuda")
        ids = torch.where(out, odd[torch.randint(0, 4, (T, k), generator=gen, device="cuda")], ids)
    return ids


def sort_plain(ids, E):
    """offsets, rows and the slots' order, on the host."""
    flat = ids.reshape(-1).tolist()
    order = sorted((s for s in range(len(flat)) if 0 <= flat[s] < E), key=lambda s: (flat[s], s))
    rows = [-1] * len(flat)
    for r, s in enumerate(order):
        rows[s] = r
    count = [0] * E
    for v in flat:
        if 0 <= v < E:
            count[v] += 1
    offsets, n = [0], 0
    for c in count:
        n += c
        offsets.append(n)
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(rows, dtype=torch.int32).reshape(ids.shape), order


SHAPES = [(1, 8, 1, 1), (1, 16, 256, 8), (3, 24, 5, 5), (8, 2048, 256, 8), (7, 1032, 32, 4), (65, 256, 3, 2),
          (255, 8, 1024, 8), (257, 40, 17, 8), (300, 2880, 32, 4), (1025, 72, 64, 2), (2049, 136, 1, 1), (700, 520, 40, 32),
          (40000, 8, 9, 7)]


@pytest.mark.parametrize("bad", [0.0, 0.3])
@pytest.mark.parametrize("T,d,E,k", SHAPES)
def test_dispatch(T, d, E, k, bad):
    gen = gen_for(T, d, E, k)
    ids, x = routing(gen, T, E, k, bad), rnd(gen, T, d)
    offsets, rows, order = sort_plain(ids, E)
    cfg = moe.exchange_cfg(d, E, k)
    o, r, xs = Guarded((E + 1,), torch.int32), Guarded((T, k), torch.int32), Guarded((T * k, d))
    ws = Guarded((moe.moe_dispatch_workspace_bytes(cfg, T),), torch.uint8)
    before = xs.t.clone()
    moe.moe_dispatch_forward(cfg, x, ids, out=moe.Dispatched(o.t, r.t, xs.t), ws=ws.t)
    assert torch.equal(o.t.cpu(), offsets) and torch.equal(r.t.cpu(), rows)
    n = len(order)
    token = torch.tensor(order, dtype=torch.long, device="cuda") // k
    assert torch.equal(xs.t[:n], x[token])
    assert torch.equal(xs.t[n:].view(torch.int16), before[n:].view(torch.int16))   # rows behind the last: untouched
    for b in (o, r, xs, ws):
        b.check()
    # the sort alone gives the same
    alone = moe.moe_dispatch_forward(cfg, None, ids)
    assert alone.xs is None and torch.equal(alone.rows, r.t) and torch.equal(alone.offsets, o.t)


@pytest.mark.parametrize("T,d,E,k", [(1, 16, 4, 2), (8, 2048, 256, 8), (33, 2880, 32, 4), (1000, 48, 7, 3), (5, 16, 2, 1),
                                     (9000, 32, 40, 1)])
def test_dispatch_8_bits(T, d, E, k):
    gen = gen_for(T, d, E, k, 8)
    ids = routing(gen, T, E, k, 0.1)
    x, scale = moe.w8_quantize(rnd(gen, T, d))
    out = moe.moe_dispatch_forward(moe.exchange_cfg(d, E, k, fmt=moe.ROWS_E4M3), x, ids, x_scale=scale)
    _, rows, order = sort_plain(ids, E)
    token = torch.tensor(order, dtype=torch.long, device="cuda") // k
    assert torch.equal(out.rows.cpu(), rows)
    assert torch.equal(out.xs.view(torch.uint8)[:len(order)], x.view(torch.uint8)[token])
    assert torch.equal(out.xs_scale[:len(order)], scale[token])


def test_dispatch_agrees_with_group_by_expert():
    gen = gen_for(5)
    for T in (64, 3000):
        ids = routing(gen, T, 256, 8)
        _, offsets, perm = moe.moe_group_by_expert(moe.qwen_cfg(), ids)
        out = moe.moe_dispatch_forward(moe.exchange_cfg(2048, 256, 8), None, ids)
        assert torch.equal(out.offsets, offsets)
        assert torch.equal(out.rows.reshape(-1)[perm.long()], torch.arange(8 * T, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("T", [5, 300, 5000, 150000])
def test_the_same_expert_twice_and_all_tokens_to_one(T):
    """Slots of one token that name the same expert keep their order; an expert may take all."""
    cfg = moe.exchange_cfg(64, 6, 3)
    ids = torch.full((T, 3), 4, dtype=torch.int32, device="cuda")
    out = moe.moe_dispatch_forward(cfg, None, ids)
    assert torch.equal(out.rows.reshape(-1), torch.arange(3 * T, dtype=torch.int32, device="cuda"))
    assert out.offsets.tolist() == [0, 0, 0, 0, 0, 3 * T, 3 * T]
    none = moe.moe_dispatch_forward(cfg, None, torch.full((T, 3), -1, dtype=torch.int32, device="cuda"))
    assert (none.rows == -1).all() and (none.offsets == 0).all()


def sums64(z, rows, w, residual):
    """y and the sum of magnitudes."""
    at = rows.long().clamp(min=0)
    live = (rows >= 0)[:, :, None]
    t = torch.where(live, z.double()[at] * (1.0 if w is None else w.double()[:, :, None]), 0.0)
    y, mag = t.sum(1), t.abs().sum(1)
    if residual is not None:
        y, mag = y + residual.double(), mag + residual.double().abs()
    return y, mag


@pytest.mark.parametrize("T,d,E,k", SHAPES)
def test_combine_and_gradients(T, d, E, k):
    gen = gen_for(T, d, E, k, 1)
    ids = routing(gen, T, E, k, 0.2)
    cfg = moe.exchange_cfg(d, E, k)
    rows = moe.moe_dispatch_forward(cfg, None, ids).rows
    z, w, residual, dy = rnd(gen, T * k, d), rnd(gen, T, k, dtype=torch.float32), rnd(gen, T, d, scale=4.0), rnd(gen, T, d)
    n = int((rows >= 0).sum())
    z[n:] = float("nan")          # rows without a slot are not read
    for weight, res in ((w, residual), (None, None), (w, None), (None, residual)):
        y = Guarded((T, d))
        moe.moe_combine_forward(cfg, z, rows, w=weight, residual=res, y=y.t)
        want, mag = sums64(z, rows, weight, res)
        close(y.t, want, H * want.abs() + 1.01 * (k + 1) * F * mag, "y")
        y.check()
    dx = moe.moe_dispatch_backward(cfg, z, rows)
    assert torch.equal(dx, moe.moe_combine_forward(cfg, z, rows))
    y = residual.clone()          # in place
    assert torch.equal(moe.moe_combine_forward(cfg, z, rows, w=w, residual=y, y=y),
                       moe.moe_combine_forward(cfg, z, rows, w=w, residual=residual))
    dz, dw = Guarded((T * k, d)), Guarded((T, k), torch.float32)
    before = dz.t.clone()
    moe.moe_combine_backward(cfg, dy, z, rows, w, dz=dz.t, dw=dw.t)
    live = rows >= 0
    at = rows.long()[live]
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)[live]
    want = w[live].double()[:, None] * dy[token].double()
    close(dz.t[at], want, H * (1 + H) * want.abs() + 1e-40, "dz")
    assert torch.equal(dz.t[n:].view(torch.int16), before[n:].view(torch.int16))
    terms = dy[token].double() * z[at].double()
    close(dw.t[live], terms.sum(1), d * F * terms.abs().sum(1), "dw")
    assert (dw.t[~live] == 0).all()
    dz.check()
    dw.check()
    # one of the two alone gives the same bits
    assert torch.equal(moe.moe_combine_backward(cfg, dy, None, rows, w, need_dw=False)[0][:n], dz.t[:n])
    assert torch.equal(moe.moe_combine_backward(cfg, dy, z, rows, w, need_dz=False)[1], dw.t)


# rows a token on both sides of each number of rows in flight; several tokens to a CTA and the last
# CTA not full (short rows), several CTAs to a row (few tokens, long rows), rows longer than a CTA
@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 8, 9, 12, 13])
@pytest.mark.parametrize("T,d", [(1, 8), (77, 40), (333, 520), (3, 16392), (700, 2056)])
def test_combine_rows_a_token(T, d, k):
    test_combine_and_gradients(T, d, 16, k)


def test_combine_gradient_against_differences():
    """Directional derivatives of sum(dy y) by central differences in 64 bits; y is linear in z and in
    w apart, so the quotient is exact but for a term of h^2."""
    T, d, E, k = 37, 136, 9, 4
    gen = gen_for(77)
    cfg = moe.exchange_cfg(d, E, k)
    ids = routing(gen, T, E, k, 0.1)
    x = rnd(gen, T, d)
    sent = moe.moe_dispatch_forward(cfg, x, ids)
    rows, n = sent.rows, int(sent.offsets[-1])
    z, w, dy = rnd(gen, T * k, d), rnd(gen, T, k, dtype=torch.float32), rnd(gen, T, d)
    dz, dw = moe.moe_combine_backward(cfg, dy, z, rows, w)
    vz, vw = rnd(gen, T * k, d).double(), rnd(gen, T, k).double()
    vz[n:] = 0
    h = 2.0 ** -10

    def loss(a, b):
        at, live = rows.long().clamp(min=0), (rows >= 0)[:, :, None]
        return (dy.double() * torch.where(live, b[:, :, None] * a[at], 0.0).sum(1)).sum()

    zd, wd = z.double(), w.double()
    num = (loss(zd + h * vz, wd + h * vw) - loss(zd - h * vz, wd - h * vw)) / (2 * h)
    live = rows >= 0
    got = (dz[:n].double() * vz[:n]).sum() + (dw.double() * vw)[live].sum()
    tol = H * 1.01 * (dz[:n].double() * vz[:n]).abs().sum() + d * F * ((dy.double().abs()[:, None] * z.double().abs()[rows.long().clamp(min=0)]).sum(2) * vw.abs())[live].sum()
    assert abs(got - num) <= tol + 1e-9 * abs(num)
    # dispatch: sum(dxs xs) along v
    dxs, v = rnd(gen, T * k, d), rnd(gen, T, d).double()
    dx = moe.moe_dispatch_backward(cfg, dxs, rows)
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)[live]
    num = (dxs.double()[rows.long()[live]] * v[token]).sum()
    assert abs((dx.double() * v).sum() - num) <= 1.01 * H * (dx.double() * v).abs().sum()


def test_rows_of_a_caller_out_of_range_are_passed_over():
    cfg = moe.exchange_cfg(32, 4, 2)
    gen = gen_for(3)
    z, w, dy = rnd(gen, 6, 32), rnd(gen, 3, 2, dtype=torch.float32), rnd(gen, 3, 32)
    rows = torch.tensor([[0, 6], [-7, 3], [1 << 30, -(1 << 31)]], dtype=torch.int32, device="cuda")
    ok = torch.tensor([[0, -1], [-1, 3], [-1, -1]], dtype=torch.int32, device="cuda")
    for a, b in zip(moe.moe_combine_backward(cfg, dy, z, rows, w, dz=torch.zeros_like(z)),
                    moe.moe_combine_backward(cfg, dy, z, ok, w, dz=torch.zeros_like(z))):
        assert torch.equal(a, b)
    assert torch.equal(moe.moe_combine_forward(cfg, z, rows, w), moe.moe_combine_forward(cfg, z, ok, w))
    assert (moe.moe_combine_forward(cfg, z, rows, w)[2] == 0).all()


def test_infinities_and_nan_stay_in_their_tokens():
    cfg = moe.exchange_cfg(64, 8, 2)
    gen = gen_for(11)
    ids = routing(gen, 40, 8, 2)
    rows = moe.moe_dispatch_forward(cfg, None, ids).rows
    z, w = rnd(gen, 80, 64), rnd(gen, 40, 2, dtype=torch.float32)
    clean = moe.moe_combine_forward(cfg, z, rows, w)
    z[rows[7, 1].long(), 3] = float("nan")
    z[rows[9, 0].long(), 5] = float("inf")
    w[9, 0] = 0.0
    got = moe.moe_combine_forward(cfg, z, rows, w)
    other = [t for t in range(40) if t not in (7, 9)]
    assert torch.equal(got[other], clean[other])
    assert torch.isnan(got[7]).tolist() == [i == 3 for i in range(64)]
    assert torch.isnan(got[9]).tolist() == [i == 5 for i in range(64)]   # 0 times infinity


def test_no_tokens():
    cfg = moe.exchange_cfg(64, 8, 2)
    x, ids = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    out = moe.moe_dispatch_forward(cfg, x, ids)
    assert (out.offsets == 0).all() and out.xs.shape == (0, 64)
    assert moe.moe_combine_forward(cfg, out.xs, out.rows, residual=x).shape == (0, 64)
    dz, dw = moe.moe_combine_backward(cfg, x, out.xs, out.rows, torch.empty(0, 2, device="cuda"))
    assert dz.shape == (0, 64) and dw.shape == (0, 2)


@pytest.mark.parametrize("T", [40, 600])
def test_captured_and_replayed_beside_eager_calls(T):
    """Two graphs with workspaces of their own, replayed on new routings in turn with eager calls."""
    d, E, k = 136, 16, 4
    cfg = moe.exchange_cfg(d, E, k)
    gen = gen_for(21)
    ids, x, w, dy = routing(gen, T, E, k), rnd(gen, T, d), rnd(gen, T, k, dtype=torch.float32), rnd(gen, T, d)

    def step():
        sent = moe.moe_dispatch_forward(cfg, x, ids)
        y = moe.moe_combine_forward(cfg, sent.xs, sent.rows, w=w, residual=x)
        dz, dw = moe.moe_combine_backward(cfg, dy, sent.xs, sent.rows, w)
        return sent.rows, y, dz, dw, moe.moe_dispatch_backward(cfg, dz, sent.rows)

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for turn in range(4):
        ids.copy_(routing(gen, T, E, k))
        x.copy_(rnd(gen, T, d))
        graphs[turn % 2].replay()
        want = step()
        for a, b in zip(outs[turn % 2], want):
            assert torch.equal(a, b)
