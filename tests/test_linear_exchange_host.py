"""Host checks of the linear layer's and the exchange's entry points that need no GPU: sizes, refusals
before anything is enqueued, and the weights' quantiser."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from sparse_moe_ffn_route_gb300 import block, exchange, linear  # noqa: E402

OK, INVALID, UNSUPPORTED, WORKSPACE, ALIGNMENT = 0, -1, -2, -3, -4
# aligned addresses that are never read, far apart: every refusal comes before the first launch
A, B, C, D, E, G, I, J = (0x1000000000 * i for i in range(1, 9))
BIG = 1 << 40
L = moe._lib


def ref(s):
    return None if s is None else ctypes.byref(s)


def lin(**kw):
    c = moe.linear_cfg(64, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def forward(c, x=A, xs=None, T=4, w=(B, None, C), res=D, y=E, pre=None, ws=G, wb=BIG):
    return L.moe_linear_forward(ref(c), x, xs, T, None if w is None else ref(block._Three(*w)), res, y, pre, ws, wb, None)


def backward(c, x=A, T=4, w=(B, None, C), pre=None, dy=D, dx=E, g=(I, J), ws=G, wb=BIG):
    return L.moe_linear_backward(ref(c), x, T, None if w is None else ref(block._Three(*w)), pre, dy, dx,
                                 None if g is None else ref(linear._Two(*g)), ws, wb, None)


@pytest.mark.parametrize("change,code", [
    (dict(n_in=0), INVALID), (dict(n_out=-8), INVALID), (dict(format=2), INVALID), (dict(format=-1), INVALID),
    (dict(glu=2), INVALID), (dict(act=4), INVALID), (dict(act=-1), INVALID), (dict(glu=1, act=2), INVALID),
    (dict(glu_limit=float("nan")), INVALID), (dict(glu_limit=-1.0), INVALID), (dict(glu_alpha=float("inf")), INVALID),
    (dict(n_in=12), UNSUPPORTED), (dict(n_out=100), UNSUPPORTED), (dict(format=1, n_in=72), UNSUPPORTED),
    (dict(n_in=(1 << 29) + 8), UNSUPPORTED), (dict(n_out=(1 << 29) + 8), UNSUPPORTED),
    (dict(glu=1, n_out=(1 << 28) + 8), UNSUPPORTED)])
def test_linear_configurations_refused(change, code):
    c = lin(**change)
    assert forward(c) == code and backward(c) == code and forward(c, T=0) == code
    assert moe.moe_linear_workspace_bytes(c, 4) == 0
    with pytest.raises(moe.MoeError):
        moe.linear_workspace(c, 4, "cpu")


def test_linear_arguments_refused():
    c = lin()
    for i in range(5):
        bad = lin()
        bad.reserved[i] = 1
        assert forward(bad) == INVALID
    assert forward(None) == INVALID and backward(None) == INVALID
    assert forward(c, T=-1) == INVALID and forward(c, T=(1 << 30) + 1) == UNSUPPORTED
    assert forward(c, T=0, x=None, w=None, y=None, ws=None) == OK
    for kw in (dict(x=None), dict(w=None), dict(w=(None, None, C)), dict(y=None), dict(ws=None), dict(xs=I), dict(w=(B, I, C))):
        assert forward(c, **kw) == INVALID, kw
    e = lin(format=moe.LINEAR_E4M3)
    assert forward(e) == INVALID and forward(e, xs=I) == INVALID and forward(e, w=(B, J, C)) == INVALID
    assert forward(lin(glu=1), pre=I) == INVALID
    for kw in (dict(x=A + 8), dict(w=(B + 2, None, C)), dict(w=(B, None, C + 4)), dict(res=D + 8), dict(y=E + 8), dict(pre=I + 8),
               dict(ws=G + 8)):
        assert forward(c, **kw) == ALIGNMENT, kw
    assert forward(e, xs=I + 2, w=(B, J, C)) == ALIGNMENT and forward(e, xs=I, w=(B, J + 4, C)) == ALIGNMENT
    assert forward(c, wb=255) == WORKSPACE
    # shared memory: y with x, the weights, the bias, half of the residual, pre and the workspace
    for kw in (dict(y=A + 16), dict(y=B), dict(y=C), dict(y=D + 64), dict(pre=E + 16), dict(pre=D), dict(y=G + 16), dict(pre=A)):
        assert forward(c, **kw) == INVALID, kw


def test_linear_backward_arguments_refused():
    c, a = lin(), lin(act=1)
    assert backward(lin(glu=1)) == UNSUPPORTED and backward(lin(format=1)) == UNSUPPORTED
    assert backward(c, T=-1) == INVALID and backward(c, T=(1 << 30) + 1) == UNSUPPORTED
    for kw in (dict(x=None), dict(w=None), dict(w=(None, None, None)), dict(dy=None), dict(ws=None)):
        assert backward(c, **kw) == INVALID, kw
    assert backward(a) == INVALID            # an activation without pre
    for kw in (dict(x=A + 8), dict(w=(B + 2, None, None)), dict(pre=C + 8), dict(dy=D + 8), dict(dx=E + 8), dict(g=(I + 8, J)),
               dict(g=(I, J + 8)), dict(ws=G + 8)):
        assert backward(c, **kw) == ALIGNMENT, kw
    for k in (c, a):
        n = moe.moe_linear_workspace_bytes(k, 4)
        assert n >= 256 and backward(k, pre=C, wb=n - 1) == WORKSPACE
    for kw in (dict(dx=A), dict(dx=D + 16), dict(dx=B), dict(g=(A, J)), dict(g=(I, I + 32)), dict(g=(E, J)), dict(dx=G), dict(g=(I, D))):
        assert backward(c, **kw) == INVALID, kw
    assert backward(a, pre=C, dx=C) == INVALID


def test_linear_workspace_grows():
    c = lin(n_in=2048, n_out=2048, act=1)
    assert moe.moe_linear_workspace_bytes(c, 0) == 256
    assert 256 < moe.moe_linear_workspace_bytes(c, 100) < moe.moe_linear_workspace_bytes(c, 8192)
    assert moe.moe_linear_workspace_bytes(c, -1) == 0 and moe.moe_linear_workspace_bytes(c, (1 << 30) + 1) == 0
    assert moe.moe_linear_workspace_bytes(lin(format=1), 8192) == 256      # forward alone
    with pytest.raises(ValueError):
        moe.moe_linear_workspace_bytes(c, 1 << 31)


def quant(c, ins=(A, B, C, D, E), T=4, y=G, q=I, s=J):
    return L.moe_block_norm_quant(ref(c), None if ins is None else ref(block._Five(*ins)), T, y, q, s, None)


def test_norm_quant_refusals():
    c = moe.norm_cfg(64)
    for kw, code in ((dict(d_model=0), INVALID), (dict(d_model=12), UNSUPPORTED), (dict(d_model=16392), UNSUPPORTED),
                     (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(residual_scale=float("inf")), INVALID),
                     (dict(branch_scale=float("nan")), INVALID)):
        bad = moe.norm_cfg(64)
        for k, v in kw.items():
            setattr(bad, k, v)
        assert quant(bad) == code, kw
    bad = moe.norm_cfg(64)
    bad.reserved[3] = 1
    assert quant(bad) == INVALID and quant(None) == INVALID
    assert quant(c, T=-1) == INVALID and quant(c, T=(1 << 30) + 1) == UNSUPPORTED
    assert quant(c, T=0, ins=None, y=None, q=None, s=None) == OK
    for kw in (dict(ins=None), dict(ins=(None, B, C, D, E)), dict(q=None), dict(s=None), dict(y=None),
               dict(ins=(A, None, C, None, E), y=None), dict(ins=(A, None, None, D, E), y=None), dict(ins=(A, None, None, None, E))):
        assert quant(c, **kw) == INVALID, kw
    for kw in (dict(ins=(A + 8, B, C, D, E)), dict(ins=(A, B, C, D + 4, E)), dict(y=G + 8), dict(q=I + 8), dict(s=J + 4)):
        assert quant(c, **kw) == ALIGNMENT, kw
    for kw in (dict(q=A), dict(q=B + 16), dict(q=G), dict(s=D), dict(s=I + 64), dict(y=B), dict(y=A + 16), dict(q=E)):
        assert quant(c, **kw) == INVALID, kw


def ex(**kw):
    c = moe.exchange_cfg(64, 8, 2)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def dispatch(c, ids=A, x=B, xscale=None, T=4, off=C, rows=D, xs=E, sscale=None, ws=G, wb=BIG):
    return L.moe_dispatch_forward(ref(c), ids, x, xscale, T, off, rows, xs, sscale, ws, wb, None)


def combine(c, z=A, rows=B, w=C, res=D, T=4, y=E):
    return L.moe_combine_forward(ref(c), z, rows, w, res, T, y, None)


def uncombine(c, dy=A, z=B, rows=C, w=D, T=4, dz=E, dw=G):
    return L.moe_combine_backward(ref(c), dy, z, rows, w, T, dz, dw, None)


@pytest.mark.parametrize("change,code", [
    (dict(d_model=0), INVALID), (dict(n_experts=0), INVALID), (dict(top_k=0), INVALID), (dict(format=2), INVALID),
    (dict(d_model=12), UNSUPPORTED), (dict(format=1, d_model=72), UNSUPPORTED), (dict(n_experts=1025), UNSUPPORTED),
    (dict(top_k=33), UNSUPPORTED), (dict(d_model=(1 << 29) + 8), UNSUPPORTED)])
def test_exchange_configurations_refused(change, code):
    c = ex(**change)
    assert dispatch(c) == code and combine(c) == code and uncombine(c) == code
    assert L.moe_dispatch_backward(ref(c), A, B, 4, C, None) == code
    assert moe.moe_dispatch_workspace_bytes(c, 4) == 0


def test_exchange_arguments_refused():
    c, e = ex(), ex(format=moe.ROWS_E4M3)
    for i in range(4):
        bad = ex()
        bad.reserved[i] = 1
        assert dispatch(bad) == INVALID
    assert dispatch(None) == INVALID and combine(None) == INVALID and uncombine(None) == INVALID
    assert dispatch(c, T=-1) == INVALID and combine(c, T=-1) == INVALID
    assert dispatch(c, T=(1 << 29) + 1) == UNSUPPORTED and combine(c, T=(1 << 29) + 1) == UNSUPPORTED   # 2^30 slots and two
    for kw in (dict(ids=None), dict(off=None), dict(rows=None), dict(ws=None), dict(x=None), dict(xs=None), dict(xscale=I),
               dict(sscale=I)):
        assert dispatch(c, **kw) == INVALID, kw
    assert dispatch(e) == INVALID and dispatch(e, xscale=I) == INVALID and dispatch(e, sscale=I) == INVALID
    for kw in (dict(ids=A + 4), dict(x=B + 8), dict(off=C + 4), dict(rows=D + 8), dict(xs=E + 8), dict(ws=G + 8)):
        assert dispatch(c, **kw) == ALIGNMENT, kw
    assert dispatch(c, wb=moe.moe_dispatch_workspace_bytes(c, 4) - 1) == WORKSPACE
    for kw in (dict(xs=B), dict(rows=A + 16), dict(off=D), dict(xs=G), dict(rows=E + 64), dict(off=A)):
        assert dispatch(c, **kw) == INVALID, kw
    for kw in (dict(z=None), dict(rows=None), dict(y=None), dict(y=A + 64), dict(y=B), dict(y=C), dict(y=D + 16)):
        assert combine(c, **kw) == INVALID, kw
    for kw in (dict(z=A + 8), dict(rows=B + 4), dict(w=C + 4), dict(res=D + 8), dict(y=E + 2)):
        assert combine(c, **kw) == ALIGNMENT, kw
    assert combine(e) == UNSUPPORTED and uncombine(e) == UNSUPPORTED
    for kw in (dict(dy=None), dict(rows=None), dict(w=None), dict(z=None), dict(dz=None, dw=None), dict(dz=A), dict(dz=B + 16),
               dict(dw=D), dict(dw=C), dict(dw=E + 32)):
        assert uncombine(c, **kw) == INVALID, kw
    assert uncombine(c, dw=G + 4) == ALIGNMENT and uncombine(c, dz=E + 8) == ALIGNMENT
    assert combine(c, T=0, z=None, rows=None, y=None) == OK and uncombine(c, T=0) == OK
    assert moe.moe_dispatch_workspace_bytes(c, -1) == 0 and moe.moe_dispatch_workspace_bytes(c, (1 << 29) + 1) == 0


def test_quantiser_of_weights():
    w = torch.randn(20, 48, generator=torch.Generator().manual_seed(0))
    w[3] = 0
    q, s = moe.w8_quantize(w)
    assert q.dtype == torch.float8_e4m3fn and s.dtype == torch.float32 and s[3] == 2.0 ** -126
    v = q.float() * s[:, None]
    # half a step of three bits behind the first, and of the smallest normal
    assert ((v - w).abs() <= torch.maximum(w.abs() * 2.0 ** -4, s[:, None] * 2.0 ** -10) * (1 + 1e-6)).all()
    assert (q.float().abs().amax(1)[[0, 1, 2, 4]] == 448).all()
    assert moe.w8_quantize(torch.empty(3, 0))[1].tolist() == [2.0 ** -126] * 3
    with pytest.raises(ValueError):
        moe.w8_quantize(w[0])


def test_binding_refuses_cpu_tensors_and_missing_scales():
    x, ids = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_linear_forward(moe.linear_cfg(64, 8, fmt=moe.LINEAR_E4M3), x, moe.LinearWeights(x))
    with pytest.raises(ValueError):
        moe.moe_dispatch_forward(moe.exchange_cfg(64, 8, 2, fmt=moe.ROWS_E4M3), x, ids)
    with pytest.raises(ValueError):
        moe.moe_dispatch_forward(moe.exchange_cfg(64, 8, 3), x, ids)
    with pytest.raises(ValueError):
        moe.linear_pre(moe.linear_cfg(64, 8), 1 << 31)
    assert exchange.EXPORTED and linear.EXPORTED
