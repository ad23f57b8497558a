"""Host checks of the dense block's entry points that need no GPU: sizes, refusals before
anything is enqueued, the Python binding's checks of its tensors, and the 4-bit quantiser."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from sparse_moe_ffn_route_gb300 import block  # noqa: E402

OK, INVALID, UNSUPPORTED, WORKSPACE, ALIGNMENT = 0, -1, -2, -3, -4
# aligned addresses that are never read: every refusal comes before the first launch
A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000
BIG = 1 << 40


def ref(s):
    return None if s is None else ctypes.byref(s)


def three(*p):
    return block._Three(*p)


def five(*p):
    return block._Five(*(list(p) + [None] * (5 - len(p))))


GLU_BAD = [(dict(d_model=0), INVALID), (dict(ff=-8), INVALID), (dict(act=2), INVALID), (dict(act=-1), INVALID),
           (dict(glu_limit=float("nan")), INVALID), (dict(glu_limit=-1.0), INVALID),
           (dict(glu_alpha=float("inf")), INVALID), (dict(d_model=12), UNSUPPORTED), (dict(ff=100), UNSUPPORTED)]


def glu(**kw):
    c = moe.glu_cfg(64, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def glu_forward(c, T=4, x=A, w=three(A, B, C), y=B, saved=None, sb=0, ws=D, wb=BIG):
    return moe._lib.moe_glu_forward(ref(c), x, T, ref(w), y, saved, sb, ws, wb, None)


def glu_backward(c, T=4, x=A, w=three(A, B, C), saved=C, sb=BIG, dy=B, dx=D, g=three(A, B, C), ws=D, wb=BIG):
    return moe._lib.moe_glu_backward(ref(c), x, T, ref(w), saved, sb, dy, dx, ref(g), ws, wb, None)


@pytest.mark.parametrize("change,code", GLU_BAD)
def test_glu_configurations_refused(change, code):
    c = glu(**change)
    assert glu_forward(c) == code and glu_backward(c) == code
    assert glu_forward(c, T=0) == code
    assert moe.moe_glu_workspace_bytes(c, 4) == 0 and moe.moe_glu_saved_bytes(c, 4) == 0
    with pytest.raises(moe.MoeError):
        moe.glu_workspace(c, 4, "cpu")


def test_glu_reserved_and_null():
    c = glu()
    c.reserved[1] = 1
    assert glu_forward(c) == INVALID
    assert glu_forward(None) == INVALID and glu_backward(None) == INVALID
    c = glu()
    for kw in (dict(T=-1), dict(x=None), dict(w=None), dict(w=three(A, None, C)), dict(y=None), dict(ws=None)):
        assert glu_forward(c, **kw) == INVALID, kw
    for kw in (dict(T=-1), dict(x=None), dict(w=None), dict(w=three(None, B, C)), dict(saved=None), dict(dy=None),
               dict(ws=None)):
        assert glu_backward(c, **kw) == INVALID, kw


def test_glu_alignment_and_sizes():
    c = glu()
    for kw in (dict(x=A + 8), dict(w=three(A, B + 2, C)), dict(y=B + 4), dict(ws=D + 8), dict(saved=C + 8, sb=BIG)):
        assert glu_forward(c, **kw) == ALIGNMENT, kw
    for kw in (dict(x=A + 8), dict(dx=D + 2), dict(g=three(A, B, C + 2)), dict(dy=B + 8), dict(saved=C + 4)):
        assert glu_backward(c, **kw) == ALIGNMENT, kw
    need, keep = moe.moe_glu_workspace_bytes(c, 4), moe.moe_glu_saved_bytes(c, 4)
    assert glu_forward(c, wb=need - 1) == WORKSPACE
    assert glu_forward(c, saved=C, sb=keep - 1) == WORKSPACE
    assert glu_backward(c, wb=need - 1) == WORKSPACE and glu_backward(c, sb=keep - 1) == WORKSPACE


def test_glu_buffer_sizes():
    c = glu()
    # dg and du in the workspace; h, and g and u of whole blocks of 128 tokens, in the saved buffer
    assert moe.moe_glu_workspace_bytes(c, 300) >= 2 * 300 * 128 * 2
    assert moe.moe_glu_saved_bytes(c, 300) >= 300 * 128 * 2 + 2 * 384 * 128 * 4
    assert moe.moe_glu_workspace_bytes(c, -1) == 0 and moe.moe_glu_saved_bytes(c, 0) > 0
    # past 32 bits
    big = moe.glu_cfg(2048, 8192)
    assert moe.moe_glu_saved_bytes(big, 1 << 20) >= (1 << 20) * 8192 * 10


def test_glu_empty_batch_is_a_no_op():
    assert glu_forward(glu(), T=0, x=None, w=None, y=None, ws=None, wb=0) == OK
    assert glu_backward(glu(), T=0, x=None, w=None, saved=None, sb=0, dy=None, dx=None, g=None, ws=None, wb=0) == OK


def norm(**kw):
    c = moe.norm_cfg(64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


FULL = (A, B, C, D, A)   # x, branch, post_w, gate, pre_w


def norm_forward(c, T=4, i=FULL, y=B, a=C):
    return moe._lib.moe_block_norm_forward(ref(c), ref(None if i is None else five(*i)), T, y, a, None)


def norm_backward(c, T=4, i=FULL, dy=A, da=B, o=(A, B, C, D, A), ws=D, wb=BIG):
    return moe._lib.moe_block_norm_backward(ref(c), ref(None if i is None else five(*i)), T, dy, da,
                                            ref(None if o is None else five(*o)), ws, wb, None)


@pytest.mark.parametrize("change,code", [
    (dict(d_model=0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(residual_scale=float("inf")), INVALID), (dict(branch_scale=float("nan")), INVALID),
    (dict(d_model=20), UNSUPPORTED), (dict(d_model=16392), UNSUPPORTED)])
def test_norm_configurations_refused(change, code):
    c = norm(**change)
    assert norm_forward(c) == code and norm_backward(c) == code
    assert moe.moe_block_norm_workspace_bytes(c, 4) == 0


def test_norm_arguments_refused():
    c = norm()
    bad = norm()
    bad.reserved[0] = 1
    assert norm_forward(bad) == INVALID and norm_forward(None) == INVALID
    for kw in (dict(T=-1), dict(i=None), dict(i=(None, B, C, D, A)), dict(i=(A,), y=None, a=None),
               dict(i=(A, None, C, None, A), y=None), dict(i=(A, None, None, D, A), y=None), dict(y=None),
               dict(a=None), dict(i=(A, B, C, D)), dict(i=(A, None, None, None, A))):
        assert norm_forward(c, **kw) == INVALID, kw
    for kw in (dict(T=-1), dict(i=None), dict(o=None), dict(dy=None, da=None), dict(ws=None),
               dict(i=(A, None, None, None, A), o=(A,)), dict(i=(A, B, C, D), o=(A,)),
               dict(i=(A, None, None, None, A), dy=None, o=(A, B)), dict(i=(A, B, C, None, A)),
               dict(i=(A, B, None, D, A))):
        assert norm_backward(c, **kw) == INVALID, kw
    for kw in (dict(i=(A + 2, B, C, D, A)), dict(y=B + 8), dict(a=C + 2)):
        assert norm_forward(c, **kw) == ALIGNMENT, kw
    for kw in (dict(dy=A + 8), dict(o=(A, B, C + 4, D, A)), dict(ws=D + 4)):
        assert norm_backward(c, **kw) == ALIGNMENT, kw
    assert norm_backward(c, wb=moe.moe_block_norm_workspace_bytes(c, 4) - 1) == WORKSPACE
    assert norm_forward(c, T=0, i=None, y=None, a=None) == OK
    assert norm_backward(c, T=0, i=None, dy=None, da=None, o=(), ws=None, wb=0) == OK


def w4(**kw):
    c = moe.w4_cfg(128, 10)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def w4_linear(c, T=4, x=A, w=three(A, B, None), y=C):
    return moe._lib.moe_w4_linear(ref(c), x, T, ref(w), y, None)


@pytest.mark.parametrize("change,code", [
    (dict(n_in=0), INVALID), (dict(n_out=0), INVALID), (dict(glu=2), INVALID), (dict(act=5), INVALID),
    (dict(glu_limit=float("nan")), INVALID), (dict(group=16), UNSUPPORTED), (dict(group=0), UNSUPPORTED),
    (dict(n_in=192), UNSUPPORTED)])
def test_w4_configurations_refused(change, code):
    assert w4_linear(w4(**change)) == code


def test_w4_arguments_refused():
    c = w4()
    bad = w4()
    bad.reserved[0] = 3
    assert w4_linear(bad) == INVALID and w4_linear(None) == INVALID
    for kw in (dict(T=-1), dict(x=None), dict(y=None), dict(w=None), dict(w=three(None, B, None)),
               dict(w=three(A, None, None))):
        assert w4_linear(c, **kw) == INVALID, kw
    for kw in (dict(x=A + 2), dict(y=C + 2), dict(w=three(A + 4, B, None)), dict(w=three(A, B + 2, None)),
               dict(w=three(A, B, C + 1))):
        assert w4_linear(c, **kw) == ALIGNMENT, kw
    assert w4_linear(c, T=0, x=None, w=None, y=None) == OK


def test_binding_checks_its_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        block._tensor(x, "x", (4, 64))
    with pytest.raises(ValueError, match="shape"):
        moe.moe_glu_forward(moe.glu_cfg(128, 64), x, None)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_block_norm_forward(moe.norm_cfg(64), x[0])
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_w4_linear(moe.w4_cfg(64, 8, 64), x, moe.w4_quantize(torch.zeros(8, 64), 64))


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantiser_is_within_half_a_code(group, zeros):
    gen = torch.Generator().manual_seed(group + zeros)
    w = torch.randn(5, 256, generator=gen) + 0.3
    w[2] = 0.0
    q = moe.w4_quantize(w, group, zeros)
    codes = torch.stack((q.codes & 15, q.codes >> 4), 2).reshape(5, -1, group).double()
    zero = 8.0 if q.zeros is None else q.zeros.double()[:, :, None]
    s = q.scales.double()[:, :, None]
    err = ((codes - zero) * s - w.double().reshape(5, -1, group)).abs()
    # half a code, half a code more from the zero point's own rounding, and the ends of the
    # range, which the scale's rounding to bf16 (2^-8 of up to 15 codes) may cut
    assert (err <= s * (1.0 + 15 * 2.0 ** -8)).all()
    assert (err[2] == 0).all()
