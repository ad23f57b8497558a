"""Sizes at which the dense block's 32-bit row and column counts would run over, and the sums
that the kernels form from the largest ones that are taken.  Needs no GPU: refusals come before
anything is enqueued."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_block_host import BIG, C, UNSUPPORTED, glu, glu_backward, glu_forward  # noqa: E402
from test_block_host import norm_backward, norm_forward, w4, w4_linear  # noqa: E402

TOKENS, INPUTS, OUTPUTS = 1 << 30, 1 << 29, 1 << 30
INT = (1 << 31) - 1


@pytest.mark.parametrize("T", [TOKENS + 1, INT - 3 * 2432, INT])
def test_too_many_tokens(T):
    c, n = moe.glu_cfg(8, 8), moe.norm_cfg(8)
    assert glu_forward(c, T=T) == UNSUPPORTED and glu_backward(c, T=T) == UNSUPPORTED
    assert glu_forward(c, T=T, saved=C, sb=BIG) == UNSUPPORTED
    assert norm_forward(n, T=T) == UNSUPPORTED and norm_backward(n, T=T) == UNSUPPORTED
    assert moe.moe_glu_workspace_bytes(c, T) == 0 and moe.moe_glu_saved_bytes(c, T) == 0
    assert moe.moe_block_norm_workspace_bytes(n, T) == 0
    assert moe.moe_glu_saved_bytes(c, TOKENS) >= TOKENS * 8 * 10 and moe.moe_block_norm_workspace_bytes(n, TOKENS) > 0


@pytest.mark.parametrize("change", [dict(d_model=INPUTS + 8), dict(ff=INPUTS + 8), dict(d_model=INT // 8 * 8)])
def test_too_wide_ffn(change):
    c = glu(**change)
    assert glu_forward(c, T=1) == UNSUPPORTED and glu_backward(c, T=1) == UNSUPPORTED
    assert moe.moe_glu_workspace_bytes(c, 1) == 0


@pytest.mark.parametrize("change", [dict(n_in=INPUTS + 128), dict(n_out=OUTPUTS + 1), dict(n_out=INT),
                                    dict(n_out=INT // 2 + 17, glu=1)])
def test_too_wide_matrix(change):
    assert w4_linear(w4(**change), T=1) == UNSUPPORTED


def test_sums_of_the_largest_sizes_fit():
    """What the kernels add to a row, column or byte count before they compare it."""
    sms = 160
    assert TOKENS + 3 * sms * 16 <= INT           # norms: rows ahead of every group's next row
    assert TOKENS + 256 + 256 <= INT              # tiles of 256 rows, rounded up
    assert INPUTS * 2 + 64 * 4 + 64 <= INT        # bytes of a row of bf16 weights, ring steps past it
    assert OUTPUTS + 32 + 16 * sms * 32 <= INT    # units of 32 rows, a grid of slots past the last
