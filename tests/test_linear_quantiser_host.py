"""The weights' quantiser on rows that are not finite, as the header has it for every row in 8 bits: a NaN
is passed over by the maximum and keeps its own place; an infinity makes the scale infinite."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")


def test_nan_and_infinities():
    w = torch.randn(5, 32, generator=torch.Generator().manual_seed(3))
    clean_q, clean_s = moe.w8_quantize(w)
    at = int(w[1].abs().argmin())         # not the largest of its row
    bad = w.clone()
    bad[1, at] = float("nan")
    bad[2] = float("nan")
    bad[3, 4] = -float("inf")
    q, s = moe.w8_quantize(bad)
    q, clean_q = q.float(), clean_q.float()
    assert torch.equal(s[[0, 1, 4]], clean_s[[0, 1, 4]]) and torch.equal(q[[0, 4]], clean_q[[0, 4]])
    assert torch.isnan(q[1]).nonzero().flatten().tolist() == [at]
    others = [i for i in range(32) if i != at]
    assert torch.equal(q[1, others], clean_q[1, others])
    assert s[2] == 2.0 ** -126 and torch.isnan(q[2]).all()
    assert torch.isinf(s[3]) and torch.isnan(q[3]).nonzero().flatten().tolist() == [4]
    assert (q[3, [i for i in range(32) if i != 4]] == 0).all()
