"""The 8-bit codes of the norm: the nearest to the quotient of a row's value and its scale, with the
second norm as without it, and over rows that a CTA takes in turn."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_gpu_block import gen_for, norm64, rnd  # noqa: E402
from test_gpu_linear import quant_close  # noqa: E402
from test_gpu_block import H, Guarded, close  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24      # half a step of fp32


def divided(a):
    """Codes (as fp32) and scale of the fp32 rows a by their definition, each division rounded once."""
    top = a.abs().amax(1)
    scale = (top / torch.full_like(top, 448.0)).clamp(min=2.0 ** -126)
    return (a / scale[:, None]).to(torch.float8_e4m3fn).float(), scale


@pytest.mark.parametrize("d", [8, 64, 1024, 2048, 4096, 16384])
def test_rows_of_ones_take_the_weights_codes(d):
    """With x = +-1 and eps = 0 the mean square is 1 and a = +-pre_w without a rounding, so that scale
    and codes are those of one division each, to the bit.  Weights of 8 significant bits give many
    quotients just between two codes (one in 16, where the largest is 1.75 times a power of 2)."""
    gen = gen_for(d, 448)
    x = torch.where(torch.rand(3, d, generator=gen, device="cuda") < 0.5, -1.0, 1.0).bfloat16()
    cfg = moe.norm_cfg(d, eps=0.0)
    for i in range(60):
        w = rnd(gen, d)
        top = 7.0 * 2.0 ** (i % 7) if i % 2 else w.float().abs().amax().item() * (1.0 + i / 128)
        w[i % d] = top
        _, q, scale = moe.moe_block_norm_quant(cfg, x, pre_w=w)
        want, s = divided(x.float() * w.float())
        assert torch.equal(scale, s), (i, scale, s)
        assert torch.equal(q.float(), want), (i, (q.float() != want).nonzero()[:4])


def code_steps(v):
    """Half a step of e4m3 at |v|."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 4.0)


@pytest.mark.parametrize("T,d", [(33, 1000), (700, 2880), (500, 4096), (40, 16384)])
def test_codes_are_the_nearest_of_a_value_six_roundings_off(T, d):
    """a / scale is (y pre_w) / max|y pre_w| * 448: 1 / rms, which multiplies both, falls out, but
    for its two products' roundings.  They, the two of y pre_w, and the two divisions' are six of at
    most U each; a code may differ from the nearest to the exact value only where a border
    lies within these."""
    gen = gen_for(T, d)
    x, w = rnd(gen, T, d, scale=3.0), 1 + rnd(gen, d, scale=0.2)
    _, q, _ = moe.moe_block_norm_quant(moe.norm_cfg(d), x, pre_w=w)
    p = x.double() * w.double()
    v = p / p.abs().amax(1, keepdim=True) * 448.0
    tol = 6.01 * U * v.abs()
    close(q.float(), v, code_steps(v) + tol, "q")


# more rows than the GPU holds CTAs, in each number of vectors that a thread takes
@pytest.mark.parametrize("T,d", [(6000, 256), (3000, 2048), (3000, 2880), (2000, 4096), (1500, 8192), (700, 16384)])
def test_a_cta_takes_several_rows(T, d):
    gen = gen_for(T, d, 5)
    x, z = rnd(gen, T, d, scale=3.0), rnd(gen, T, d)
    post, gate, pre = 1 + rnd(gen, d, scale=0.2), rnd(gen, T, dtype=torch.float32), 1 + rnd(gen, d, scale=0.2)
    cfg = moe.norm_cfg(d, residual_scale=0.9, branch_scale=0.7)
    y, q, s = Guarded((T, d)), Guarded((T, d), torch.float8_e4m3fn), Guarded((T,), torch.float32)
    moe.moe_block_norm_quant(cfg, x, branch=z, post_w=post, gate=gate, pre_w=pre, y=y.t, q=q.t, scale=s.t)
    out = norm64(x, z, post, gate, pre, None, None, 0.9, 0.7)
    close(y.t, *out["y"], "y")
    a, ea = out["a"]
    quant_close(q.t, s.t, a, ea - H * a.abs())       # (a is not rounded to bf16)
    for b in (y, q, s):
        b.check()
    # each row by itself gives the same bits, and so does y in the place of x
    some = torch.randint(0, T, (5,), generator=torch.Generator().manual_seed(T)).tolist() + [T - 1]
    for t in some:
        y1, q1, s1 = moe.moe_block_norm_quant(cfg, x[t:t + 1], branch=z[t:t + 1], post_w=post, gate=gate[t:t + 1].clone(), pre_w=pre)
        assert torch.equal(y1[0], y.t[t]) and torch.equal(q1.float()[0], q.t.float()[t]) and s1[0] == s.t[t]
    y2, q2, s2 = moe.moe_block_norm_quant(cfg, x, branch=z, post_w=post, gate=gate, pre_w=pre, y=x)
    assert y2 is x and torch.equal(x, y.t) and torch.equal(q2.view(torch.uint8), q.t.view(torch.uint8)) and torch.equal(s2, s.t)
    # no norm before the codes, no branch: the quotients' roundings alone
    _, q, s = moe.moe_block_norm_quant(cfg, z)
    want, scale = divided(z.float())
    assert torch.equal(s, scale) and torch.equal(q.float(), want)


@pytest.mark.parametrize("branch", [False, True])
def test_infinities_before_the_norm(branch):
    """An infinity makes its row's 1 / rms 0: the other elements become 0, its own NaN, and the scale,
    which passes the NaN over, the least one.  In a normed branch it makes y NaN at its place, and
    with it the row's mean square and all of its a."""
    d = 64
    gen = gen_for(9)
    x, z, w = rnd(gen, 5, d), rnd(gen, 5, d), 1 + rnd(gen, d, scale=0.2)
    at, kw = (z, dict(branch=z, post_w=w)) if branch else (x, {})
    cfg = moe.norm_cfg(d)
    _, q, clean_s = moe.moe_block_norm_quant(cfg, x, pre_w=w, **kw)
    clean_q = q.float()
    at[2, 7] = float("inf")
    at[4, 9] = -float("inf")
    y, q, s = moe.moe_block_norm_quant(cfg, x, pre_w=w, **kw)
    q = q.float()
    for t, i in ((2, 7), (4, 9)):
        assert s[t] == 2.0 ** -126
        if branch:
            assert torch.isnan(y[t]).tolist() == [j == i for j in range(d)] and torch.isnan(q[t]).all()
        else:
            assert torch.isnan(q[t]).tolist() == [j == i for j in range(d)]
            assert (q[t][[j for j in range(d) if j != i]] == 0).all()
    rest = [0, 1, 3]
    assert torch.equal(q[rest], clean_q[rest]) and torch.equal(s[rest], clean_s[rest])
