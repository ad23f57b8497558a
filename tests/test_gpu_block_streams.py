"""The dense block's calls on streams other than the current one: what they allocate stays
theirs until their stream is done, whatever the caller allocates meanwhile."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")

pytestmark = pytest.mark.gpu

T, D, FF = 300, 512, 264


def inputs(T=T):
    gen = torch.Generator(device="cuda").manual_seed(7 * T)

    def rnd(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()

    w = moe.GluWeights(rnd(FF, D, scale=D ** -0.5), rnd(FF, D, scale=D ** -0.5), rnd(D, FF, scale=FF ** -0.5))
    parts = dict(branch=rnd(T, D), post_w=rnd(D), gate=rnd(T).float(), pre_w=rnd(D))
    return rnd(T, D), w, rnd(T, D), rnd(T, D), parts


def flat(out):
    if out is None:
        return []
    if torch.is_tensor(out):
        return [out]
    return [t for o in (out if isinstance(out, (tuple, list)) else vars(out).values()) for t in flat(o)]


@pytest.mark.parametrize("T", [4, 300, 6000])
def test_buffers_of_a_call_on_a_given_stream(T):
    x, w, dy, da, parts = inputs(T)
    glu, norm = moe.glu_cfg(D, FF), moe.norm_cfg(D)
    saved = moe.glu_saved(glu, T)
    moe.moe_glu_forward(glu, x, w, saved=saved)
    calls = {"forward": lambda s: moe.moe_glu_forward(glu, x, w, stream=s),
             "backward": lambda s: moe.moe_glu_backward(glu, x, w, saved, dy, stream=s),
             "norm": lambda s: moe.moe_block_norm_forward(norm, x, **parts, stream=s),
             "norm backward": lambda s: moe.moe_block_norm_backward(norm, x, dy=dy, da=da, **parts, stream=s)}
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    sizes = {moe.moe_glu_workspace_bytes(glu, T), moe.moe_block_norm_workspace_bytes(norm, T), 2 * T * D, 2 * D * FF,
             4 * T, 4 * D}
    for name, call in calls.items():
        want = [t.clone() for t in flat(call(None))]
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):     # some milliseconds of ordinary work before the call's
            hold = big
            for _ in range(40):
                hold = (hold @ big).clamp_(-1, 1)
        got = call(side)
        # meanwhile the current stream allocates buffers of the same sizes and fills them
        junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(flat(got), want):
            assert torch.equal(a, b), name
        assert all((j == 0x55).all() for j in junk), name


def test_bound_call_dropped_while_its_stream_works():
    x, w, dy, _, _ = inputs()
    glu = moe.glu_cfg(D, FF)
    saved = moe.glu_saved(glu, T)
    moe.moe_glu_forward(glu, x, w, saved=saved)
    call = moe.bind_glu_backward(glu, x, w, saved, dy)
    want = [t.clone() for t in flat(call())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    big = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    with torch.cuda.stream(side):
        hold = big
        for _ in range(40):
            hold = (hold @ big).clamp_(-1, 1)
        got = call()
        results = [t.clone() for t in flat(got)]
    n = moe.moe_glu_workspace_bytes(glu, T)
    del call, got
    junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(results, want)) and all((j == 0x55).all() for j in junk)
