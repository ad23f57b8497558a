"""The sparse layer's binding on the stand-in for torch's allocator and the library: memory,
streams and devices of its calls, as for the dense block's."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from sparse_moe_ffn_route_gb300 import block  # noqa: E402
from test_block_binding import DEVICE, Stream, World, freed_sizes, refill  # noqa: E402

T, D, E, K, FF = 6, 64, 8, 2, 32


@pytest.fixture
def world(monkeypatch):
    w = World(monkeypatch)
    shim = block.torch
    shim.int32 = torch.int32
    monkeypatch.setattr(moe, "torch", shim)
    monkeypatch.setattr(moe, "_lib", block._lib)
    return w


def operators(w, device=DEVICE):
    """{name: call taking stream=}."""
    def t(*shape, dtype=torch.bfloat16):
        return w.tensor(*shape, dtype=dtype, device=device)

    cfg = moe.qwen_cfg(D, E, K, FF, FF)
    x, router = t(T, D), moe.Router(t(E, D))
    experts = moe.Experts(gate=t(E, FF, D), up=t(E, FF, D), down=t(E, D, FF))
    shared = moe.Shared(t(FF, D), t(FF, D), t(D, FF), t(D))
    ids, weights = t(T, K, dtype=torch.int32), t(T, K, dtype=torch.float32)
    logits = t(T, E, dtype=torch.float32)
    blocks, scales = t(4, 2, 16, dtype=torch.uint8), t(4, 2, dtype=torch.uint8)
    return {
        "route": lambda **kw: moe.moe_route(cfg, x, router, shared, **kw),
        "topk": lambda **kw: moe.moe_topk_from_logits(cfg, logits, **kw),
        "group": lambda **kw: moe.moe_group_by_expert(cfg, ids, **kw),
        "forward": lambda **kw: moe.moe_ffn_forward(cfg, x, router, experts, shared, **kw),
        "noalloc": lambda **kw: moe.moe_ffn_forward_noalloc(cfg, x, router, experts, shared, **kw),
        "routed": lambda **kw: moe.moe_ffn_forward_routed(cfg, x, ids, weights, experts, shared, **kw),
        "mxfp4": lambda **kw: moe.moe_mxfp4_to_bf16(blocks, scales, **kw),
    }


NAMES = ("route", "topk", "group", "forward", "noalloc", "routed", "mxfp4")


def pointers(call):
    return {a for a in call.args[:-1] if isinstance(a, int) and a > 0x100000}


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_a_given_stream_is_not_handed_out(world, name):
    ops = operators(world)
    ops[name](stream=Stream(0x77))
    noted = world.calls[-1]
    assert noted.stream == 0x77
    mine = pointers(noted)
    del noted, ops
    world.calls.clear()
    got, _ = refill(world, freed_sizes(world))
    assert mine and not got & mine


@pytest.mark.parametrize("name", NAMES)
def test_memory_freed_by_the_current_stream_is_not_written_by_another(world, name):
    ops = operators(world)
    cfg = moe.qwen_cfg(D, E, K, FF, FF)
    old = [world.tensor(n, dtype=torch.uint8) for n in
           (T * D * 2, T * K * 4, E * 4, E * 4 + 4, 4 * 64 * 2, moe.moe_workspace_bytes(cfg, T)) for _ in range(8)]
    busy = {t.data_ptr() for t in old}
    del old
    ops[name](stream=0x77)
    assert world.calls[-1].stream == 0x77 and not pointers(world.calls[-1]) & busy


@pytest.mark.parametrize("name", NAMES)
def test_calls_run_on_the_device_of_their_tensors(world, name):
    other = torch.device("cuda", 1)
    world.current[1] = Stream(0x31, other)
    ops = operators(world, other)
    ops[name]()
    ops[name](stream=Stream(0x33, other))
    assert [(c.device, c.stream) for c in world.calls] == [(1, 0x31), (1, 0x33)] and world.selected == 0
    with pytest.raises(ValueError, match="stream"):
        ops[name](stream=Stream(0x34, DEVICE))


@pytest.mark.parametrize("name", NAMES)
def test_memory_on_one_stream_is_free_at_once(world, name):
    ops = operators(world)
    ops[name]()
    assert world.calls[-1].stream == 0
    mine = pointers(world.calls[-1])
    del ops
    world.calls.clear()
    got, _ = refill(world, freed_sizes(world))
    assert got & mine




class HostRows:
    """Host tensors of the synchronous call."""
    is_cuda, shape, dtype = False, torch.Size((T, D)), torch.bfloat16

    def data_ptr(self):
        return 0x1000


@pytest.mark.parametrize("bound", [False, True])
def test_workspace_of_a_host_call_is_made_for_its_stream_and_device(world, bound):
    other = torch.device("cuda", 1)
    cfg = moe.qwen_cfg(D, E, K, FF, 0)
    t = lambda *s: world.tensor(*s, device=other)   # noqa: E731
    router, experts = moe.Router(t(E, D)), moe.Experts(gate=t(E, FF, D), up=t(E, FF, D), down=t(E, D, FF))
    old = [world.tensor(moe.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device=other) for _ in range(4)]
    busy = {o.data_ptr() for o in old}
    del old
    stream = Stream(0x44, other)
    if bound:
        moe.BoundForwardHost(cfg, HostRows(), router, experts, y_host=HostRows(), stream=stream)()
    else:
        moe.moe_ffn_forward_host(cfg, HostRows(), router, experts, y_host=HostRows(), stream=stream)
    call = world.calls[-1]
    assert call.stream == 0x44 and call.device == 1 and not pointers(call) & busy
