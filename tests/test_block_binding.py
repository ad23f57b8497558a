"""The dense block's binding on a stand-in for torch's allocator and for the library, without
a GPU: what memory, streams, devices and arguments a call leaves to the kernels.

The allocator hands freed memory out again to the stream that it belongs to, unless it was
recorded on another stream, whose work (which never ends here) may still use it."""
import ctypes
import gc
import types

import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from sparse_moe_ffn_route_gb300 import block  # noqa: E402

DEVICE = torch.device("cuda", 0)


class Stream:
    def __init__(self, handle, device=DEVICE):
        self.cuda_stream, self.device = handle, device


class Memory:
    """Blocks by stream: freed ones are taken again first."""

    def __init__(self):
        self.free, self.next, self.made = {}, 0x100000, []

    def take(self, size, stream):
        free = self.free.setdefault(stream, [])
        for i, (at, n) in enumerate(free):
            if n == size:
                return free.pop(i)[0]
        self.next += size + (-size) % 4096 + 4096
        return self.next


class Tensor:
    is_cuda = True

    def __init__(self, world, shape, dtype=torch.bfloat16, device=DEVICE):
        self.world, self.shape, self.dtype, self.device = world, torch.Size(shape), dtype, device
        self.size = self.numel() * dtype.itemsize
        self.home, self.used = world.current[device.index].cuda_stream, set()
        self.at = world.memory.take(self.size, self.home)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at

    def record_stream(self, stream):
        self.used.add(stream.cuda_stream)

    def __del__(self):
        if not self.used - {self.home}:
            self.world.memory.free[self.home].append((self.at, self.size))


class World:
    """The parts of torch that the binding uses, and a library that notes its calls."""

    def __init__(self, monkeypatch):
        self.memory, self.calls, self.selected, self.sized = Memory(), [], 0, []
        self.current = {0: Stream(0), 1: Stream(0, torch.device("cuda", 1))}
        world = self

        class using:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                at = self.stream.device.index
                self.before = world.current[at], world.selected
                world.current[at], world.selected = self.stream, at

            def __exit__(self, *_):
                world.current[self.stream.device.index], world.selected = self.before

        self.using = using

        class selecting:
            def __init__(self, device):
                self.device = device

            def __enter__(self):
                self.before = world.selected
                world.selected = getattr(self.device, "index", self.device)

            def __exit__(self, *_):
                world.selected = self.before

        def current_stream(device=None):
            return self.current[self.selected if device is None else getattr(device, "index", device)]

        cuda = types.SimpleNamespace(Stream=Stream, stream=using, device=selecting, current_stream=current_stream,
                                     current_device=lambda: self.selected, device_count=lambda: 2,
                                     default_stream=lambda d=None: Stream(0, d or DEVICE),
                                     ExternalStream=lambda h, device=DEVICE: Stream(h, device))

        def empty(*shape, dtype=torch.float32, device=DEVICE):
            shape = shape[0] if isinstance(shape[0], tuple) else shape
            return Tensor(self, shape, dtype, torch.device(device) if isinstance(device, str) else device)

        monkeypatch.setattr(block, "torch", types.SimpleNamespace(
            cuda=cuda, empty=empty, empty_like=lambda t: Tensor(self, t.shape, t.dtype, t.device),
            bfloat16=torch.bfloat16, uint8=torch.uint8, float32=torch.float32, device=torch.device))
        monkeypatch.setattr(block, "_raw_stream", lambda index: self.current[index].cuda_stream)
        if hasattr(block, "_current_device"):
            monkeypatch.setattr(block, "_current_device", lambda: self.selected)
        real = moe._lib

        def noted(name):
            def call(*args):
                self.calls.append(types.SimpleNamespace(name=name, args=args, stream=args[-1], device=self.selected))
                return 0
            return call

        class Library:
            def __getattr__(self, name):
                if not name.endswith("_bytes"):
                    return noted(name)
                world.sized.append(world.selected)
                return getattr(real, name)

        monkeypatch.setattr(block, "_lib", Library())

    def tensor(self, *shape, dtype=torch.bfloat16, device=DEVICE):
        return Tensor(self, shape, dtype, device)


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def operators(w, T=300, d=64, ff=128, device=DEVICE):
    """{name: (cfg, bind, call, arguments)} of every entry point."""
    def t(*shape, dtype=torch.bfloat16):
        return w.tensor(*shape, dtype=dtype, device=device)

    glu, norm, w4 = moe.glu_cfg(d, ff), moe.norm_cfg(d), moe.w4_cfg(d, ff, 32)
    weights = moe.GluWeights(t(ff, d), t(ff, d), t(d, ff))
    saved = t(moe.moe_glu_saved_bytes(glu, T), dtype=torch.uint8)
    parts = dict(branch=t(T, d), post_w=t(d), gate=t(T, dtype=torch.float32), pre_w=t(d))
    codes = moe.W4Weights(t(ff, d // 2, dtype=torch.uint8), t(ff, d // 32), t(ff, d // 32, dtype=torch.uint8))
    return {
        "glu_forward": (glu, block.bind_glu_forward, block.moe_glu_forward, dict(x=t(T, d), w=weights)),
        "glu_training": (glu, block.bind_glu_forward, block.moe_glu_forward, dict(x=t(T, d), w=weights, saved=saved)),
        "glu_backward": (glu, block.bind_glu_backward, block.moe_glu_backward,
                         dict(x=t(T, d), w=weights, saved=saved, dy=t(T, d))),
        "norm_forward": (norm, block.bind_block_norm_forward, block.moe_block_norm_forward, dict(x=t(T, d), **parts)),
        "norm_backward": (norm, block.bind_block_norm_backward, block.moe_block_norm_backward,
                          dict(x=t(T, d), dy=t(T, d), da=t(T, d), **parts)),
        "w4_linear": (w4, block.bind_w4_linear, block.moe_w4_linear, dict(x=t(T, d), w=codes)),
    }


NAMES = ("glu_forward", "glu_training", "glu_backward", "norm_forward", "norm_backward", "w4_linear")


def pointers(call):
    """Every address that a noted call was given, those in its structures too."""
    out = set()
    for a in call.args[:-1]:
        out.add(a if isinstance(a, int) else ctypes.cast(a, ctypes.c_void_p).value)
    for a in call.args:
        if isinstance(a, ctypes.c_void_p) and a.value:
            out.update(ctypes.cast(a, ctypes.POINTER(ctypes.c_uint64))[i] for i in range(3))
    return out


def refill(w, sizes):
    """Addresses that the current stream's next allocations of these sizes get."""
    gc.collect()
    new = [w.tensor(n, dtype=torch.uint8) for n in sizes for _ in range(8)]
    return {t.data_ptr() for t in new}, new


def freed_sizes(w):
    return {n for blocks in w.memory.free.values() for _, n in blocks} | {2, 64}


@pytest.mark.parametrize("kind", ["object", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_a_given_stream_is_not_handed_out(world, name, kind):
    """Results dropped at once, and the workspace with them, while the call's stream is busy."""
    cfg, _, call, kw = operators(world)[name]
    side = Stream(0x77)
    call(cfg, **kw, stream=side if kind == "object" else 0x77)
    noted = world.calls[-1]
    assert noted.stream == 0x77
    mine = pointers(noted)
    del kw, noted
    world.calls.clear()
    got, _ = refill(world, freed_sizes(world))
    assert not got & mine


@pytest.mark.parametrize("name", NAMES)
def test_memory_freed_by_the_current_stream_is_not_written_by_another(world, name):
    """Buffers that a call makes for a given stream are no memory that the current stream has
    freed and may still work on."""
    cfg, _, call, kw = operators(world)[name]
    old = [world.tensor(n, dtype=torch.uint8) for n in
           (300 * 64 * 2, 300 * 128 * 2, 128 * 64 * 2, 300 * 4, 64 * 4, moe.moe_glu_workspace_bytes(moe.glu_cfg(64, 128), 300),
            moe.moe_block_norm_workspace_bytes(moe.norm_cfg(64), 300)) for _ in range(8)]
    busy = {t.data_ptr() for t in old}
    del old
    gc.collect()
    call(cfg, **kw, stream=Stream(0x77))
    assert not pointers(world.calls[-1]) & busy


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_bound_call_on_other_streams_is_not_handed_out(world, name):
    """A bound call follows the current stream; its buffers belong to the stream at bind."""
    cfg, bind, _, kw = operators(world)[name]
    call = bind(cfg, **kw)
    call()
    with world.using(Stream(0x99)):
        call()
    assert [c.stream for c in world.calls] == [0, 0x99]
    mine = pointers(world.calls[-1])
    del call, kw
    world.calls.clear()
    got, _ = refill(world, freed_sizes(world))
    assert not got & mine


@pytest.mark.parametrize("name", NAMES)
def test_memory_on_one_stream_is_free_at_once(world, name):
    """On the stream that everything belongs to nothing is held back."""
    cfg, _, call, kw = operators(world)[name]
    call(cfg, **kw)
    mine = pointers(world.calls[-1])
    del kw
    world.calls.clear()
    got, _ = refill(world, freed_sizes(world))
    assert got & mine


def test_stream_handle_zero_is_the_default_stream(world):
    cfg, _, call, kw = operators(world)["w4_linear"]
    with world.using(Stream(0x55)):
        call(cfg, **kw, stream=0)
    assert world.calls[-1].stream == 0


@pytest.mark.parametrize("name", NAMES)
def test_a_bound_call_keeps_its_configuration_and_tensors(world, name):
    """Changing the configuration, or replacing the tensors in the structures that were given,
    after the checks changes nothing that the kernels get."""
    cfg, bind, _, kw = operators(world)[name]
    before = bytes(cfg)
    call = bind(cfg, **kw)
    call()
    first = pointers(world.calls[-1])
    for field in ("d_model", "ff", "n_in", "n_out"):
        if hasattr(cfg, field):
            setattr(cfg, field, 1 << 20)
    if "w" in kw:
        for f in vars(kw["w"]):
            setattr(kw["w"], f, None)
    out = call()
    for o in out if isinstance(out, tuple) else (out,):
        if isinstance(o, (moe.GluGrads, moe.NormGrads)):
            for f in vars(o):
                setattr(o, f, None)
    del kw, out
    call()
    assert ctypes.string_at(world.calls[-1].args[0], len(before)) == before
    assert pointers(world.calls[-1]) == first
    world.calls.clear()
    got, _ = refill(world, freed_sizes(world))
    assert not got & first


def test_pointers_of_replaced_tensors_are_not_handed_out(world):
    cfg, bind, _, kw = operators(world)["glu_backward"]
    call = bind(cfg, **kw)
    call()
    mine = pointers(world.calls[-1])
    kw["w"].gate = kw["w"].up = kw["w"].down = None
    got, _ = refill(world, freed_sizes(world))
    assert not got & mine


@pytest.mark.parametrize("name", NAMES)
def test_calls_run_on_the_device_of_their_tensors(world, name):
    """The library sizes grids and launches on the current device: that of the tensors."""
    other = torch.device("cuda", 1)
    world.current[1] = Stream(0x31, other)
    cfg, bind, call, kw = operators(world, device=other)[name]
    world.sized.clear()
    call(cfg, **kw)
    bound = bind(cfg, **kw)
    bound()
    with world.using(Stream(0x32, other)):
        bound()
    call(cfg, **kw, stream=Stream(0x33, other))
    assert [(c.device, c.stream) for c in world.calls] == [(1, 0x31), (1, 0x31), (1, 0x32), (1, 0x33)]
    assert world.selected == 0 and set(world.sized) <= {1}
    with pytest.raises(ValueError, match="stream"):
        call(cfg, **kw, stream=Stream(0x34, DEVICE))
    assert len(world.calls) == 4


@pytest.mark.parametrize("T", [1 << 31, (1 << 32) + 3])
def test_more_tokens_than_the_library_counts(T):
    """Sizes are int32 in the library: a larger T must not arrive there without its upper bits."""
    glu, norm, w4 = moe.glu_cfg(8, 8), moe.norm_cfg(8), moe.w4_cfg(32, 8, 32)
    x, wide = torch.empty(T, 8, dtype=torch.bfloat16, device="meta"), torch.empty(T, 32, dtype=torch.bfloat16, device="meta")
    w = moe.GluWeights(x[:8], x[:8], x[:8])
    for call in (lambda: moe.moe_glu_forward(glu, x, w), lambda: moe.moe_block_norm_forward(norm, x, pre_w=x[0]),
                 lambda: moe.moe_block_norm_backward(norm, x, da=x, pre_w=x[0]),
                 lambda: moe.moe_w4_linear(w4, wide, moe.W4Weights(x, x)),
                 lambda: moe.moe_glu_workspace_bytes(glu, T), lambda: moe.moe_glu_saved_bytes(glu, T),
                 lambda: moe.moe_block_norm_workspace_bytes(norm, T), lambda: moe.glu_workspace(glu, T, "meta"),
                 lambda: moe.glu_saved(glu, T, "meta"), lambda: moe.block_norm_workspace(norm, T, "meta")):
        with pytest.raises(ValueError, match="tokens"):
            call()
