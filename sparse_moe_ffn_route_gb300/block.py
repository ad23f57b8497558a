"""The dense block around the sparse layer -- Python binding of include/moe_block.h.

Three operators, each with the C ABI's name: the gated FFN (``moe_glu_forward``,
``moe_glu_backward``), the norms either side of a block with its gate and residual scale
(``moe_block_norm_forward``, ``moe_block_norm_backward``) and the linear layer with 4-bit
weights and group scales (``moe_w4_linear``).  Every function checks its tensors (device,
type, shape, contiguity: ValueError), allocates the outputs and the workspace that are
not passed in, and runs on the given stream or torch's current one.  What it allocates
belongs to the stream that it runs on, and every tensor is recorded (record_stream) on a
stream other than the one that was current at the call, so that torch's allocator gives
none of them away before the kernels are done with it; ordering the streams is left to the
caller, as with any torch operation.  Its ``bind_*`` twin takes the same arguments and
returns a ``BoundCall``: the call with its arguments marshalled once, for steps repeated on
the same buffers.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
from typing import Optional

import torch

from . import ACT_SWIGLU, MOE_OK, MoeError, _lib

_P, _I, _S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t


class GluCfg(ctypes.Structure):
    """moe_glu_cfg_t."""
    _fields_ = [("d_model", _I), ("ff", _I), ("act", _I), ("glu_limit", ctypes.c_float),
                ("glu_alpha", ctypes.c_float), ("reserved", _I * 3)]


class NormCfg(ctypes.Structure):
    """moe_norm_cfg_t."""
    _fields_ = [("d_model", _I), ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("reserved", _I * 4)]


class W4Cfg(ctypes.Structure):
    """moe_w4_cfg_t."""
    _fields_ = [("n_in", _I), ("n_out", _I), ("group", _I), ("glu", _I), ("act", _I),
                ("glu_limit", ctypes.c_float), ("glu_alpha", ctypes.c_float), ("reserved", _I * 1)]


class _Three(ctypes.Structure):
    """moe_glu_weights_t, moe_glu_grads_t, moe_w4_weights_t: three pointers."""
    _fields_ = [("p0", _P), ("p1", _P), ("p2", _P)]


class _Five(ctypes.Structure):
    """moe_norm_inputs_t, moe_norm_grads_t: five pointers."""
    _fields_ = [("p%d" % i, _P) for i in range(5)]


def _declare(name, args, res=ctypes.c_int):
    f = getattr(_lib, name)
    f.argtypes, f.restype = args, res
    return f


_declare("moe_glu_workspace_bytes", [_P, _I], _S)
_declare("moe_glu_saved_bytes", [_P, _I], _S)
_declare("moe_glu_forward", [_P, _P, _I, _P, _P, _P, _S, _P, _S, _P])
_declare("moe_glu_backward", [_P, _P, _I, _P, _P, _S, _P, _P, _P, _P, _S, _P])
_declare("moe_block_norm_forward", [_P, _P, _I, _P, _P, _P])
_declare("moe_block_norm_workspace_bytes", [_P, _I], _S)
_declare("moe_block_norm_backward", [_P, _P, _I, _P, _P, _P, _P, _S, _P])
_declare("moe_w4_linear", [_P, _P, _I, _P, _P, _P])
EXPORTED = ("moe_glu_workspace_bytes", "moe_glu_saved_bytes", "moe_glu_forward", "moe_glu_backward",
            "moe_block_norm_forward", "moe_block_norm_workspace_bytes", "moe_block_norm_backward",
            "moe_w4_linear")


# ----------------------------------------------------------------------------- arguments
def _tensor(t: Optional[torch.Tensor], name: str, shape, dtype=torch.bfloat16) -> Optional[int]:
    """The device pointer of a tensor that is what the call takes it for; None for None."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(x: torch.Tensor, width: int, name: str = "x") -> int:
    if x.dim() != 2 or x.shape[1] != width:
        raise ValueError(f"{name} must have shape (T, {width}), not {tuple(x.shape)}")
    return _tokens(x.shape[0])


def _tokens(T: int) -> int:
    """T as the library's int32 takes it: ctypes would drop what does not fit."""
    if T >= 1 << 31:
        raise ValueError(f"{T} tokens are more than the library's sizes hold")
    return T


def _bytes(t: Optional[torch.Tensor], name: str):
    """(pointer, size) of a byte buffer."""
    if t is None:
        return None, 0
    if not t.is_cuda or t.dtype != torch.uint8 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of torch.uint8")
    return t.data_ptr(), t.numel()


def _one_device(x: torch.Tensor, *others) -> None:
    for t in others:
        if t is not None and t.device != x.device:
            raise ValueError(f"tensors on {x.device} and {t.device}")


def _current_stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# The same handle without the Stream object around it, 0.1 us instead of 2, where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

# The current device's index; torch's own function without its check for initialisation, where
# torch has it (a CUDA tensor exists by then).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _current_handle(device: torch.device) -> int:
    return _raw_stream(device.index) if _raw_stream is not None else _current_stream(device)


def _stream_object(stream, device: torch.device):
    """What a caller gives as `stream` (a torch stream, or a cudaStream_t's value) as torch's
    object; None stays None."""
    if stream is None:
        return None
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != device:
            raise ValueError(f"tensors on {device} and a stream of {stream.device}")
        return stream
    handle = int(getattr(stream, "cuda_stream", stream))
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


_here = contextlib.nullcontext()


def _allocating_on(stream):
    """What is allocated inside belongs to `stream` (None: the current one), where it is used:
    memory that the current stream has freed but still works on is not handed out there."""
    return _here if stream is None else torch.cuda.stream(stream)


class BoundCall:
    """A library call with its arguments marshalled once.  Each call enqueues the same work
    on the same buffers (their contents are read when it runs) on the stream given to
    ``bind_*``, or, where none was given, on torch's current stream of that moment, and
    returns the same output tensors.  It runs on the tensors' device, whichever is current.
    The configuration and the tensors are those of the moment it was bound (a field of ``w``
    or ``grads`` that is replaced later does not count).  The tensors stay alive as long as
    the object, and their memory until the streams that it was called on are done with it."""

    __slots__ = ("_fn", "_args", "_out", "_keep", "_where", "_device", "_stream", "_tensors", "_here", "_seen", "_only")

    def __init__(self, where, args, out, keep, tensors, device, stream):
        self._fn, self._where = getattr(_lib, where), where
        self._args, self._out, self._keep = args, out, (keep, stream)
        self._tensors = [t for t in tensors if t is not None]
        self._device = device.index
        self._only = torch.cuda.device_count() == 1   # then it is the current one
        self._stream = None if stream is None else stream.cuda_stream
        # streams whose work the allocator knows to use the tensors: the current one owns
        # them, or, beside one that is given, is where the caller will use the outputs
        self._here = _current_handle(device)
        self._seen = {self._here}
        if stream is not None and self._stream != self._here:
            self._record(self._stream, stream)
            for t in self._tensors:
                t.record_stream(torch.cuda.current_stream(device))

    def _record(self, handle, stream):
        for t in self._tensors:
            t.record_stream(stream)
        self._seen.add(handle)

    def __call__(self):
        stream = self._stream
        if stream is None:
            stream = (_raw_stream or _current_stream)(self._device)
            if stream != self._here and stream not in self._seen:
                self._record(stream, torch.cuda.current_stream(self._device))
        if self._only or _current_device() == self._device:
            status = self._fn(*self._args, stream)
        else:   # the library launches on the current device
            with torch.cuda.device(self._device):
                status = self._fn(*self._args, stream)
        if status != MOE_OK:
            raise MoeError(status, self._where)
        return self._out


def _ref(struct):
    return ctypes.cast(ctypes.pointer(struct), _P)


def _own(cfg):
    """The configuration as it is now: sizes that change after a call's tensors were checked
    would send its kernels past their ends."""
    return type(cfg).from_buffer_copy(cfg)


# ----------------------------------------------------------------------------- gated FFN
def glu_cfg(d_model: int, ff: int, act: int = ACT_SWIGLU, glu_limit: float = 7.0, glu_alpha: float = 1.702) -> GluCfg:
    return GluCfg(d_model=d_model, ff=ff, act=act, glu_limit=glu_limit, glu_alpha=glu_alpha)


@dataclasses.dataclass
class GluWeights:
    gate: torch.Tensor    # bf16 [ff, d]
    up: torch.Tensor      # bf16 [ff, d]
    down: torch.Tensor    # bf16 [d, ff]


@dataclasses.dataclass
class GluGrads:
    gate: Optional[torch.Tensor]    # bf16, shaped as the weights; None: not computed
    up: Optional[torch.Tensor]
    down: Optional[torch.Tensor]


def _buffer(fn: str, cfg, T: int, device) -> torch.Tensor:
    device = torch.device(device or "cuda")
    # sizes may depend on the GPU: those of the one that the buffer is for
    with torch.cuda.device(device) if device.type == "cuda" else _here:
        n = int(getattr(_lib, fn)(ctypes.byref(cfg), _tokens(T)))
    if n == 0:
        raise MoeError(-1, fn)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_glu_workspace_bytes(cfg: GluCfg, T: int) -> int:
    return int(_lib.moe_glu_workspace_bytes(ctypes.byref(cfg), _tokens(T)))


def moe_glu_saved_bytes(cfg: GluCfg, T: int) -> int:
    return int(_lib.moe_glu_saved_bytes(ctypes.byref(cfg), _tokens(T)))


def glu_workspace(cfg: GluCfg, T: int, device=None) -> torch.Tensor:
    """A device byte buffer of moe_glu_workspace_bytes(cfg, T), for forward and backward."""
    return _buffer("moe_glu_workspace_bytes", cfg, T, device)


def glu_saved(cfg: GluCfg, T: int, device=None) -> torch.Tensor:
    """A device byte buffer for what a training forward pass leaves to its backward pass."""
    return _buffer("moe_glu_saved_bytes", cfg, T, device)


def _glu_weights(cfg: GluCfg, w: GluWeights) -> _Three:
    up = (cfg.ff, cfg.d_model)
    return _Three(_tensor(w.gate, "w.gate", up), _tensor(w.up, "w.up", up),
                  _tensor(w.down, "w.down", (cfg.d_model, cfg.ff)))


def bind_glu_forward(cfg: GluCfg, x: torch.Tensor, w: GluWeights, saved=None, y=None, ws=None,
                     stream=None) -> BoundCall:
    cfg, T, stream = _own(cfg), _rows(x, cfg.d_model), _stream_object(stream, x.device)
    with _allocating_on(stream):
        y = torch.empty_like(x) if y is None else y
        ws = glu_workspace(cfg, T, x.device) if ws is None else ws
    tensors = (x, w.gate, w.up, w.down, saved, y, ws)
    _one_device(*tensors)
    shape, keep = (T, cfg.d_model), (cfg, x, w, saved, y, ws, _glu_weights(cfg, w))
    args = (_ref(cfg), _tensor(x, "x", shape), T, _ref(keep[-1]), _tensor(y, "y", shape),
            *_bytes(saved, "saved"), *_bytes(ws, "ws"))
    return BoundCall("moe_glu_forward", args, y, keep, tensors, x.device, stream)


def moe_glu_forward(cfg: GluCfg, x: torch.Tensor, w: GluWeights, saved=None, y=None, ws=None,
                    stream=None) -> torch.Tensor:
    """y [T, d] bf16 of the gated FFN.  saved (glu_saved): kept for moe_glu_backward."""
    return bind_glu_forward(cfg, x, w, saved, y, ws, stream)()


def bind_glu_backward(cfg: GluCfg, x: torch.Tensor, w: GluWeights, saved: torch.Tensor, dy: torch.Tensor, dx=None,
                      grads: Optional[GluGrads] = None, ws=None, need_dx: bool = True, stream=None) -> BoundCall:
    cfg, T, stream = _own(cfg), _rows(x, cfg.d_model), _stream_object(stream, x.device)
    with _allocating_on(stream):
        if need_dx and dx is None:
            dx = torch.empty_like(x)
        if grads is None:
            grads = GluGrads(*(torch.empty_like(t) for t in (w.gate, w.up, w.down)))
        ws = glu_workspace(cfg, T, x.device) if ws is None else ws
    tensors = (x, w.gate, w.up, w.down, saved, dy, dx, grads.gate, grads.up, grads.down, ws)
    _one_device(*tensors)
    shape, up = (T, cfg.d_model), (cfg.ff, cfg.d_model)
    g = _Three(_tensor(grads.gate, "grads.gate", up), _tensor(grads.up, "grads.up", up),
               _tensor(grads.down, "grads.down", (cfg.d_model, cfg.ff)))
    keep = (cfg, x, w, saved, dy, dx, grads, ws, _glu_weights(cfg, w), g)
    args = (_ref(cfg), _tensor(x, "x", shape), T, _ref(keep[-2]), *_bytes(saved, "saved"),
            _tensor(dy, "dy", shape), _tensor(dx, "dx", shape), _ref(g), *_bytes(ws, "ws"))
    return BoundCall("moe_glu_backward", args, (dx, grads), keep, tensors, x.device, stream)


def moe_glu_backward(cfg: GluCfg, x: torch.Tensor, w: GluWeights, saved: torch.Tensor, dy: torch.Tensor, dx=None,
                     grads: Optional[GluGrads] = None, ws=None, need_dx: bool = True, stream=None):
    """(dx, GluGrads) from dy and the saved buffer of the forward pass on the same x and w."""
    return bind_glu_backward(cfg, x, w, saved, dy, dx, grads, ws, need_dx, stream)()


# ----------------------------------------------------------------------------- norms
def norm_cfg(d_model: int, eps: float = 1e-6, residual_scale: float = 1.0, branch_scale: float = 1.0) -> NormCfg:
    return NormCfg(d_model=d_model, eps=eps, residual_scale=residual_scale, branch_scale=branch_scale)


@dataclasses.dataclass
class NormGrads:
    dx: Optional[torch.Tensor] = None         # bf16 [T, d]
    dbranch: Optional[torch.Tensor] = None    # bf16 [T, d]
    dgate: Optional[torch.Tensor] = None      # fp32 [T]
    dpost_w: Optional[torch.Tensor] = None    # fp32 [d]
    dpre_w: Optional[torch.Tensor] = None     # fp32 [d]


def _norm_inputs(cfg: NormCfg, T: int, x, branch, post_w, gate, pre_w) -> _Five:
    shape, d = (T, cfg.d_model), (cfg.d_model,)
    return _Five(_tensor(x, "x", shape), _tensor(branch, "branch", shape), _tensor(post_w, "post_w", d),
                 _tensor(gate, "gate", (T,), torch.float32), _tensor(pre_w, "pre_w", d))


def bind_block_norm_forward(cfg: NormCfg, x: torch.Tensor, branch=None, post_w=None, gate=None, pre_w=None, y=None,
                            a=None, stream=None) -> BoundCall:
    cfg, T, stream = _own(cfg), _rows(x, cfg.d_model), _stream_object(stream, x.device)
    with _allocating_on(stream):
        if branch is not None and y is None:
            y = torch.empty_like(x)
        if pre_w is not None and a is None:
            a = torch.empty_like(x)
    tensors = (x, branch, post_w, gate, pre_w, y, a)
    _one_device(*tensors)
    shape, keep = (T, cfg.d_model), (cfg, x, branch, post_w, gate, pre_w, y, a,
                                     _norm_inputs(cfg, T, x, branch, post_w, gate, pre_w))
    args = (_ref(cfg), _ref(keep[-1]), T, _tensor(y, "y", shape), _tensor(a, "a", shape))
    return BoundCall("moe_block_norm_forward", args, (y, a), keep, tensors, x.device, stream)


def moe_block_norm_forward(cfg: NormCfg, x: torch.Tensor, branch=None, post_w=None, gate=None, pre_w=None, y=None,
                           a=None, stream=None):
    """(y, a): y = residual_scale x + branch_scale sigmoid(gate) norm(branch) post_w (None
    without branch), a = norm(y) pre_w (None without pre_w)."""
    return bind_block_norm_forward(cfg, x, branch, post_w, gate, pre_w, y, a, stream)()


def moe_block_norm_workspace_bytes(cfg: NormCfg, T: int) -> int:
    return int(_lib.moe_block_norm_workspace_bytes(ctypes.byref(cfg), _tokens(T)))


def block_norm_workspace(cfg: NormCfg, T: int, device=None) -> torch.Tensor:
    return _buffer("moe_block_norm_workspace_bytes", cfg, T, device)


def bind_block_norm_backward(cfg: NormCfg, x: torch.Tensor, dy=None, da=None, branch=None, post_w=None, gate=None,
                             pre_w=None, grads: Optional[NormGrads] = None, ws=None, stream=None) -> BoundCall:
    cfg, T, dev = _own(cfg), _rows(x, cfg.d_model), x.device
    stream = _stream_object(stream, dev)

    def f32(n):
        return torch.empty(n, dtype=torch.float32, device=dev)

    with _allocating_on(stream):
        if grads is None:
            grads = NormGrads(torch.empty_like(x), None if branch is None else torch.empty_like(x),
                              None if gate is None else f32(T), None if post_w is None else f32(cfg.d_model),
                              None if pre_w is None else f32(cfg.d_model))
        ws = block_norm_workspace(cfg, T, dev) if ws is None else ws
    tensors = (x, dy, da, branch, post_w, gate, pre_w, grads.dx, grads.dbranch, grads.dgate, grads.dpost_w,
               grads.dpre_w, ws)
    _one_device(*tensors)
    shape, d = (T, cfg.d_model), (cfg.d_model,)
    g = _Five(_tensor(grads.dx, "grads.dx", shape), _tensor(grads.dbranch, "grads.dbranch", shape),
              _tensor(grads.dgate, "grads.dgate", (T,), torch.float32),
              _tensor(grads.dpost_w, "grads.dpost_w", d, torch.float32),
              _tensor(grads.dpre_w, "grads.dpre_w", d, torch.float32))
    keep = (cfg, x, dy, da, branch, post_w, gate, pre_w, grads, ws,
            _norm_inputs(cfg, T, x, branch, post_w, gate, pre_w), g)
    args = (_ref(cfg), _ref(keep[-2]), T, _tensor(dy, "dy", shape), _tensor(da, "da", shape), _ref(g),
            *_bytes(ws, "ws"))
    return BoundCall("moe_block_norm_backward", args, grads, keep, tensors, dev, stream)


def moe_block_norm_backward(cfg: NormCfg, x: torch.Tensor, dy=None, da=None, branch=None, post_w=None, gate=None,
                            pre_w=None, grads: Optional[NormGrads] = None, ws=None, stream=None) -> NormGrads:
    """Gradients of moe_block_norm_forward from dy (of y) and da (of a), either None for zero."""
    return bind_block_norm_backward(cfg, x, dy, da, branch, post_w, gate, pre_w, grads, ws, stream)()


# ----------------------------------------------------------------------------- 4-bit linear
def w4_cfg(n_in: int, n_out: int, group: int = 128, glu: bool = False, act: int = ACT_SWIGLU, glu_limit: float = 7.0,
           glu_alpha: float = 1.702) -> W4Cfg:
    return W4Cfg(n_in=n_in, n_out=n_out, group=group, glu=int(glu), act=act, glu_limit=glu_limit, glu_alpha=glu_alpha)


@dataclasses.dataclass
class W4Weights:
    codes: torch.Tensor                     # u8 [rows, n_in / 2], low half = even input
    scales: torch.Tensor                    # bf16 [rows, n_in / group]
    zeros: Optional[torch.Tensor] = None    # u8 [rows, n_in / group]; None: 8


def w4_quantize(w: torch.Tensor, group: int = 128, zeros: bool = True) -> W4Weights:
    """Rounds a weight matrix [rows, n_in] to 4-bit codes with a scale (and, with zeros, a
    zero point) per `group` inputs.  Made once per matrix, on whichever device holds it."""
    if w.dim() != 2 or w.shape[1] % group:
        raise ValueError(f"w must have shape (rows, a multiple of {group}), not {tuple(w.shape)}")
    v = w.float().reshape(w.shape[0], -1, group)
    if zeros:
        lo, hi = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
        s = ((hi - lo) / 15).to(torch.bfloat16)
    else:
        s = (v.abs().amax(2) / 7).to(torch.bfloat16)
    s = torch.where(s == 0, torch.ones_like(s), s)
    z = (-lo / s.float()).round().clamp(0, 15) if zeros else torch.full_like(s, 8, dtype=torch.float32)
    q = ((v / s.float()[:, :, None]).round() + z[:, :, None]).clamp(0, 15).to(torch.uint8).reshape(w.shape)
    return W4Weights((q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), s, z.to(torch.uint8) if zeros else None)


def bind_w4_linear(cfg: W4Cfg, x: torch.Tensor, w: W4Weights, y=None, stream=None) -> BoundCall:
    cfg, T, stream = _own(cfg), _rows(x, cfg.n_in), _stream_object(stream, x.device)
    with _allocating_on(stream):
        y = torch.empty((T, cfg.n_out), dtype=torch.bfloat16, device=x.device) if y is None else y
    tensors = (x, w.codes, w.scales, w.zeros, y)
    _one_device(*tensors)
    rows, groups = cfg.n_out * (2 if cfg.glu else 1), cfg.n_in // max(cfg.group, 1)
    keep = (cfg, x, w, y, _Three(_tensor(w.codes, "w.codes", (rows, cfg.n_in // 2), torch.uint8),
                                 _tensor(w.scales, "w.scales", (rows, groups)),
                                 _tensor(w.zeros, "w.zeros", (rows, groups), torch.uint8)))
    args = (_ref(cfg), _tensor(x, "x", (T, cfg.n_in)), T, _ref(keep[-1]), _tensor(y, "y", (T, cfg.n_out)))
    return BoundCall("moe_w4_linear", args, y, keep, tensors, x.device, stream)


def moe_w4_linear(cfg: W4Cfg, x: torch.Tensor, w: W4Weights, y=None, stream=None) -> torch.Tensor:
    """y [T, n_out] bf16 of the linear layer with 4-bit weights (cfg.glu: with its gate)."""
    return bind_w4_linear(cfg, x, w, y, stream)()
