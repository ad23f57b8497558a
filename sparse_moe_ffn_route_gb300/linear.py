"""The linear layer with bias, activation and residual in its epilogue -- Python binding of
include/moe_linear.h.

``moe_linear_forward`` and ``moe_linear_backward`` in bf16; the forward pass also with operands in
8 bits (torch.float8_e4m3fn with an fp32 scale per row), which ``moe_block_norm_quant`` writes and
``w8_quantize`` makes of weights.  Checks of arguments, allocation, streams and the ``bind_*``
twins are those of the dense block (``block``)."""
from __future__ import annotations

import ctypes
import dataclasses
import math
from typing import Optional

import torch

from .block import (BoundCall, NormCfg, _allocating_on, _buffer, _bytes, _declare, _I, _lib, _norm_inputs, _one_device,
                    _own, _P, _ref, _rows, _S, _stream_object, _tensor, _Three, _tokens)

LINEAR_BF16, LINEAR_E4M3 = 0, 1
LINEAR_NONE, LINEAR_SILU, LINEAR_GELU, LINEAR_GELU_TANH = 0, 1, 2, 3
E4M3_MAX, LEAST_SCALE = 448.0, 2.0 ** -126
_TYPES = {LINEAR_BF16: torch.bfloat16, LINEAR_E4M3: torch.float8_e4m3fn}


class LinearCfg(ctypes.Structure):
    """moe_linear_cfg_t."""
    _fields_ = [("n_in", _I), ("n_out", _I), ("format", _I), ("glu", _I), ("act", _I), ("glu_limit", ctypes.c_float),
                ("glu_alpha", ctypes.c_float), ("reserved", _I * 5)]


class _Two(ctypes.Structure):
    """moe_linear_grads_t."""
    _fields_ = [("p0", _P), ("p1", _P)]


_declare("moe_block_norm_quant", [_P, _P, _I, _P, _P, _P, _P])
_declare("moe_linear_workspace_bytes", [_P, _I], _S)
_declare("moe_linear_forward", [_P, _P, _P, _I, _P, _P, _P, _P, _P, _S, _P])
_declare("moe_linear_backward", [_P, _P, _I, _P, _P, _P, _P, _P, _P, _S, _P])
EXPORTED = ("moe_block_norm_quant", "moe_linear_workspace_bytes", "moe_linear_forward", "moe_linear_backward")


# ----------------------------------------------------------------------------- 8 bits
def w8_quantize(w: torch.Tensor):
    """(codes, scale): a matrix [rows, n_in] as torch.float8_e4m3fn with an fp32 scale per row.
    A NaN does not count for its row's scale.  Made once per weight matrix, on whichever device holds it."""
    if w.dim() != 2:
        raise ValueError(f"w must have two dimensions, not {w.dim()}")
    v = w.float()
    # (torch would multiply by the rounded reciprocal of a plain number)
    top = v.abs().nan_to_num(nan=0.0, posinf=math.inf).amax(1) if w.shape[1] else v.new_zeros(w.shape[0])
    scale = (top / torch.full_like(top, E4M3_MAX)).clamp(min=LEAST_SCALE)
    return (v / scale[:, None]).to(torch.float8_e4m3fn), scale


def bind_block_norm_quant(cfg: NormCfg, x: torch.Tensor, branch=None, post_w=None, gate=None, pre_w=None, y=None,
                          q=None, scale=None, stream=None) -> BoundCall:
    cfg, T, stream = _own(cfg), _rows(x, cfg.d_model), _stream_object(stream, x.device)
    with _allocating_on(stream):
        if branch is not None and y is None:
            y = torch.empty_like(x)
        q = torch.empty((T, cfg.d_model), dtype=torch.float8_e4m3fn, device=x.device) if q is None else q
        scale = torch.empty(T, dtype=torch.float32, device=x.device) if scale is None else scale
    tensors = (x, branch, post_w, gate, pre_w, y, q, scale)
    _one_device(*tensors)
    shape, inputs = (T, cfg.d_model), _norm_inputs(cfg, T, x, branch, post_w, gate, pre_w)
    args = (_ref(cfg), _ref(inputs), T, _tensor(y, "y", shape), _tensor(q, "q", shape, torch.float8_e4m3fn),
            _tensor(scale, "scale", (T,), torch.float32))
    return BoundCall("moe_block_norm_quant", args, (y, q, scale), (cfg, tensors, inputs), tensors, x.device, stream)


def moe_block_norm_quant(cfg: NormCfg, x: torch.Tensor, branch=None, post_w=None, gate=None, pre_w=None, y=None,
                         q=None, scale=None, stream=None):
    """(y, q, scale): moe_block_norm_forward with a in 8 bits, a = scale q row by row (y None without
    branch).  Without pre_w a is y (or x), so that x alone is taken to 8 bits."""
    return bind_block_norm_quant(cfg, x, branch, post_w, gate, pre_w, y, q, scale, stream)()


# ----------------------------------------------------------------------------- linear layer
def linear_cfg(n_in: int, n_out: int, act: int = LINEAR_NONE, glu: bool = False, fmt: int = LINEAR_BF16,
               glu_limit: float = 7.0, glu_alpha: float = 1.702) -> LinearCfg:
    """act: LINEAR_*, or with glu (twice the weight rows, gate rows first) ACT_*."""
    return LinearCfg(n_in=n_in, n_out=n_out, format=fmt, glu=int(glu), act=act, glu_limit=glu_limit, glu_alpha=glu_alpha)


@dataclasses.dataclass
class LinearWeights:
    w: torch.Tensor                         # bf16 or e4m3 [rows, n_in]
    bias: Optional[torch.Tensor] = None     # bf16 [rows]
    scale: Optional[torch.Tensor] = None    # fp32 [rows], e4m3


@dataclasses.dataclass
class LinearGrads:
    w: Optional[torch.Tensor]               # bf16 [n_out, n_in]; None: not computed
    bias: Optional[torch.Tensor]            # bf16 [n_out]


def _weights(cfg: LinearCfg, w: LinearWeights) -> _Three:
    rows = cfg.n_out * (2 if cfg.glu else 1)
    kind = _TYPES.get(cfg.format, torch.bfloat16)
    if cfg.format == LINEAR_E4M3 and w.scale is None:
        raise ValueError("w.scale is needed with weights in 8 bits")
    return _Three(_tensor(w.w, "w.w", (rows, cfg.n_in), kind), _tensor(w.scale, "w.scale", (rows,), torch.float32),
                  _tensor(w.bias, "w.bias", (rows,)))


def moe_linear_workspace_bytes(cfg: LinearCfg, T: int) -> int:
    return int(_lib.moe_linear_workspace_bytes(ctypes.byref(cfg), _tokens(T)))


def linear_workspace(cfg: LinearCfg, T: int, device=None) -> torch.Tensor:
    """A device byte buffer of moe_linear_workspace_bytes(cfg, T), for forward and backward."""
    return _buffer("moe_linear_workspace_bytes", cfg, T, device)


def linear_pre(cfg: LinearCfg, T: int, device=None) -> torch.Tensor:
    """A buffer for what a training forward pass leaves to its backward pass (not needed without
    an activation)."""
    return torch.empty((_tokens(T), cfg.n_out), dtype=torch.bfloat16, device=device or "cuda")


def bind_linear_forward(cfg: LinearCfg, x: torch.Tensor, w: LinearWeights, x_scale=None, residual=None, pre=None,
                        y=None, ws=None, stream=None) -> BoundCall:
    cfg, T, stream = _own(cfg), _rows(x, cfg.n_in), _stream_object(stream, x.device)
    if cfg.format == LINEAR_E4M3 and x_scale is None:
        raise ValueError("x_scale is needed with x in 8 bits")
    with _allocating_on(stream):
        y = torch.empty((T, cfg.n_out), dtype=torch.bfloat16, device=x.device) if y is None else y
        ws = linear_workspace(cfg, T, x.device) if ws is None else ws
    tensors = (x, x_scale, w.w, w.scale, w.bias, residual, pre, y, ws)
    _one_device(*tensors)
    shape, weights = (T, cfg.n_out), _weights(cfg, w)
    args = (_ref(cfg), _tensor(x, "x", (T, cfg.n_in), _TYPES.get(cfg.format, torch.bfloat16)),
            _tensor(x_scale, "x_scale", (T,), torch.float32), T, _ref(weights), _tensor(residual, "residual", shape),
            _tensor(y, "y", shape), _tensor(pre, "pre", shape), *_bytes(ws, "ws"))
    return BoundCall("moe_linear_forward", args, y, (cfg, tensors, weights), tensors, x.device, stream)


def moe_linear_forward(cfg: LinearCfg, x: torch.Tensor, w: LinearWeights, x_scale=None, residual=None, pre=None,
                       y=None, ws=None, stream=None) -> torch.Tensor:
    """y [T, n_out] bf16 = act(x W^T + bias) + residual.  pre (linear_pre): kept for
    moe_linear_backward.  y may be residual's tensor."""
    return bind_linear_forward(cfg, x, w, x_scale, residual, pre, y, ws, stream)()


def bind_linear_backward(cfg: LinearCfg, x: torch.Tensor, w: LinearWeights, dy: torch.Tensor, pre=None, dx=None,
                         grads: Optional[LinearGrads] = None, ws=None, need_dx: bool = True, stream=None) -> BoundCall:
    cfg, T, stream = _own(cfg), _rows(x, cfg.n_in), _stream_object(stream, x.device)
    with _allocating_on(stream):
        if need_dx and dx is None:
            dx = torch.empty_like(x)
        if grads is None:
            grads = LinearGrads(torch.empty_like(w.w), None if w.bias is None else torch.empty_like(w.bias))
        ws = linear_workspace(cfg, T, x.device) if ws is None else ws
    tensors = (x, w.w, w.bias, w.scale, dy, pre, dx, grads.w, grads.bias, ws)
    _one_device(*tensors)
    shape, weights = (T, cfg.n_out), _weights(cfg, w)
    g = _Two(_tensor(grads.w, "grads.w", (cfg.n_out, cfg.n_in)), _tensor(grads.bias, "grads.bias", (cfg.n_out,)))
    args = (_ref(cfg), _tensor(x, "x", (T, cfg.n_in)), T, _ref(weights), _tensor(pre, "pre", shape),
            _tensor(dy, "dy", shape), _tensor(dx, "dx", (T, cfg.n_in)), _ref(g), *_bytes(ws, "ws"))
    out = (dx, LinearGrads(grads.w, grads.bias))
    return BoundCall("moe_linear_backward", args, out, (cfg, tensors, weights, g), tensors, x.device, stream)


def moe_linear_backward(cfg: LinearCfg, x: torch.Tensor, w: LinearWeights, dy: torch.Tensor, pre=None, dx=None,
                        grads: Optional[LinearGrads] = None, ws=None, need_dx: bool = True, stream=None):
    """(dx, LinearGrads) from dy and, with an activation, the pre of the forward pass on the same x
    and w.  The residual's gradient is dy."""
    return bind_linear_backward(cfg, x, w, dy, pre, dx, grads, ws, need_dx, stream)()
