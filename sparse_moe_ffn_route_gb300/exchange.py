"""The exchange around a sparse layer's experts -- Python binding of include/moe_exchange.h.

Tokens sorted by expert (``moe_dispatch_forward``) and the experts' rows back at their tokens with
the routing weights applied (``moe_combine_forward``), with the gradients of both
(``moe_dispatch_backward``, ``moe_combine_backward``).  Checks of arguments, allocation, streams
and the ``bind_*`` twins are those of the dense block (``block``)."""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from .block import (BoundCall, _allocating_on, _buffer, _bytes, _declare, _I, _lib, _one_device, _own, _P, _ref, _rows,
                    _S, _stream_object, _tensor, _tokens)

ROWS_BF16, ROWS_E4M3 = 0, 1
_ROW_TYPES = {ROWS_BF16: torch.bfloat16, ROWS_E4M3: torch.float8_e4m3fn}


class ExchangeCfg(ctypes.Structure):
    """moe_exchange_cfg_t."""
    _fields_ = [("d_model", _I), ("n_experts", _I), ("top_k", _I), ("format", _I), ("reserved", _I * 4)]


_declare("moe_dispatch_workspace_bytes", [_P, _I], _S)
_declare("moe_dispatch_forward", [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _S, _P])
_declare("moe_dispatch_backward", [_P, _P, _P, _I, _P, _P])
_declare("moe_combine_forward", [_P, _P, _P, _P, _P, _I, _P, _P])
_declare("moe_combine_backward", [_P, _P, _P, _P, _P, _I, _P, _P, _P])
EXPORTED = ("moe_dispatch_workspace_bytes", "moe_dispatch_forward", "moe_dispatch_backward", "moe_combine_forward",
            "moe_combine_backward")


def exchange_cfg(d_model: int, n_experts: int, top_k: int, fmt: int = ROWS_BF16) -> ExchangeCfg:
    return ExchangeCfg(d_model=d_model, n_experts=n_experts, top_k=top_k, format=fmt)


@dataclasses.dataclass
class Dispatched:
    offsets: torch.Tensor                     # int32 [E + 1]: expert e's rows are offsets[e] .. offsets[e + 1] - 1
    rows: torch.Tensor                        # int32 [T, k]: the row of each choice, -1 for none
    xs: Optional[torch.Tensor] = None         # bf16 or e4m3 [T k, d], sorted by expert
    xs_scale: Optional[torch.Tensor] = None   # fp32 [T k], e4m3


def moe_dispatch_workspace_bytes(cfg: ExchangeCfg, T: int) -> int:
    return int(_lib.moe_dispatch_workspace_bytes(ctypes.byref(cfg), _tokens(T)))


def dispatch_workspace(cfg: ExchangeCfg, T: int, device=None) -> torch.Tensor:
    """A device byte buffer of moe_dispatch_workspace_bytes(cfg, T)."""
    return _buffer("moe_dispatch_workspace_bytes", cfg, T, device)


def bind_dispatch_forward(cfg: ExchangeCfg, x: Optional[torch.Tensor], topk_ids: torch.Tensor, x_scale=None,
                          out: Optional[Dispatched] = None, ws=None, stream=None) -> BoundCall:
    cfg, T = _own(cfg), _rows(topk_ids, cfg.top_k, "topk_ids")
    dev, kind = topk_ids.device, _ROW_TYPES.get(cfg.format, torch.bfloat16)
    stream = _stream_object(stream, dev)
    S, eight = T * cfg.top_k, x is not None and cfg.format == ROWS_E4M3
    if eight and x_scale is None:
        raise ValueError("x_scale is needed with rows in 8 bits")
    with _allocating_on(stream):
        if out is None:
            out = Dispatched(torch.empty(cfg.n_experts + 1, dtype=torch.int32, device=dev),
                             torch.empty((T, cfg.top_k), dtype=torch.int32, device=dev),
                             None if x is None else torch.empty((S, cfg.d_model), dtype=kind, device=dev),
                             torch.empty(S, dtype=torch.float32, device=dev) if eight else None)
        ws = dispatch_workspace(cfg, T, dev) if ws is None else ws
    out = dataclasses.replace(out)
    tensors = (topk_ids, x, x_scale, out.offsets, out.rows, out.xs, out.xs_scale, ws)
    _one_device(*tensors)
    args = (_ref(cfg), _tensor(topk_ids, "topk_ids", (T, cfg.top_k), torch.int32),
            _tensor(x, "x", (T, cfg.d_model), kind), _tensor(x_scale, "x_scale", (T,), torch.float32), T,
            _tensor(out.offsets, "out.offsets", (cfg.n_experts + 1,), torch.int32),
            _tensor(out.rows, "out.rows", (T, cfg.top_k), torch.int32),
            _tensor(out.xs, "out.xs", (S, cfg.d_model), kind),
            _tensor(out.xs_scale, "out.xs_scale", (S,), torch.float32), *_bytes(ws, "ws"))
    return BoundCall("moe_dispatch_forward", args, out, (cfg, tensors), tensors, dev, stream)


def moe_dispatch_forward(cfg: ExchangeCfg, x: Optional[torch.Tensor], topk_ids: torch.Tensor, x_scale=None,
                         out: Optional[Dispatched] = None, ws=None, stream=None) -> Dispatched:
    """The slots of topk_ids int32 [T, k] sorted by expert, and x's rows copied along (x None: the
    sort alone).  Rows behind out.offsets[E] are left as they are."""
    return bind_dispatch_forward(cfg, x, topk_ids, x_scale, out, ws, stream)()


def bind_dispatch_backward(cfg: ExchangeCfg, dxs: torch.Tensor, rows: torch.Tensor, dx=None, stream=None) -> BoundCall:
    cfg, T, stream = _own(cfg), _rows(rows, cfg.top_k, "rows"), _stream_object(stream, rows.device)
    with _allocating_on(stream):
        dx = torch.empty((T, cfg.d_model), dtype=torch.bfloat16, device=rows.device) if dx is None else dx
    tensors = (dxs, rows, dx)
    _one_device(*tensors)
    args = (_ref(cfg), _tensor(dxs, "dxs", (T * cfg.top_k, cfg.d_model)),
            _tensor(rows, "rows", (T, cfg.top_k), torch.int32), T, _tensor(dx, "dx", (T, cfg.d_model)))
    return BoundCall("moe_dispatch_backward", args, dx, (cfg, tensors), tensors, rows.device, stream)


def moe_dispatch_backward(cfg: ExchangeCfg, dxs: torch.Tensor, rows: torch.Tensor, dx=None, stream=None) -> torch.Tensor:
    """dx [T, d] bf16: the sum of a token's rows of dxs [T k, d]."""
    return bind_dispatch_backward(cfg, dxs, rows, dx, stream)()


def bind_combine_forward(cfg: ExchangeCfg, z: torch.Tensor, rows: torch.Tensor, w=None, residual=None, y=None,
                         stream=None) -> BoundCall:
    cfg, T, stream = _own(cfg), _rows(rows, cfg.top_k, "rows"), _stream_object(stream, rows.device)
    with _allocating_on(stream):
        y = torch.empty((T, cfg.d_model), dtype=torch.bfloat16, device=rows.device) if y is None else y
    tensors = (z, rows, w, residual, y)
    _one_device(*tensors)
    choices, shape = (T, cfg.top_k), (T, cfg.d_model)
    args = (_ref(cfg), _tensor(z, "z", (T * cfg.top_k, cfg.d_model)), _tensor(rows, "rows", choices, torch.int32),
            _tensor(w, "w", choices, torch.float32), _tensor(residual, "residual", shape), T, _tensor(y, "y", shape))
    return BoundCall("moe_combine_forward", args, y, (cfg, tensors), tensors, rows.device, stream)


def moe_combine_forward(cfg: ExchangeCfg, z: torch.Tensor, rows: torch.Tensor, w=None, residual=None, y=None,
                        stream=None) -> torch.Tensor:
    """y [T, d] bf16 = residual + the sum of a token's rows of z [T k, d], weighted by w fp32 [T, k]
    (None: 1).  y may be residual's tensor."""
    return bind_combine_forward(cfg, z, rows, w, residual, y, stream)()


def bind_combine_backward(cfg: ExchangeCfg, dy: torch.Tensor, z: Optional[torch.Tensor], rows: torch.Tensor,
                          w: torch.Tensor, dz=None, dw=None, need_dz: bool = True, need_dw: bool = True,
                          stream=None) -> BoundCall:
    cfg, T, dev = _own(cfg), _rows(rows, cfg.top_k, "rows"), rows.device
    stream = _stream_object(stream, dev)
    S, choices = T * cfg.top_k, (T, cfg.top_k)
    with _allocating_on(stream):
        if need_dz and dz is None:
            dz = torch.empty((S, cfg.d_model), dtype=torch.bfloat16, device=dev)
        if need_dw and dw is None:
            dw = torch.empty(choices, dtype=torch.float32, device=dev)
    tensors = (dy, z, rows, w, dz, dw)
    _one_device(*tensors)
    args = (_ref(cfg), _tensor(dy, "dy", (T, cfg.d_model)), _tensor(z, "z", (S, cfg.d_model)),
            _tensor(rows, "rows", choices, torch.int32), _tensor(w, "w", choices, torch.float32), T,
            _tensor(dz, "dz", (S, cfg.d_model)), _tensor(dw, "dw", choices, torch.float32))
    return BoundCall("moe_combine_backward", args, (dz, dw), (cfg, tensors), tensors, dev, stream)


def moe_combine_backward(cfg: ExchangeCfg, dy: torch.Tensor, z: Optional[torch.Tensor], rows: torch.Tensor,
                         w: torch.Tensor, dz=None, dw=None, need_dz: bool = True, need_dw: bool = True, stream=None):
    """(dz, dw) from dy: dz bf16 [T k, d] by row (rows without a slot are left as they are), dw fp32
    [T, k], for which z is needed.  The residual's gradient is dy."""
    return bind_combine_backward(cfg, dy, z, rows, w, dz, dw, need_dz, need_dw, stream)()
