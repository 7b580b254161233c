"""ctypes binding of the C ABI in ``include/based_ops.h`` (argument marshalling only).

The operators of a language model around the Based forward pass: the gated linear recurrence
(``based_scan_*``), the per-token group norm with an activation (``based_norm_*``) and the scaled
embedding with its gradient (``based_embed_*``). Every step runs in the CUDA kernels of
``libbased_gb300.so``; there is no fallback.

All functions launch on ``stream`` (default: the current stream of the inputs' device). What they
allocate (outputs that are not passed in, workspaces) comes from that stream's pool, so a call on a
side stream needs ordering only for its inputs and for the use of its results. Inputs may be
strided as long as their last axis has stride 1; outputs are contiguous.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import based
from .based import _check, _on_device, _stream_ptr

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
MODES = {"log": 0, "sigmoid": 1}
ACTS = {"none": 0, "silu": 1, "sigmoid": 2}
SAVE_ROWS = 64  # BASED_SCAN_SAVE_ROWS

_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    L = based.library()
    p, i, l, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    z = ctypes.c_size_t
    L.based_scan_fwd.argtypes = [p, l, l, p, l, l, i, i, i, i, i, p, p, p, p, p, p]
    L.based_scan_bwd.argtypes = [p, l, l, p, l, l, p, l, l, p, i, i, i, i, i, p, p, p, p, p, p]
    L.based_scan_step.argtypes = [p, l, p, l, i, i, i, i, i, p, p, p, p]
    L.based_norm_fwd.argtypes = [p, l, i, p, l, p, p, i, l, i, i, f, i, p, i, p]
    L.based_norm_bwd.argtypes = [p, l, p, l, i, p, l, p, p, i, l, i, i, f, i, p, p, p, p, i, p, z, p]
    L.based_norm_bwd_workspace_size.argtypes = [l, i, i]
    L.based_embed_fwd.argtypes = [p, i, p, l, l, i, i, i, f, p, p]
    L.based_embed_bwd.argtypes = [p, i, p, l, l, i, i, i, f, p, i, p, z, p]
    L.based_embed_bwd_workspace_size.argtypes = [l, i, i]
    for name in ("scan_fwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd", "embed_fwd", "embed_bwd"):
        getattr(L, "based_" + name).restype = i
    L.based_norm_bwd_workspace_size.restype = z
    L.based_embed_bwd_workspace_size.restype = z
    _lib = L
    return L


# ------------------------------------------------------------------------------------------------
# Checks
# ------------------------------------------------------------------------------------------------
def _dtype(t: torch.Tensor) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"expected a float32, bfloat16 or float16 tensor, got {t.dtype}")
    return code


def _code(table, key, what):
    code = table.get(key)
    if code is None:
        raise ValueError(f"{what} must be one of {', '.join(table)}, got {key!r}")
    return code


def _input(t: torch.Tensor, name: str, shape, dtype, dev):
    """t is a tensor of this shape and type on this device whose last axis has stride 1."""
    if t.device != dev or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the other inputs")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"the last axis of {name} must have stride 1")


def _output(t: Optional[torch.Tensor], name: str, shape, dtype, dev) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if t.device != dev or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}")
    return t


def _whole(t: Optional[torch.Tensor], name: str, shape, dtype, dev) -> Optional[int]:
    """The address of an optional contiguous input."""
    if t is None:
        return None
    if t.device != dev or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


_here = contextlib.nullcontext()


def _pool(stream: Optional[torch.cuda.Stream]):
    # allocations of a call on a side stream come from that stream's pool
    return _here if stream is None else torch.cuda.stream(stream)


def _rows(t: torch.Tensor, name: str) -> torch.Tensor:
    """t (..., C) as (R, C) without a copy."""
    if t.dim() == 2:
        return t
    try:
        return t.view(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"the leading axes of {name} must have one common stride") from None


# ------------------------------------------------------------------------------------------------
# Gated linear recurrence
# ------------------------------------------------------------------------------------------------
def based_scan_fwd(gate: torch.Tensor, x: torch.Tensor, mode: str = "sigmoid",
                   state: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                   save: bool = False, out: Optional[torch.Tensor] = None,
                   final_state: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """h_t = a_t h_{t-1} + u_t along axis 1 of gate, x (B,T,D), float32 inside.

    mode "log": a = exp(gate), u = x. mode "sigmoid": a = sigmoid(gate), u = (1 - a) x.
    ``state`` (B,D) float32 is h before the first row (default zero); ``lengths`` (B) int32 marks
    rows t >= lengths[b] as padding (zero output, state kept). Returns (h in the type of x, the last
    state (B,D) float32, the states every 64 rows that based_scan_bwd needs, or None without
    ``save``). ``final_state`` may be ``state``, to update it in place.
    """
    L = _load()
    if x.dim() != 3:
        raise ValueError("expected gate and x of shape (B,T,D)")
    dev, shape, dtype = x.device, x.shape, x.dtype
    B, T, D = shape
    code = _dtype(x)
    _input(x, "x", shape, dtype, dev)
    _input(gate, "gate", shape, dtype, dev)
    f32 = torch.float32
    with _pool(stream):
        y = _output(out, "out", shape, dtype, dev)
        last = _output(final_state, "final_state", (B, D), f32, dev)
        saved = torch.empty(B, -(-T // SAVE_ROWS), D, dtype=f32, device=dev) if save else None
    rc = _on_device(dev, L.based_scan_fwd, gate.data_ptr(), gate.stride(0), gate.stride(1), x.data_ptr(),
                    x.stride(0), x.stride(1), B, T, D, code, _code(MODES, mode, "mode"),
                    _whole(state, "state", (B, D), f32, dev), _whole(lengths, "lengths", (B,), torch.int32, dev),
                    y.data_ptr(), last.data_ptr(), _ptr(saved), _stream_ptr(dev, stream))
    _check(rc, "based_scan_fwd")
    return y, last, saved


def based_scan_bwd(gate: torch.Tensor, x: torch.Tensor, dy: torch.Tensor, saved: torch.Tensor,
                   mode: str = "sigmoid", dfinal: Optional[torch.Tensor] = None,
                   lengths: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of based_scan_fwd for the gradients dy (B,T,D) of its output and dfinal (B,D)
    float32 of its last state: (dgate, dx, dstate). ``saved`` is what the forward call returned."""
    L = _load()
    if x.dim() != 3:
        raise ValueError("expected gate, x and dy of shape (B,T,D)")
    dev, shape, dtype = x.device, x.shape, x.dtype
    B, T, D = shape
    code = _dtype(x)
    _input(x, "x", shape, dtype, dev)
    _input(gate, "gate", shape, dtype, dev)
    _input(dy, "dy", shape, dtype, dev)
    f32 = torch.float32
    if saved is None:
        raise ValueError("based_scan_bwd needs the saved states of based_scan_fwd(..., save=True)")
    with _pool(stream):
        dgate = torch.empty(shape, dtype=dtype, device=dev)
        dx = torch.empty(shape, dtype=dtype, device=dev)
        dstate = torch.empty(B, D, dtype=f32, device=dev)
    rc = _on_device(dev, L.based_scan_bwd, gate.data_ptr(), gate.stride(0), gate.stride(1), x.data_ptr(),
                    x.stride(0), x.stride(1), dy.data_ptr(), dy.stride(0), dy.stride(1),
                    _whole(saved, "saved", (B, -(-T // SAVE_ROWS), D), f32, dev), B, T, D, code,
                    _code(MODES, mode, "mode"), _whole(dfinal, "dfinal", (B, D), f32, dev),
                    _whole(lengths, "lengths", (B,), torch.int32, dev), dgate.data_ptr(), dx.data_ptr(),
                    dstate.data_ptr(), _stream_ptr(dev, stream))
    _check(rc, "based_scan_bwd")
    return dgate, dx, dstate


def based_scan_step(gate: torch.Tensor, x: torch.Tensor, pool: torch.Tensor, mode: str = "sigmoid",
                    slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One row of the recurrence for gate, x (N,D): ``pool`` (S,D) float32 holds the states and is
    updated in place; sequence i uses row slots[i] (int32; i without ``slots``). A slot outside
    [0, S) marks an idle sequence: its output is zero. Slots must not repeat. Returns h (N,D)."""
    L = _load()
    if x.dim() != 2 or pool.dim() != 2:
        raise ValueError("expected gate and x of shape (N,D) and pool of shape (S,D)")
    dev, shape, dtype = x.device, x.shape, x.dtype
    N, D = shape
    code = _dtype(x)
    _input(x, "x", shape, dtype, dev)
    _input(gate, "gate", shape, dtype, dev)
    S = pool.shape[0]
    with _pool(stream):
        y = _output(out, "out", shape, dtype, dev)
    rc = _on_device(dev, L.based_scan_step, gate.data_ptr(), gate.stride(0), x.data_ptr(), x.stride(0), N, D, S,
                    code, _code(MODES, mode, "mode"), _whole(pool, "pool", (S, D), torch.float32, dev),
                    _whole(slots, "slots", (N,), torch.int32, dev), y.data_ptr(), _stream_ptr(dev, stream))
    _check(rc, "based_scan_step")
    return y


# ------------------------------------------------------------------------------------------------
# Group norm with an activation
# ------------------------------------------------------------------------------------------------
def _norm_params(weight, bias, C, dev, fallback):
    given = weight if weight is not None else bias
    dtype = fallback if given is None else given.dtype
    if dtype not in DTYPES:
        raise TypeError(f"weight and bias must be float32, bfloat16 or float16, got {dtype}")
    return dtype, _whole(weight, "weight", (C,), dtype, dev), _whole(bias, "bias", (C,), dtype, dev)


def based_norm_fwd(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, act: str = "silu",
                   eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Group norm over the channels of each row of x (..., C), then v * act(gate), or act(v) without
    a gate; v = (x - mean) / sqrt(var + eps) * weight + bias with mean and var of each row's C /
    groups consecutive channels. act: "none", "silu" or "sigmoid".

    The output has the type of ``gate``, or ``out_dtype``, or the type of x; a type other than x's
    needs a float32 x (such as the output of based_fwd, viewed as (B, T, H * V) with groups = H).
    weight and bias (C) share one type.
    """
    L = _load()
    dev, shape = x.device, x.shape
    C = shape[-1]
    dtype = gate.dtype if gate is not None else out_dtype if out_dtype is not None else x.dtype
    if out_dtype is not None and out_dtype != dtype:
        raise TypeError(f"the output has the type of gate ({dtype}), not {out_dtype}")
    if dtype not in DTYPES:
        raise TypeError(f"expected a float32, bfloat16 or float16 output, got {dtype}")
    xcode = _dtype(x)
    _input(x, "x", shape, x.dtype, dev)
    x2 = _rows(x, "x")
    g2 = None
    if gate is not None:
        _input(gate, "gate", shape, dtype, dev)
        g2 = _rows(gate, "gate")
    pdtype, w, b = _norm_params(weight, bias, C, dev, dtype)
    with _pool(stream):
        y = _output(out, "out", shape, dtype, dev)
    rc = _on_device(dev, L.based_norm_fwd, x2.data_ptr(), x2.stride(0), xcode, _ptr(g2),
                    0 if g2 is None else g2.stride(0), w, b, DTYPES[pdtype], x2.shape[0], C, groups, eps,
                    _code(ACTS, act, "act"), y.data_ptr(), DTYPES[dtype], _stream_ptr(dev, stream))
    _check(rc, "based_norm_fwd")
    return y


def based_norm_bwd(dy: torch.Tensor, x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, act: str = "silu",
                   eps: float = 1e-5, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """Gradients of based_norm_fwd: (dx, dgate, dweight, dbias), None for what was not given.
    ``workspace``: a CUDA byte tensor of at least norm_bwd_workspace_size(...) bytes (default: one is
    allocated)."""
    L = _load()
    dev, shape = x.device, x.shape
    C = shape[-1]
    dtype = dy.dtype
    code, xcode = _dtype(dy), _dtype(x)
    _input(x, "x", shape, x.dtype, dev)
    _input(dy, "dy", shape, dtype, dev)
    x2, d2, g2 = _rows(x, "x"), _rows(dy, "dy"), None
    if gate is not None:
        _input(gate, "gate", shape, dtype, dev)
        g2 = _rows(gate, "gate")
    pdtype, w, b = _norm_params(weight, bias, C, dev, dtype)
    R = x2.shape[0]
    with _pool(stream):
        dx = torch.empty(shape, dtype=x.dtype, device=dev)
        dgate = None if gate is None else torch.empty(shape, dtype=dtype, device=dev)
        dweight = None if weight is None else torch.empty(C, dtype=pdtype, device=dev)
        dbias = None if bias is None else torch.empty(C, dtype=pdtype, device=dev)
        if workspace is None and (w is not None or b is not None):
            workspace = torch.empty(_on_device(dev, L.based_norm_bwd_workspace_size, R, C, groups),
                                    dtype=torch.uint8, device=dev)
    rc = _on_device(dev, L.based_norm_bwd, d2.data_ptr(), d2.stride(0), x2.data_ptr(), x2.stride(0), xcode,
                    _ptr(g2), 0 if g2 is None else g2.stride(0), w, b, DTYPES[pdtype], R, C, groups, eps,
                    _code(ACTS, act, "act"), dx.data_ptr(), _ptr(dgate), _ptr(dweight), _ptr(dbias), code,
                    _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
                    _stream_ptr(dev, stream))
    _check(rc, "based_norm_bwd")
    return dx, dgate, dweight, dbias


def norm_bwd_workspace_size(rows: int, channels: int, groups: int, device=None) -> int:
    """Bytes of workspace based_norm_bwd takes for these sizes."""
    L = _load()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(L.based_norm_bwd_workspace_size(rows, channels, groups))


# ------------------------------------------------------------------------------------------------
# Embedding
# ------------------------------------------------------------------------------------------------
def _ids(ids: torch.Tensor, dev) -> int:
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.device != dev or not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous CUDA tensor on the device of the other inputs")
    return 1 if ids.dtype == torch.int64 else 0


def based_embed_fwd(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
                    out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """scale * table[ids] for ids (...) int32 or int64 and table (V,D): (..., D) in the type of table.
    An id outside [0, V) is padding: its row is zero."""
    L = _load()
    if table.dim() != 2:
        raise ValueError("expected a table of shape (V,D)")
    dev, dtype = table.device, table.dtype
    V, D = table.shape
    code, wide = _dtype(table), _ids(ids, dev)
    _input(table, "table", table.shape, dtype, dev)
    with _pool(stream):
        y = _output(out, "out", (*ids.shape, D), dtype, dev)
    rc = _on_device(dev, L.based_embed_fwd, ids.data_ptr(), wide, table.data_ptr(), table.stride(0), ids.numel(),
                    V, D, code, scale, y.data_ptr(), _stream_ptr(dev, stream))
    _check(rc, "based_embed_fwd")
    return y


def based_embed_bwd(ids: torch.Tensor, dy: torch.Tensor, rows: int, scale: float = 1.0,
                    dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The gradient (rows, D) of a table of ``rows`` rows for the gradient dy (..., D) of
    based_embed_fwd's output: float32, or the type of dy. Summed in float32 by sorted tokens, with
    the same bits every time. ``workspace``: a CUDA byte tensor of at least
    embed_bwd_workspace_size(...) bytes (default: one is allocated)."""
    L = _load()
    dev = dy.device
    D = dy.shape[-1]
    code, wide = _dtype(dy), _ids(ids, dev)
    if dtype not in DTYPES:
        raise TypeError(f"expected a float32, bfloat16 or float16 gradient, got {dtype}")
    _input(dy, "dy", (*ids.shape, D), dy.dtype, dev)
    d2, N = _rows(dy, "dy"), ids.numel()
    with _pool(stream):
        dtable = _output(out, "out", (rows, D), dtype, dev)
        if workspace is None:
            workspace = torch.empty(L.based_embed_bwd_workspace_size(N, rows, D), dtype=torch.uint8, device=dev)
    rc = _on_device(dev, L.based_embed_bwd, ids.data_ptr(), wide, d2.data_ptr(), d2.stride(0), N, rows, D, code,
                    scale, dtable.data_ptr(), DTYPES[dtype], workspace.data_ptr(),
                    workspace.numel() * workspace.element_size(), _stream_ptr(dev, stream))
    _check(rc, "based_embed_bwd")
    return dtable


def embed_bwd_workspace_size(n: int, rows: int, channels: int) -> int:
    """Bytes of workspace based_embed_bwd takes for n tokens and a table of these sizes."""
    return int(_load().based_embed_bwd_workspace_size(n, rows, channels))
