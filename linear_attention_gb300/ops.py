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

import ctypes
from typing import Optional, Tuple

import torch

from . import based
from .based import _check

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
# Checks. A small call is bound by the host, so these look at each tensor once and by the cheapest
# accessors (a device by its index, -1 for host tensors).
# ------------------------------------------------------------------------------------------------
_raw_stream = torch._C._cuda_getCurrentRawStream  # the handle alone, without a Stream object


def _code(table, key, what):
    code = table.get(key)
    if code is None:
        if table is DTYPES:
            raise TypeError(f"{what} must be float32, bfloat16 or float16, got {key}")
        raise ValueError(f"{what} must be one of {', '.join(table)}, got {key!r}")
    return code


def _input(t: torch.Tensor, name: str, shape, dtype, idx: int):
    """t is a tensor of this shape and type on this device whose last axis has stride 1."""
    if t.shape == shape and t.dtype == dtype and t.get_device() == idx >= 0 and t.stride(-1) == 1:
        return
    if t.get_device() != idx or idx < 0:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the other inputs")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape[-1] != 1:
        raise ValueError(f"the last axis of {name} must have stride 1")


def _whole(t: torch.Tensor, name: str, shape, dtype, idx: int) -> int:
    """The address of a contiguous tensor of this shape and type."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != idx or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _workspace(t: torch.Tensor, idx: int) -> torch.Tensor:
    if t.get_device() != idx or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the device of the inputs")
    return t


def _run(what: str, fn, idx: int, stream: Optional[torch.cuda.Stream], *args):
    """fn(*args, stream) with device idx as the current one."""
    if torch.cuda.current_device() == idx:
        rc = fn(*args, _raw_stream(idx) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(idx):
            rc = fn(*args, _raw_stream(idx) if stream is None else stream.cuda_stream)
    if rc != 0:
        _check(rc, what)


def _empty(shape, dtype, dev, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A new tensor; for a call on a side stream it comes from that stream's pool."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


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
    L = _lib or _load()
    shape, dtype, idx, dev = x.shape, x.dtype, x.get_device(), x.device
    if len(shape) != 3:
        raise ValueError("expected gate and x of shape (B,T,D)")
    B, T, D = shape
    code = _code(DTYPES, dtype, "x")
    _input(x, "x", shape, dtype, idx)
    _input(gate, "gate", shape, dtype, idx)
    f32 = torch.float32
    y = _empty(shape, dtype, dev, stream) if out is None else out
    last = _empty((B, D), f32, dev, stream) if final_state is None else final_state
    saved = _empty((B, -(-T // SAVE_ROWS), D), f32, dev, stream) if save else None
    _run("based_scan_fwd", L.based_scan_fwd, idx, stream, gate.data_ptr(), gate.stride(0), gate.stride(1),
         x.data_ptr(), x.stride(0), x.stride(1), B, T, D, code, _code(MODES, mode, "mode"),
         None if state is None else _whole(state, "state", (B, D), f32, idx),
         None if lengths is None else _whole(lengths, "lengths", (B,), torch.int32, idx),
         y.data_ptr() if out is None else _whole(out, "out", shape, dtype, idx),
         last.data_ptr() if final_state is None else _whole(final_state, "final_state", (B, D), f32, idx),
         None if saved is None else saved.data_ptr())
    return y, last, saved


def based_scan_bwd(gate: torch.Tensor, x: torch.Tensor, dy: torch.Tensor, saved: torch.Tensor,
                   mode: str = "sigmoid", dfinal: Optional[torch.Tensor] = None,
                   lengths: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of based_scan_fwd for the gradients dy (B,T,D) of its output and dfinal (B,D)
    float32 of its last state: (dgate, dx, dstate). ``saved`` is what the forward call returned."""
    L = _lib or _load()
    shape, dtype, idx, dev = x.shape, x.dtype, x.get_device(), x.device
    if len(shape) != 3:
        raise ValueError("expected gate, x and dy of shape (B,T,D)")
    B, T, D = shape
    code = _code(DTYPES, dtype, "x")
    _input(x, "x", shape, dtype, idx)
    _input(gate, "gate", shape, dtype, idx)
    _input(dy, "dy", shape, dtype, idx)
    f32 = torch.float32
    if saved is None:
        raise ValueError("based_scan_bwd needs the saved states of based_scan_fwd(..., save=True)")
    dgate, dx = _empty(shape, dtype, dev, stream), _empty(shape, dtype, dev, stream)
    dstate = _empty((B, D), f32, dev, stream)
    _run("based_scan_bwd", L.based_scan_bwd, idx, stream, gate.data_ptr(), gate.stride(0), gate.stride(1),
         x.data_ptr(), x.stride(0), x.stride(1), dy.data_ptr(), dy.stride(0), dy.stride(1),
         _whole(saved, "saved", (B, -(-T // SAVE_ROWS), D), f32, idx), B, T, D, code, _code(MODES, mode, "mode"),
         None if dfinal is None else _whole(dfinal, "dfinal", (B, D), f32, idx),
         None if lengths is None else _whole(lengths, "lengths", (B,), torch.int32, idx),
         dgate.data_ptr(), dx.data_ptr(), dstate.data_ptr())
    return dgate, dx, dstate


def based_scan_step(gate: torch.Tensor, x: torch.Tensor, pool: torch.Tensor, mode: str = "sigmoid",
                    slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One row of the recurrence for gate, x (N,D): ``pool`` (S,D) float32 holds the states and is
    updated in place; sequence i uses row slots[i] (int32; i without ``slots``). A slot outside
    [0, S) marks an idle sequence: its output is zero. Slots must not repeat. Returns h (N,D)."""
    L = _lib or _load()
    shape, dtype, idx = x.shape, x.dtype, x.get_device()
    if len(shape) != 2 or pool.dim() != 2:
        raise ValueError("expected gate and x of shape (N,D) and pool of shape (S,D)")
    N, D = shape
    code = _code(DTYPES, dtype, "x")
    _input(x, "x", shape, dtype, idx)
    _input(gate, "gate", shape, dtype, idx)
    S = pool.shape[0]
    y = _empty(shape, dtype, x.device, stream) if out is None else out
    _run("based_scan_step", L.based_scan_step, idx, stream, gate.data_ptr(), gate.stride(0), x.data_ptr(), x.stride(0),
         N, D, S, code, _code(MODES, mode, "mode"), _whole(pool, "pool", (S, D), torch.float32, idx),
         None if slots is None else _whole(slots, "slots", (N,), torch.int32, idx),
         y.data_ptr() if out is None else _whole(out, "out", shape, dtype, idx))
    return y


# ------------------------------------------------------------------------------------------------
# Group norm with an activation
# ------------------------------------------------------------------------------------------------
def _norm_params(weight, bias, C, idx, fallback):
    """The type code and the addresses of weight and bias."""
    dtype = weight.dtype if weight is not None else bias.dtype if bias is not None else fallback
    return (_code(DTYPES, dtype, "weight and bias"),
            None if weight is None else _whole(weight, "weight", (C,), dtype, idx),
            None if bias is None else _whole(bias, "bias", (C,), dtype, idx))


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
    L = _lib or _load()
    shape, xdtype, idx = x.shape, x.dtype, x.get_device()
    C = shape[-1]
    dtype = gate.dtype if gate is not None else out_dtype if out_dtype is not None else xdtype
    if out_dtype is not None and out_dtype != dtype:
        raise TypeError(f"the output has the type of gate ({dtype}), not {out_dtype}")
    code, xcode = _code(DTYPES, dtype, "the output"), _code(DTYPES, xdtype, "x")
    _input(x, "x", shape, xdtype, idx)
    x2 = _rows(x, "x")
    if gate is not None:
        _input(gate, "gate", shape, dtype, idx)
        g2 = _rows(gate, "gate")
        gp, gs = g2.data_ptr(), g2.stride(0)
    else:
        gp, gs = None, 0
    pcode, w, b = _norm_params(weight, bias, C, idx, dtype)
    y = _empty(shape, dtype, x.device, stream) if out is None else out
    _run("based_norm_fwd", L.based_norm_fwd, idx, stream, x2.data_ptr(), x2.stride(0), xcode, gp, gs, w, b, pcode,
         x2.shape[0], C, groups, eps, _code(ACTS, act, "act"),
         y.data_ptr() if out is None else _whole(out, "out", shape, dtype, idx), code)
    return y


def based_norm_bwd(dy: torch.Tensor, x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, act: str = "silu",
                   eps: float = 1e-5, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """Gradients of based_norm_fwd: (dx, dgate, dweight, dbias), None for what was not given.
    ``workspace``: a CUDA byte tensor of at least norm_bwd_workspace_size(...) bytes (default: one is
    allocated)."""
    L = _lib or _load()
    shape, xdtype, idx, dev = x.shape, x.dtype, x.get_device(), x.device
    C, dtype = shape[-1], dy.dtype
    code, xcode = _code(DTYPES, dtype, "dy"), _code(DTYPES, xdtype, "x")
    _input(x, "x", shape, xdtype, idx)
    _input(dy, "dy", shape, dtype, idx)
    x2, d2 = _rows(x, "x"), _rows(dy, "dy")
    R = x2.shape[0]
    if gate is not None:
        _input(gate, "gate", shape, dtype, idx)
        g2 = _rows(gate, "gate")
        gp, gs, dgate = g2.data_ptr(), g2.stride(0), _empty(shape, dtype, dev, stream)
    else:
        gp, gs, dgate = None, 0, None
    pcode, w, b = _norm_params(weight, bias, C, idx, dtype)
    dx = _empty(shape, xdtype, dev, stream)
    dweight = None if weight is None else _empty(C, weight.dtype, dev, stream)
    dbias = None if bias is None else _empty(C, bias.dtype, dev, stream)
    if workspace is not None:
        _workspace(workspace, idx)
    elif w is not None or b is not None:
        workspace = _empty(norm_bwd_workspace_size(R, C, groups, idx), torch.uint8, dev, stream)
    _run("based_norm_bwd", L.based_norm_bwd, idx, stream, d2.data_ptr(), d2.stride(0), x2.data_ptr(), x2.stride(0),
         xcode, gp, gs, w, b, pcode, R, C, groups, eps, _code(ACTS, act, "act"), dx.data_ptr(),
         None if dgate is None else dgate.data_ptr(), None if dweight is None else dweight.data_ptr(),
         None if dbias is None else dbias.data_ptr(), code, None if workspace is None else workspace.data_ptr(),
         0 if workspace is None else workspace.numel() * workspace.element_size())
    return dx, dgate, dweight, dbias


def norm_bwd_workspace_size(rows: int, channels: int, groups: int, device=None) -> int:
    """Bytes of workspace based_norm_bwd takes for these sizes."""
    L = _lib or _load()
    if device is None or device == torch.cuda.current_device():
        return L.based_norm_bwd_workspace_size(rows, channels, groups)
    with torch.cuda.device(device):
        return L.based_norm_bwd_workspace_size(rows, channels, groups)


# ------------------------------------------------------------------------------------------------
# Embedding
# ------------------------------------------------------------------------------------------------
def _ids(ids: torch.Tensor, idx: int) -> int:
    """Whether ids are 64 bits wide."""
    dtype = ids.dtype
    if dtype is not torch.int32 and dtype is not torch.int64:
        raise TypeError(f"ids must be int32 or int64, got {dtype}")
    if ids.get_device() != idx or idx < 0 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous CUDA tensor on the device of the other inputs")
    return 1 if dtype is torch.int64 else 0


def based_embed_fwd(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
                    out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """scale * table[ids] for ids (...) int32 or int64 and table (V,D): (..., D) in the type of table.
    An id outside [0, V) is padding: its row is zero."""
    L = _lib or _load()
    dtype, idx = table.dtype, table.get_device()
    if table.dim() != 2:
        raise ValueError("expected a table of shape (V,D)")
    V, D = table.shape
    code, wide = _code(DTYPES, dtype, "table"), _ids(ids, idx)
    _input(table, "table", table.shape, dtype, idx)
    shape = (*ids.shape, D)
    y = _empty(shape, dtype, table.device, stream) if out is None else out
    _run("based_embed_fwd", L.based_embed_fwd, idx, stream, ids.data_ptr(), wide, table.data_ptr(), table.stride(0),
         ids.numel(), V, D, code, scale, y.data_ptr() if out is None else _whole(out, "out", shape, dtype, idx))
    return y


def based_embed_bwd(ids: torch.Tensor, dy: torch.Tensor, rows: int, scale: float = 1.0,
                    dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The gradient (rows, D) of a table of ``rows`` rows for the gradient dy (..., D) of
    based_embed_fwd's output: float32, or the type of dy. Summed in float32 by sorted tokens, with
    the same bits every time. ``workspace``: a CUDA byte tensor of at least
    embed_bwd_workspace_size(...) bytes (default: one is allocated)."""
    L = _lib or _load()
    idx, dev, D, N = dy.get_device(), dy.device, dy.shape[-1], ids.numel()
    code, gcode, wide = _code(DTYPES, dy.dtype, "dy"), _code(DTYPES, dtype, "the gradient"), _ids(ids, idx)
    _input(dy, "dy", (*ids.shape, D), dy.dtype, idx)
    d2 = _rows(dy, "dy")
    dtable = _empty((rows, D), dtype, dev, stream) if out is None else out
    if workspace is not None:
        _workspace(workspace, idx)
    else:
        workspace = _empty(L.based_embed_bwd_workspace_size(N, rows, D), torch.uint8, dev, stream)
    _run("based_embed_bwd", L.based_embed_bwd, idx, stream, ids.data_ptr(), wide, d2.data_ptr(), d2.stride(0), N,
         rows, D, code, scale, dtable.data_ptr() if out is None else _whole(out, "out", (rows, D), dtype, idx), gcode,
         workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dtable


def embed_bwd_workspace_size(n: int, rows: int, channels: int) -> int:
    """Bytes of workspace based_embed_bwd takes for n tokens and a table of these sizes."""
    return (_lib or _load()).based_embed_bwd_workspace_size(n, rows, channels)
