"""Python functions of the C ABI in ``include/based_ops.h``.

The operators of a language model around the Based forward pass: the gated linear recurrence
(``based_scan_*``), the per-token group norm with an activation (``based_norm_*``) and the scaled
embedding with its gradient (``based_embed_*``). Every step runs in the CUDA kernels of
``libbased_gb300.so``; there is no fallback. Arguments are checked and passed on by the compiled
binding ``csrc/ops_binding.cpp``: wrong shapes, strides and devices raise ValueError, wrong types
TypeError, and what the C functions refuse raises BasedError.

All functions launch on ``stream`` (default: the current stream of the inputs' device). What they
allocate (outputs that are not passed in, workspaces) comes from that stream's pool, so a call on a
side stream needs ordering only for its inputs and for the use of its results. Inputs may be
strided as long as their last axis has stride 1; the leading axes of the norm's inputs and of the
embedding's dy need one common stride (rows at equal distances), states, lengths, slots, weights and
biases are contiguous, and ids may have any strides. Outputs are contiguous. Batches without rows, tokens
or sequences, which the C functions refuse, give empty outputs, the state they were given and
gradients of zero.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional, Tuple

import torch

from . import based
from .build import binding_path

SAVE_ROWS = 64  # BASED_SCAN_SAVE_ROWS


def _binding():
    path = binding_path()
    if not os.path.exists(path):
        raise based.BasedError(f"binding not built: {path} is missing (run linear_attention_gb300.build.build())")
    based.library()
    spec = importlib.util.spec_from_file_location("based_ops_binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.set_check(based._check)
    return module


class _Unloaded:
    """Stands for the binding until the first call, so that this module can be imported before build()."""

    def __getattr__(self, name):
        global _C
        _C = _binding()
        return getattr(_C, name)


_C = _Unloaded()


def library():
    """The loaded ctypes library with the signatures of include/based_ops.h."""
    L = based.library()
    p, i, l, f, z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
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
    return L


_load = library


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
    return _C.scan_fwd(gate, x, mode, state, lengths, save, out, final_state, stream)


def based_scan_bwd(gate: torch.Tensor, x: torch.Tensor, dy: torch.Tensor, saved: torch.Tensor,
                   mode: str = "sigmoid", dfinal: Optional[torch.Tensor] = None,
                   lengths: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of based_scan_fwd for the gradients dy (B,T,D) of its output and dfinal (B,D)
    float32 of its last state: (dgate, dx, dstate). ``saved`` is what the forward call returned."""
    return _C.scan_bwd(gate, x, dy, saved, mode, dfinal, lengths, stream)


def based_scan_step(gate: torch.Tensor, x: torch.Tensor, pool: torch.Tensor, mode: str = "sigmoid",
                    slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One row of the recurrence for gate, x (N,D): ``pool`` (S,D) float32 holds the states and is
    updated in place; sequence i uses row slots[i] (int32; i without ``slots``). A slot outside
    [0, S) marks an idle sequence: its output is zero. Slots must not repeat. Returns h (N,D)."""
    return _C.scan_step(gate, x, pool, mode, slots, out, stream)


# ------------------------------------------------------------------------------------------------
# Group norm with an activation
# ------------------------------------------------------------------------------------------------
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
    return _C.norm_fwd(x, groups, weight, bias, gate, act, eps, out_dtype, out, stream)


def based_norm_bwd(dy: torch.Tensor, x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, act: str = "silu",
                   eps: float = 1e-5, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """Gradients of based_norm_fwd: (dx, dgate, dweight, dbias), None for what was not given.
    ``workspace``: a CUDA byte tensor of at least norm_bwd_workspace_size(...) bytes (default: one is
    allocated)."""
    return _C.norm_bwd(dy, x, groups, weight, bias, gate, act, eps, workspace, stream)


def norm_bwd_workspace_size(rows: int, channels: int, groups: int, device=None) -> int:
    """Bytes of workspace based_norm_bwd takes for these sizes."""
    L = library()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return L.based_norm_bwd_workspace_size(rows, channels, groups)


# ------------------------------------------------------------------------------------------------
# Embedding
# ------------------------------------------------------------------------------------------------
def based_embed_fwd(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
                    out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """scale * table[ids] for ids (...) int32 or int64 and table (V,D): (..., D) in the type of table.
    An id outside [0, V) is padding: its row is zero."""
    return _C.embed_fwd(ids, table, scale, out, stream)


def based_embed_bwd(ids: torch.Tensor, dy: torch.Tensor, rows: int, scale: float = 1.0,
                    dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The gradient (rows, D) of a table of ``rows`` rows for the gradient dy (..., D) of
    based_embed_fwd's output: float32, or the type of dy. Summed in float32 by sorted tokens, with
    the same bits every time. ``workspace``: a CUDA byte tensor of at least
    embed_bwd_workspace_size(...) bytes (default: one is allocated)."""
    return _C.embed_bwd(ids, dy, rows, scale, dtype, out, workspace, stream)


def embed_bwd_workspace_size(n: int, rows: int, channels: int) -> int:
    """Bytes of workspace based_embed_bwd takes for n tokens and a table of these sizes."""
    return library().based_embed_bwd_workspace_size(n, rows, channels)
