"""Python functions of the C ABI in ``include/based_ops.h``.

The operators of a language model around the Based forward pass: the gated linear recurrence
(``based_scan_*``), the per-token group norm with an activation (``based_norm_*``), the scaled
embedding with its gradient (``based_embed_*``), the gated delta rule (``based_delta_*``), the
root-mean-square norm of a residual stream (``based_rms_*``) and the choice of a next token
(``based_sample``). Every step runs in the CUDA kernels of
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
from typing import Optional, Tuple, Union

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
    heads = [l, l, l]
    L.based_delta_fwd.argtypes = [p, *heads, p, *heads, p, *heads, p, l, l, p, l, l, i, i, i, i, i, i, i, f, p, p, p, p, p, p, z, p]
    L.based_delta_bwd.argtypes = [p, *heads, p, *heads, p, *heads, p, l, l, p, l, l, p, *heads, p, i, i, i, i, i, i, i, f, p, p,
                                  p, p, p, p, p, p, p, z, p]
    L.based_delta_step.argtypes = [p, l, l, p, l, l, p, l, l, p, l, p, l, i, i, i, i, i, i, i, f, p, p, p, p]
    L.based_delta_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
    L.based_delta_workspace_size.restype = z
    L.based_delta_saved_size.argtypes = [i, i, i, i, i, i]
    L.based_delta_saved_size.restype = z
    L.based_rms_fwd.argtypes = [p, l, p, l, i, p, i, l, i, f, p, p, i, p, p]
    L.based_rms_bwd.argtypes = [p, l, p, l, i, p, i, p, l, l, i, f, p, p, p, i, p, z, p]
    L.based_rms_bwd_workspace_size.argtypes = [l, i]
    L.based_rms_bwd_workspace_size.restype = z
    L.based_sample.argtypes = [p, l, i, i, i, p, p, f, p, i, p, f, p, f, p, p, p]
    for name in ("scan_fwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd", "embed_fwd", "embed_bwd", "delta_fwd", "delta_bwd",
                 "delta_step", "rms_fwd", "rms_bwd", "sample"):
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


# ------------------------------------------------------------------------------------------------
# Gated delta rule
# ------------------------------------------------------------------------------------------------
def based_delta_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, gate: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, state: Optional[torch.Tensor] = None,
                    lengths: Optional[torch.Tensor] = None, save: bool = False, out: Optional[torch.Tensor] = None,
                    final_state: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """S_t = a_t S_{t-1} + k_t u_t^T with u_t = beta_t (v_t - a_t S_{t-1}^T k_t), o_t = scale S_t^T q_t along axis 1 of
    q, k (B,T,HK,K) and v (B,T,H,V); a = exp(gate), or 1 without a gate; beta and gate (B,T,H) have the type of v.

    Heads of v share the HK heads of q and k in consecutive groups. ``scale`` defaults to K^-0.5. ``state`` (B,H,K,V)
    float32 is S before the first row (default zero); ``lengths`` (B) int32 marks rows t >= lengths[b] as padding
    (zero output, state kept). An infinity or NaN leaves a head undefined from its chunk of 64 rows on. Products are as accurate as
    float32's; with bfloat16 what is in outputs and gradients alone has 11 bits (include/based_ops.h says which). Returns (o
    (B,T,H,V) in the type of v, the last state (B,H,K,V) float32, the bytes that based_delta_bwd needs, or None without
    ``save``). ``final_state`` may be ``state``, to update it in place. ``workspace``: a CUDA byte tensor of at
    least delta_workspace_size(...) bytes (default: one is allocated).
    """
    return _C.delta_fwd(q, k, v, beta, gate, scale, state, lengths, save, out, final_state, workspace, stream)


def based_delta_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, gate: Optional[torch.Tensor],
                    dout: torch.Tensor, saved: torch.Tensor, scale: Optional[float] = None, dfinal: Optional[torch.Tensor] = None,
                    lengths: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None):
    """Gradients of based_delta_fwd for the gradients dout (B,T,H,V) of its output and dfinal (B,H,K,V) float32 of its
    last state: (dq, dk, dv, dbeta, dgate, dstate), dgate None without a gate. ``saved`` is what the forward call returned."""
    return _C.delta_bwd(q, k, v, beta, gate, dout, saved, scale, dfinal, lengths, workspace, stream)


def based_delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, gate: Optional[torch.Tensor],
                     pool: torch.Tensor, scale: Optional[float] = None, slots: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One row of the delta rule for q, k (N,HK,K), v (N,H,V), beta and gate (N,H): ``pool`` (S,H,K,V) float32 holds the
    states and is updated in place; slots as in based_scan_step. Returns o (N,H,V)."""
    return _C.delta_step(q, k, v, beta, gate, pool, scale, slots, out, stream)


def delta_workspace_size(batch: int, rows: int, heads: int, key_heads: int, key_size: int, value_size: int,
                         dtype: torch.dtype = torch.bfloat16, backward: bool = False) -> int:
    """Bytes of workspace based_delta_fwd or based_delta_bwd takes for these sizes."""
    code = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[dtype]
    return library().based_delta_workspace_size(batch, rows, heads, key_heads, key_size, value_size, code, int(backward))


# ------------------------------------------------------------------------------------------------
# Root-mean-square norm of a residual stream
# ------------------------------------------------------------------------------------------------
def based_rms_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                  eps: float = 1e-6, quantize: bool = False, out: Optional[torch.Tensor] = None,
                  sum_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(y, s, scales): s = x + residual (..., C) in the type of ``residual`` (that of x, or float32), x itself without one, and
    y = s / sqrt(mean(s^2) + eps) * weight in the type of x. The norm is that of the s that is written.

    ``quantize``: y is float8_e4m3fn, with scales (...) float32 so that y * scales is the norm and each row's largest is 448;
    else scales is None. weight (C) has the type of x or float32. ``sum_out`` may be ``residual``, to add in place.
    """
    return _C.rms_fwd(x, weight, residual, eps, quantize, out, sum_out, stream)


def based_rms_bwd(dy: torch.Tensor, s: torch.Tensor, weight: Optional[torch.Tensor] = None,
                  dsum: Optional[torch.Tensor] = None, eps: float = 1e-6, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None):
    """Gradients of based_rms_fwd for the gradients dy of y and dsum of s: (ds, dx, dweight). ds is that of the residual, in the
    type of s, dx that of x: the same values in the type of dy, the same tensor where the types are. ``s`` is what the
    forward call returned. ``workspace``: a CUDA byte tensor of at least rms_bwd_workspace_size(...) bytes (default: one
    is allocated)."""
    return _C.rms_bwd(dy, s, weight, dsum, eps, workspace, stream)


def rms_bwd_workspace_size(rows: int, channels: int) -> int:
    """Bytes of workspace based_rms_bwd takes for these sizes."""
    return library().based_rms_bwd_workspace_size(rows, channels)


# ------------------------------------------------------------------------------------------------
# Sampling
# ------------------------------------------------------------------------------------------------
PerRow = Union[float, torch.Tensor, None]


def based_sample(logits: torch.Tensor, u: torch.Tensor, temperature: PerRow = 1.0, top_k: PerRow = None, top_p: PerRow = None,
                 min_p: PerRow = None, out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The next token of each row of logits (N,V) from random numbers u (N) float32 in [0, 1): (tokens (N) int32, their
    probabilities (N) float32 among what their rows keep).

    A row keeps the top_k largest logits (of equal ones the first), of these the fewest of the largest whose probabilities
    reach top_p of theirs, and of these the ones of at least min_p times the largest's; the token is the first, in the order
    of indices, at which the kept probabilities exceed u. Each limit is a number, a tensor (N) (float32; top_k
    int32) or None. temperature <= 0 takes the largest logit. -inf is never taken, NaN counts as -inf, and a row
    with nothing else gives token -1.
    """
    return _C.sample(logits, u, temperature, top_k, top_p, min_p, out, stream)
