"""The operators of ``linear_attention_gb300.ops`` as differentiable torch functions.

Each function runs the forward kernel, keeps what the backward kernel needs, and gives its gradients
to torch's autograd. Inputs may have any strides: those that the kernels do not read are copied first. Forward and backward passes run on the stream that is current at the forward
call (autograd replays it). Gradients of gradients are not defined.

Capturing a training step into a CUDA graph follows torch's rules: run a few steps on the capturing
stream first, and let every loss of eager steps on the same parameters go before the capture begins.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd import Function
from torch.autograd.function import once_differentiable

from . import ops


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t as the kernels can read it: transposes, and gradients of sums and broadcasts, have a last axis of another
    stride than 1."""
    return t if t.dim() == 0 or t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _rows(t: torch.Tensor) -> torch.Tensor:
    """... and with one common stride of its leading axes."""
    if t.dim() == 0:
        return t
    try:
        t.view(-1, t.shape[-1])
    except RuntimeError:
        return t.contiguous()
    return _dense(t)


class _Scan(Function):
    @staticmethod
    def forward(ctx, gate, x, state, lengths, mode):
        needed = any(ctx.needs_input_grad[:3])
        gate, x = _dense(gate), _dense(x)
        state, lengths = (t if t is None else t.contiguous() for t in (state, lengths))
        y, final, saved = ops.based_scan_fwd(gate, x, mode=mode, state=state, lengths=lengths, save=needed)
        ctx.save_for_backward(gate, x, saved, lengths)
        ctx.mode = mode
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal):
        gate, x, saved, lengths = ctx.saved_tensors
        if dy is None and dfinal is None:
            return None, None, None, None, None
        dy = torch.zeros_like(x, memory_format=torch.contiguous_format) if dy is None else _dense(dy)
        dgate, dx, dstate = ops.based_scan_bwd(gate, x, dy, saved, mode=ctx.mode,
                                               dfinal=None if dfinal is None else dfinal.contiguous(), lengths=lengths)
        return dgate, dx, dstate if ctx.needs_input_grad[2] else None, None, None


class _Norm(Function):
    @staticmethod
    def forward(ctx, x, weight, bias, gate, groups, act, eps, out_dtype):
        x, gate = _rows(x), gate if gate is None else _rows(gate)
        weight, bias = (t if t is None else t.contiguous() for t in (weight, bias))
        ctx.save_for_backward(x, weight, bias, gate)
        ctx.args = dict(groups=groups, act=act, eps=eps)
        return ops.based_norm_fwd(x, weight=weight, bias=bias, gate=gate, out_dtype=out_dtype, **ctx.args)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, gate = ctx.saved_tensors
        dx, dgate, dweight, dbias = ops.based_norm_bwd(_rows(dy), x, weight=weight, bias=bias, gate=gate, **ctx.args)
        return dx, dweight, dbias, dgate, None, None, None, None


class _Embed(Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        table = _dense(table)
        ctx.save_for_backward(ids)
        ctx.args = (table.shape[0], scale, table.dtype)
        return ops.based_embed_fwd(ids, table, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, scale, dtype = ctx.args
        return None, ops.based_embed_bwd(ctx.saved_tensors[0], _rows(dy), rows, scale, dtype=dtype), None


def gated_scan(gate: torch.Tensor, x: torch.Tensor, mode: str = "sigmoid", state: Optional[torch.Tensor] = None,
               lengths: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gated linear recurrence (ops.based_scan_fwd): (h of every row, the last state)."""
    return _Scan.apply(gate, x, state, lengths, mode)


def group_norm(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, act: str = "silu",
               eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The per-token group norm with an activation (ops.based_norm_fwd)."""
    return _Norm.apply(x, weight, bias, gate, groups, act, eps, out_dtype)


def embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """The scaled embedding (ops.based_embed_fwd); the gradient has the type of the table."""
    return _Embed.apply(ids, table, scale)
