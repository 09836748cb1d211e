"""torch.autograd binding of the chunkwise forward and backward.

``delta_rule(variant, q, k, v, beta, g=None, wgate=None, S0=None)`` returns
(o, S_T) like ``ops.delta_fwd`` and differentiates through ``ops.delta_bwd``:
the forward and the backward both run in the library's kernels, this module
only routes tensors.  Gradients flow to every tensor argument that requires
them (grouped query/key heads included); the backward recomputes the forward
states itself, so nothing but the inputs is saved.

``linear_recurrence(x, g, beta=None, h0=None)`` does the same for the gated linear
recurrence (``ops.linrec_fwd``, ``ops.linrec_bwd``); it saves the inputs and the
fp32 state before every 16th token.

To capture a training step in a HIP graph, take its gradients with
``torch.autograd.grad`` inside the capture, after the eager graphs of the same leaves
are gone: torch's accumulation of ``.grad`` belongs to the stream that first used the
leaf, and may not join a capture on another.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import ops


def _gradient(t: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """A gradient as the library takes it: contiguous, of ``dtype``, at a multiple of 16
    bytes.  torch hands out contiguous gradients at any address (a part of the gradient
    of a ``cat`` or ``stack``)."""
    t = t.contiguous().to(dtype)
    return t.clone() if t.data_ptr() % 16 else t


class _DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, variant, q, k, v, beta, g, wgate, S0):
        o, S_T = ops.delta_fwd(variant, q, k, v, beta, wgate=wgate, g=g, S0=S0)
        ctx.variant = variant
        ctx.save_for_backward(q, k, v, beta, g, wgate, S0)
        return o, S_T

    @staticmethod
    def backward(ctx, dO, dS_T):
        q, k, v, beta, g, wgate, S0 = ctx.saved_tensors
        if dO is None:
            dO = torch.zeros(v.shape, dtype=v.dtype, device=v.device)
        dO = _gradient(dO, v.dtype)
        if dS_T is not None:
            dS_T = _gradient(dS_T, torch.float32)
        gr = ops.delta_bwd(ctx.variant, q, k, v, beta, dO, g=g, S0=S0, dS_T=dS_T, wgate=wgate,
                           want_dS0=S0 is not None and ctx.needs_input_grad[7])
        return (None, gr["dq"], gr["dk"], gr["dv"], gr["dbeta"], gr["dg"], gr["dwgate"], gr["dS0"])


def delta_rule(variant: str, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
               beta: torch.Tensor, g: Optional[torch.Tensor] = None,
               wgate: Optional[torch.Tensor] = None, S0: Optional[torch.Tensor] = None
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable chunkwise forward: (o, S_T) with gradients through delta_bwd."""
    return _DeltaRule.apply(variant, q, k, v, beta, g, wgate, S0)


class _LinearRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, beta, h0):
        o, h_T, states = ops.linrec_fwd(x, g, beta=beta, h0=h0, want_states=any(ctx.needs_input_grad))
        ctx.save_for_backward(x, g, beta, states)
        return o, h_T

    @staticmethod
    @once_differentiable
    def backward(ctx, dO, dh_T):
        x, g, beta, states = ctx.saved_tensors
        gr = ops.linrec_bwd(x, g, states, _gradient(dO, x.dtype), beta=beta, dh_T=_gradient(dh_T, torch.float32),
                            want_dh0=ctx.needs_input_grad[3])
        return gr["dx"], gr["dg"], gr["dbeta"], gr["dh0"]


def linear_recurrence(x: torch.Tensor, g: torch.Tensor, beta: Optional[torch.Tensor] = None,
                      h0: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable gated linear recurrence over [B, T, D]: (o, h_T), with gradients
    for x, g, beta and h0 through linrec_bwd."""
    return _LinearRecurrence.apply(x, g, beta, h0)
