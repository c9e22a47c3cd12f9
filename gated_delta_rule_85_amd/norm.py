"""Group norm of every token's channels with an activation, as layers use it on the operators' output.

A token's C channels are ``num_groups`` groups, each normalised by itself (one group per v
head for the output of :func:`chunk_gated_delta_rule` and :func:`chunk_linear_attention`),

    n = (x - mean) / sqrt(mean((x - mean)^2) + eps),  or  x / sqrt(mean(x^2) + eps) with center=False,
    y = n * weight + bias,   out = y * act(gate),   or   act(y) without a gate.

Every step runs in libgdr's HIP kernels.
"""
import torch
from torch.autograd import forward_ad

from . import _lib
from .pool import _gdr_torch

_ACT = {None: _lib.ACT_NONE, "silu": _lib.ACT_SILU, "sigmoid": _lib.ACT_SIGMOID}


def _activation(name):
    if name not in _ACT:
        raise ValueError("activation must be 'silu', 'sigmoid' or None")
    return _ACT[name]


def group_norm_bwd(x, num_groups, dout, weight=None, bias=None, gate=None, eps=1e-5, *, activation="silu", center=True,
                   weight_grads=True):
    """Low-level backward.  Returns ``(dx, dweight, dbias, dgate)``: dx and dgate in the dtypes
    of x and gate, dweight and dbias float32; None for what was not given (dweight and dbias
    also without ``weight_grads``).  ``dout`` may be bfloat16 or float32."""
    return _gdr_torch.norm_bwd(x, num_groups, dout, weight, bias, gate, eps, _activation(activation), center, weight_grads)


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, num_groups, weight, bias, gate, eps, activation, center, output_dtype):
        out = _gdr_torch.norm(x, num_groups, weight, bias, gate, eps, _activation(activation), center, output_dtype)
        ctx.save_for_backward(x, weight, bias, gate)
        ctx.rest = num_groups, eps, activation, center
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        x, weight, bias, gate = ctx.saved_tensors
        num_groups, eps, activation, center = ctx.rest
        sums = ctx.needs_input_grad[2] or ctx.needs_input_grad[3]
        dx, dw, db, dz = group_norm_bwd(x, num_groups, dout, weight, bias, gate, eps, activation=activation,
                                        center=center, weight_grads=sums)
        like = lambda d, t: None if d is None else d.to(t.dtype)  # noqa: E731
        return dx, None, like(dw, weight), like(db, bias), dz, None, None, None, None


def group_norm(x, num_groups, weight=None, bias=None, gate=None, eps=1e-5, *, activation="silu", center=True,
               output_dtype=None):
    """Differentiable group norm with an activation, channels last.  Returns x's shape.

    x [..., C] bfloat16 or float32, of groups of at most 8192 channels; ``gate`` like x (its
    dtype may differ); weight and bias [C].  ``activation``: "silu", "sigmoid" or None, of the
    gate or, without one, of the result.  ``center=False`` normalises by the root mean square.
    ``output_dtype``: default that of gate, else of x.  x and gate may be slices of wider rows:
    they are read in place where their rows are one distance apart.  Statistics and sums run in
    float32.  A value that is not finite stays in its token's group.
    """
    if forward_ad._current_level >= 0 or torch.is_grad_enabled() and any(
            t is not None and t.requires_grad for t in (x, weight, bias, gate)):
        return _GroupNorm.apply(x, num_groups, weight, bias, gate, eps, activation, center, output_dtype)
    return _gdr_torch.norm(x, num_groups, weight, bias, gate, eps, _activation(activation), center, output_dtype)
