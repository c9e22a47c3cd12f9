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
from .api import _DT, _ptr
from .pool import _gdr_torch

_ACT = {None: _lib.ACT_NONE, "silu": _lib.ACT_SILU, "sigmoid": _lib.ACT_SIGMOID}


def _activation(name):
    if name not in _ACT:
        raise ValueError("activation must be 'silu', 'sigmoid' or None")
    return _ACT[name]


def _matrix(x, C):
    """x [..., C] as rows [M, C] with one distance between them (a copy where it has none)."""
    x = x.reshape(-1, C)
    if C > 1 and x.stride(1) != 1:
        x = x.contiguous()
    return x, (x.stride(0) if x.shape[0] > 1 else 0)


def group_norm_bwd(x, num_groups, dout, weight=None, bias=None, gate=None, eps=1e-5, *, activation="silu", center=True,
                   weight_grads=True):
    """Low-level backward.  Returns ``(dx, dweight, dbias, dgate)``: dx and dgate in the dtypes
    of x and gate, dweight and dbias float32; None for what was not given (dweight and dbias
    also without ``weight_grads``).  ``dout`` may be bfloat16 or float32."""
    act, dev, C = _activation(activation), x.device, x.shape[-1]
    if dout.shape != x.shape or dout.dtype not in _DT:
        raise ValueError("dout must be like x, bfloat16 or float32")
    if gate is not None and gate.shape != x.shape:
        raise ValueError("gate must be like x, bfloat16 or float32")
    for t in (x, gate):
        if t is not None and t.dtype not in _DT:
            raise ValueError("x and gate must be bfloat16 or float32")
    for t in (weight, bias):
        if t is not None and (t.shape != (C,) or not t.is_floating_point()):
            raise ValueError("weight and bias must be [C]")
    if num_groups < 1 or C < 1 or C % num_groups:
        raise ValueError("the channels of x must be a multiple of num_groups")
    if not x.is_cuda:
        raise ValueError("inputs must be on the GPU")
    for t in (dout, weight, bias, gate):
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on one GPU")
    with torch.cuda.device(dev):
        a = _lib.NormBwdArgs()
        xm, a.x_row = _matrix(x, C)
        zm, a.gate_row = (None, 0) if gate is None else _matrix(gate, C)
        dout = dout.contiguous()
        w, b = (None if t is None else t.float().contiguous() for t in (weight, bias))
        dx, dz = torch.empty(x.shape, dtype=x.dtype, device=dev), None
        if gate is not None:
            dz = torch.empty(gate.shape, dtype=gate.dtype, device=dev)
        dw = torch.empty(C, dtype=torch.float32, device=dev) if weight is not None and weight_grads else None
        db = torch.empty(C, dtype=torch.float32, device=dev) if bias is not None and weight_grads else None
        a.M, a.C, a.groups = xm.shape[0], C, num_groups
        a.x_dtype, a.out_dtype = _DT[x.dtype], _DT[dout.dtype]
        a.gate_dtype = a.x_dtype if gate is None else _DT[gate.dtype]
        a.activation, a.center, a.eps = act, int(center), float(eps)
        a.x, a.weight, a.bias, a.gate, a.dout = _ptr(xm), _ptr(w), _ptr(b), _ptr(zm), _ptr(dout)
        a.dx, a.dgate, a.dweight, a.dbias = _ptr(dx), _ptr(dz), _ptr(dw), _ptr(db)
        ws = None
        if dw is not None or db is not None:
            nbytes = _lib.group_norm_bwd_workspace(a)
            ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
            a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes
        _lib.group_norm_bwd(a, torch.cuda.current_stream(dev).cuda_stream)
    return dx, dw, db, dz


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
