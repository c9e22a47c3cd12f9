"""Linear attention with a decay for each head, in chunks, and its backward.

The gated delta rule without its correction: per (sequence, v head)

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t,

with the same states [K,V], head groups, gates and packed sequences as
:func:`chunk_gated_delta_rule`.  ``g`` is per token and v head, [B,T,H_v], or fixed for
each v head, [H_v].  The recurrent form on a pool of states is
:func:`recurrent_linear_attention`.  Every step runs in libgdr's HIP kernels.
"""
import torch
from torch.autograd import forward_ad

from .pool import _gdr_torch


def chunk_linear_attention_fwd(q, k, v, g, scale=None, initial_state=None, cu_seqlens=None, output_final_state=True,
                               *, output_dtype=torch.float32, segment_chunks=0):
    """Low-level forward.  Returns ``(o, final_state)``: o [B,T,H_v,V] in ``output_dtype``,
    final_state [N,H_v,K,V] float32 (None unless output_final_state).

    q, k and v may be slices of a wider projection: they are read in place where a token's
    heads are contiguous.  A long sequence of few heads is split into segments of
    ``segment_chunks`` chunks of 64 tokens (0: chosen for the device; the split is exact: a
    segment's part of the state is carried on by a scalar decay).  Sequences (segments) times H_v
    are below 2^22.  A gate of -104 or less,
    -inf among them, empties the state.  Rows of o that belong to no sequence are zero, and so
    are those of its gradients.
    """
    return _gdr_torch.la_fwd(q, k, v, g, scale, initial_state, cu_seqlens, output_final_state, output_dtype, segment_chunks)


def chunk_linear_attention_bwd(q, k, v, g, do, dht=None, scale=None, initial_state=None, cu_seqlens=None, *,
                               grad_dtype=None, segment_chunks=0):
    """Low-level backward.  Returns ``(dq, dk, dv, dg, dh0)``: dq, dk, dv in ``grad_dtype``
    (default: the dtype of q), dg float32 in the shape of g, dh0 float32 (None without
    initial_state).

    bfloat16 inputs with a float32 ``do`` are taken as float32, so that do is not rounded: several
    times slower than with ``do`` in bfloat16 (a forward with ``output_dtype=torch.bfloat16`` gets
    that).  Sums run in float32, those of dg in 64 bits.
    """
    return _gdr_torch.la_bwd(q, k, v, g, do, dht, scale, initial_state, cu_seqlens, grad_dtype, segment_chunks)


class _ChunkLA(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, scale, initial_state, output_final_state, cu_seqlens, output_dtype):
        o, ht = chunk_linear_attention_fwd(q, k, v, g, scale, initial_state, cu_seqlens, output_final_state,
                                           output_dtype=output_dtype)
        ctx.save_for_backward(q, k, v, g, initial_state, cu_seqlens)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, ht

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do, dht):
        q, k, v, g, h0, cu = ctx.saved_tensors
        if do is None:
            if dht is None:
                return (None,) * 9
            do = torch.zeros(v.shape, dtype=q.dtype, device=q.device)
        dq, dk, dv, dg, dh0 = chunk_linear_attention_bwd(q, k, v, g, do, dht, ctx.scale, h0, cu)
        return dq, dk, dv, dg.to(g.dtype), None, None if h0 is None else dh0.to(h0.dtype), None, None, None


def chunk_linear_attention(q, k, v, g, scale=None, initial_state=None, output_final_state=False, cu_seqlens=None, *,
                           output_dtype=torch.float32):
    """High-level differentiable API.  Returns ``(o, final_state)``.

    q, k [B,T,H_q,K], v [B,T,H_v,V] (bfloat16 or float32, K and V 64 or 128), g [B,T,H_v] or
    [H_v], initial_state [N,H_v,K,V]; packed sequences with ``cu_seqlens`` int32 [N+1].  The
    arguments are those of :func:`chunk_gated_delta_rule` without beta, and
    :func:`chunk_linear_attention_fwd` says more of them.  All five inputs have gradients
    (:func:`chunk_linear_attention_bwd`).  Training on bfloat16 inputs is several times faster
    with ``output_dtype=torch.bfloat16``: the gradient of a float32 output takes the inputs as
    float32."""
    if forward_ad._current_level >= 0 or torch.is_grad_enabled() and any(
            x is not None and x.requires_grad for x in (q, k, v, g, initial_state)):  # (forward mode is refused there)
        return _ChunkLA.apply(q, k, v, g, scale, initial_state, output_final_state, cu_seqlens, output_dtype)
    return chunk_linear_attention_fwd(q, k, v, g, scale, initial_state, cu_seqlens, output_final_state,
                                      output_dtype=output_dtype)
