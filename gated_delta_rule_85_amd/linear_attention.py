"""Linear attention with a decay for each head, in chunks, and its backward.

The gated delta rule without its correction: per (sequence, v head)

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t,

with the same states [K,V], head groups, gates and packed sequences as
:func:`chunk_gated_delta_rule`.  ``g`` is per token and v head, [B,T,H_v], or fixed for
each v head, [H_v].  The recurrent form on a pool of states is
:func:`recurrent_linear_attention`.  Every step runs in libgdr's HIP kernels.
"""
import math

import torch
from torch.autograd import forward_ad

from . import _lib
from .api import _DT, _c, _ptr, check_offsets


def _check(q, k, v, g, cu_seqlens, initial_state=None, **others):
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:2] != q.shape[:2]:
        raise ValueError("expected q, k [B,T,H_q,K] and v [B,T,H_v,V]")
    if q.dtype not in _DT or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype, bfloat16 or float32")
    B, T, Hv, V = v.shape
    if g.shape != (B, T, Hv) and g.shape != (Hv,):
        raise ValueError("g must be [B,T,H_v] or [H_v]")
    if not g.is_floating_point():
        raise ValueError("g must be floating point")
    if cu_seqlens is not None and (B != 1 or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1
                                   or cu_seqlens.numel() < 1):
        raise ValueError("cu_seqlens must be int32 [N+1] with B == 1")
    if cu_seqlens is not None and not cu_seqlens.is_cuda:
        # offsets on the host are checked here; on the device the library clamps them
        check_offsets(cu_seqlens, T)
    n_seq = B if cu_seqlens is None else cu_seqlens.numel() - 1
    for name, x in (("initial_state", initial_state), ("dht", others.get("dht"))):
        if x is not None and x.shape != (n_seq, Hv, q.shape[3], V):
            raise ValueError("%s must be [N,H_v,K,V]" % name)
    if others.get("do") is not None and others["do"].shape != v.shape:
        raise ValueError("do must be [B,T,H_v,V]")
    if not q.is_cuda:
        raise ValueError("inputs must be on the GPU")
    for x in (k, v, g, initial_state, *others.values()):
        if x is not None and x.device != q.device:
            raise ValueError("all tensors must be on one GPU")
    if cu_seqlens is not None and cu_seqlens.is_cuda and cu_seqlens.device != q.device:
        raise ValueError("all tensors must be on one GPU")
    return n_seq


def _rows(x):
    """x [B,T,H,D] where the kernels can read it in place (a token's heads contiguous, rows at
    multiples of 16 bytes less than 2^23 elements apart), else a contiguous copy."""
    B, T, H, D = x.shape
    per16 = 16 // x.element_size()
    batch, row = (x.stride(0) if B > 1 else 0), (x.stride(1) if T > 1 else 0)
    if not (x.stride(3) == 1 and (H < 2 or x.stride(2) == D) and batch % per16 == 0 and row % per16 == 0
            and row < 1 << 23 and x.data_ptr() % 16 == 0):
        x, batch, row = x.clone(memory_format=torch.contiguous_format), T * H * D, H * D
    return x, row, batch


def _floats(x):
    """x as the kernels read it: float32, contiguous, 16-byte aligned."""
    x = _c(x, torch.float32)
    return x.clone() if x is not None and x.data_ptr() % 16 else x


def _fill(a, q, k, v, g, scale, h0, cu, n_seq, segment_chunks):
    """The arguments that both directions share; returns what has to outlive the call."""
    B, T, Hq, K = q.shape
    a.B, a.T, a.H_q, a.H_v, a.K, a.V, a.n_seq = B, T, Hq, v.shape[2], K, v.shape[3], n_seq
    a.dtype, a.scale = _DT[q.dtype], 1.0 / math.sqrt(K) if scale is None else float(scale)
    a.g_per_head, a.segment_chunks = int(g.dim() == 1), int(segment_chunks)
    (q, a.q_row, a.q_batch), (k, a.k_row, a.k_batch), (v, a.v_row, a.v_batch) = _rows(q), _rows(k), _rows(v)
    g, h0 = _floats(g), _floats(h0)
    cu = None if cu is None else _c(cu).to(q.device)
    a.q, a.k, a.v, a.g, a.initial_state, a.cu_seqlens = _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(h0), _ptr(cu)
    return q, k, v, g, h0, cu


def _workspace(a, nbytes, dev):
    if nbytes == 0:
        return None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes
    return ws


def chunk_linear_attention_fwd(q, k, v, g, scale=None, initial_state=None, cu_seqlens=None, output_final_state=True,
                               *, output_dtype=torch.float32, segment_chunks=0):
    """Low-level forward.  Returns ``(o, final_state)``: o [B,T,H_v,V] in ``output_dtype``,
    final_state [N,H_v,K,V] float32 (None unless output_final_state).

    q, k and v may be slices of a wider projection: they are read in place where a token's
    heads are contiguous.  A long sequence of few heads is split into segments of
    ``segment_chunks`` chunks of 64 tokens (0: chosen for the device; the split is exact: a
    segment's part of the state is carried on by a scalar decay).  A gate of -104 or less,
    -inf among them, empties the state.  Rows of o that belong to no sequence are undefined.
    """
    n_seq = _check(q, k, v, g, cu_seqlens, initial_state)
    if output_dtype not in _DT:
        raise ValueError("output_dtype must be bfloat16 or float32")
    dev = q.device
    with torch.cuda.device(dev):
        a = _lib.LaFwdArgs()
        held = _fill(a, q, k, v, g, scale, initial_state, cu_seqlens, n_seq, segment_chunks)
        o = torch.empty(v.shape, dtype=output_dtype, device=dev)
        ht = None
        if output_final_state:
            ht = torch.empty((n_seq, v.shape[2], q.shape[3], v.shape[3]), dtype=torch.float32, device=dev)
        a.out_dtype, a.o, a.final_state = _DT[output_dtype], _ptr(o), _ptr(ht)
        held += (_workspace(a, _lib.la_fwd_workspace(a), dev),)
        _lib.la_fwd(a, torch.cuda.current_stream(dev).cuda_stream)
    return o, ht


def chunk_linear_attention_bwd(q, k, v, g, do, dht=None, scale=None, initial_state=None, cu_seqlens=None, *,
                               grad_dtype=None, segment_chunks=0):
    """Low-level backward.  Returns ``(dq, dk, dv, dg, dh0)``: dq, dk, dv in ``grad_dtype``
    (default: the dtype of q), dg float32 in the shape of g, dh0 float32 (None without
    initial_state).

    bfloat16 inputs with a float32 ``do`` are taken as float32, so that do is not rounded: several
    times slower than with ``do`` in bfloat16 (a forward with ``output_dtype=torch.bfloat16`` gets
    that).  Sums run in float32, those of dg in 64 bits.
    """
    n_seq = _check(q, k, v, g, cu_seqlens, initial_state, do=do, dht=dht)
    gdt = q.dtype if grad_dtype is None else grad_dtype
    if gdt not in _DT:
        raise ValueError("grad_dtype must be bfloat16 or float32")
    dev = q.device
    with torch.cuda.device(dev):
        if do.dtype != q.dtype:
            if q.dtype == torch.bfloat16:
                q, k, v = q.float(), k.float(), v.float()
            do = do.to(q.dtype)
        a = _lib.LaBwdArgs()
        held = _fill(a, q, k, v, g, scale, initial_state, cu_seqlens, n_seq, segment_chunks)
        do, dht = _c(do), _floats(dht)
        if do.data_ptr() % 16:
            do = do.clone()
        dq, dk = torch.empty(q.shape, dtype=gdt, device=dev), torch.empty(q.shape, dtype=gdt, device=dev)
        dv = torch.empty(v.shape, dtype=gdt, device=dev)
        dg = torch.empty(g.shape, dtype=torch.float32, device=dev)
        dh0 = None
        if initial_state is not None:
            dh0 = torch.empty(initial_state.shape, dtype=torch.float32, device=dev)
        a.grad_dtype, a.dout, a.dht = _DT[gdt], _ptr(do), _ptr(dht)
        a.dq, a.dk, a.dv, a.dg, a.dh0 = _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dh0)
        held += (_workspace(a, _lib.la_bwd_workspace(a), dev),)
        _lib.la_bwd(a, torch.cuda.current_stream(dev).cuda_stream)
    return dq, dk, dv, dg, dh0


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
    (:func:`chunk_linear_attention_bwd`)."""
    if forward_ad._current_level >= 0 or torch.is_grad_enabled() and any(
            x is not None and x.requires_grad for x in (q, k, v, g, initial_state)):  # (forward mode is refused there)
        return _ChunkLA.apply(q, k, v, g, scale, initial_state, output_final_state, cu_seqlens, output_dtype)
    return chunk_linear_attention_fwd(q, k, v, g, scale, initial_state, cu_seqlens, output_final_state,
                                      output_dtype=output_dtype)
