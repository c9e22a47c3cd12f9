"""Serving operators of the gated delta rule on a pool of recurrent states.

A serving program keeps one K x V state (fp32) per (sequence, v head) in a pool
``states [n_slots, H_v, K, V]``, the layout of the chunked operator's initial and
final states, and names a sequence's state by its slot:

- :func:`recurrent_gated_delta_rule` takes every sequence's next token (or few
  tokens) into its state, in place;
- :func:`tree_gated_delta_rule` evaluates trees of drafted tokens against the
  states, which stay as they are, and :func:`tree_gated_delta_rule_accept` takes the
  accepted path into them;
- :func:`copy_states` copies, forks, moves and clears states.

They are inference operators: no gradients (the chunked operator has them), no
workspace, no synchronisation, and all of them may be captured into a graph.
``slots``, ``parents``, ``accepted`` and ``cu_seqlens`` are int32.  On the host
they are checked here; on the device the library clamps or skips what is out of
range (reading them here would synchronise the stream).
"""
import torch

from . import _lib
from .api import _DT, _c, check_offsets


# torch.cuda.current_stream(i).cuda_stream, current_device() and
# torch.autograd.graph.increment_version without what they wrap around these (2.5 us a call)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_increment_version = torch._C._increment_version


def _refuse_gradients():
    raise ValueError("the operators on a pool of states have no gradient: use chunk_gated_delta_rule, or torch.no_grad()")


def _rows(x, per16):
    """x with the elements between its tokens and between its batch rows, copied if the
    kernels cannot read it in place: they need one token's [H, D] contiguous and rows at
    multiples of 16 bytes (per16 elements), less than 2^23 elements apart."""
    B, T, H, D = x.shape
    batch, row, head, one = x.stride()
    if B < 2:
        batch = 0
    if T < 2:
        row = 0
    if one != 1 or (head != D and H > 1) or batch % per16 or row % per16 or row >= 1 << 23 or x.data_ptr() % 16:
        x = x.clone(memory_format=torch.contiguous_format)  # (also where it is contiguous, but unaligned)
        batch, row = T * H * D, H * D
    return x, row, batch


def _check_states(states, name="states"):
    if states.is_contiguous() and states.shape[0] and not states.data_ptr() % 16:
        return
    n, H, K, V = states.shape
    slot, head, row, one = states.stride()
    if n < 1 or one != 1 or row != V or (head != K * V and H > 1) or states.data_ptr() % 16 or \
            (n > 1 and (slot % 4 or slot < H * K * V)):
        raise ValueError("a slot of %s must be contiguous and 16-byte aligned" % name)


def _indices(x, n, what, lo, hi):
    """An int32 index array of n entries; on the host its range is checked."""
    if x.dtype != torch.int32 or x.dim() != 1 or x.numel() != n:
        raise ValueError("%s must be int32 [%d]" % (what, n))
    if not x.is_cuda and n and (int(x.min()) < lo or int(x.max()) >= hi):
        raise ValueError("%s out of range [%d, %d)" % (what, lo, hi))


def _check_distinct(slots):
    used = slots[slots >= 0]
    if used.unique().numel() != used.numel():
        raise ValueError("slots names a slot twice")


def _check_parents(parents, B, T, cu_seqlens):
    if parents.dtype != torch.int32 or parents.shape != (B, T):
        raise ValueError("parents must be int32 [B,T]")
    if cu_seqlens is None and T > _lib.TREE_MAX:
        raise ValueError("a tree has at most %d nodes" % _lib.TREE_MAX)
    lens = None
    if cu_seqlens is not None and not cu_seqlens.is_cuda:
        lens = (cu_seqlens[1:] - cu_seqlens[:-1]).long()
        if lens.numel() and int(lens.max()) > _lib.TREE_MAX:
            raise ValueError("a tree has at most %d nodes" % _lib.TREE_MAX)
    if not parents.is_cuda and (cu_seqlens is None or lens is not None):
        at = torch.arange(T, dtype=torch.int32).expand(B, T)
        if lens is not None:
            at = at - torch.repeat_interleave(cu_seqlens[:-1], lens)
        if bool((parents < -1).any()) or bool((parents >= at).any()):
            raise ValueError("a node's parent is -1 or an earlier node of its tree")


def _check_out(out, v, *inputs):
    if out.shape != v.shape or out.dtype not in _DT or not out.is_contiguous() or out.data_ptr() % 16:
        raise ValueError("out must be contiguous [B,T,H_v,V], bfloat16 or float32, 16-byte aligned")
    if out.device != v.device:
        raise ValueError("all tensors must be on one GPU")
    for x in (v,) + inputs:
        if _overlap(out, x):
            raise ValueError("out overlaps an input")


def _span(t):
    """First byte of a tensor and the byte past its last one."""
    a = t.data_ptr()
    return a, a + ((sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size() if t.numel() else 0)


def _overlap(a, b):
    (a0, a1), (b0, b1) = _span(a), _span(b)
    return a.device == b.device and a0 < b1 and b0 < a1


def _launch(call, args, dev, written):
    """`written`: what the kernels write in place.  Autograd is told, so that a backward that
    has saved it raises an error instead of using the new values."""
    index = dev.index
    if index == _current_device():
        call(args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            call(args, _raw_stream(index))
    if written:
        _increment_version(written)


def _on(x, dev):
    """An index array where the kernels read it."""
    if x.device != dev:
        x = x.to(dev)
    return x.contiguous()


def _run(call, q, k, v, g, beta, parents, accepted, states, scale, cu_seqlens, slots, output_dtype, out):
    """Checks the arguments of an operator and launches it; returns its output (None for an
    acceptance, which has no q).  Written out in one piece, since it runs once per token."""
    if k.dim() != 4 or v.dim() != 4 or (q is not None and q.shape != k.shape):
        raise ValueError("expected q, k [B,T,H_q,K] and v [B,T,H_v,V]")
    B, T, H_q, K = k.shape
    B_v, T_v, H_v, V = v.shape
    if B_v != B or T_v != T:
        raise ValueError("expected q, k [B,T,H_q,K] and v [B,T,H_v,V]")
    dtype = _DT.get(k.dtype)
    if dtype is None or v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        raise ValueError("q, k, v must share one dtype, bfloat16 or float32")
    tokens = (B, T, H_v)
    if g.shape != tokens or beta.shape != tokens:
        raise ValueError("g and beta must be [B,T,H_v]")
    n_seq = B
    if cu_seqlens is not None:
        if B != 1 or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be int32 [N+1] with B == 1")
        if not cu_seqlens.is_cuda:
            check_offsets(cu_seqlens, T)
        n_seq = cu_seqlens.numel() - 1
    if parents is not None:
        _check_parents(parents, B, T, cu_seqlens)
    if states.dtype != torch.float32 or states.dim() != 4 or states.shape[1:] != (H_v, K, V):
        raise ValueError("states must be float32 [n_slots,H_v,K,V]")
    _check_states(states)
    n_slots = states.shape[0]
    if slots is None:
        if n_slots < n_seq:
            raise ValueError("states has %d slots for %d sequences" % (n_slots, n_seq))
    else:
        _indices(slots, n_seq, "slots", -1, n_slots)
        if not slots.is_cuda and (parents is None or accepted is not None):
            _check_distinct(slots)  # (trees that are only read may share one)
    if accepted is not None:
        _indices(accepted, n_seq, "accepted", -1, _lib.TREE_MAX if cu_seqlens is not None else T)
    if torch.is_grad_enabled() and (k.requires_grad or v.requires_grad or g.requires_grad or beta.requires_grad
                                    or states.requires_grad or (q is not None and q.requires_grad)):
        _refuse_gradients()
    dev = states.device
    if dev.type != "cuda":
        raise ValueError("inputs must be on the GPU")
    if k.device != dev or v.device != dev or g.device != dev or beta.device != dev or (q is not None and q.device != dev):
        raise ValueError("all tensors must be on one GPU")
    o = None
    if q is not None:
        if out is not None:
            _check_out(out, v, q, k, g, beta, states)
            o = out
        elif output_dtype not in _DT:
            raise ValueError("output_dtype must be bfloat16 or float32")
        else:
            o = torch.empty_like(v, dtype=output_dtype, memory_format=torch.contiguous_format)
    # contiguous rows of 16-byte aligned tensors are read as they are; _rows looks at others
    per16 = 8 if dtype == _lib.BF16 else 4
    q_row, k_row, v_row = H_q * K, H_q * K, H_v * V
    q_batch, k_batch, v_batch = T * q_row, T * k_row, T * v_row
    kp, vp, qp = k.data_ptr(), v.data_ptr(), 0
    if kp % 16 or not k.is_contiguous():
        k, k_row, k_batch = _rows(k, per16)
        kp = k.data_ptr()
    if vp % 16 or not v.is_contiguous():
        v, v_row, v_batch = _rows(v, per16)
        vp = v.data_ptr()
    if q is not None:
        qp = q.data_ptr()
        if qp % 16 or not q.is_contiguous():
            q, q_row, q_batch = _rows(q, per16)
            qp = q.data_ptr()
    g, beta = _c(g, torch.float32), _c(beta, torch.float32)
    cu, sl, pa, ac = cu_seqlens, slots, parents, accepted
    if cu is not None:
        cu = _on(cu, dev)
    if sl is not None:
        sl = _on(sl, dev)
    if pa is not None:
        pa = _on(pa, dev)
    if ac is not None:
        ac = _on(ac, dev)
    args = _lib.PoolArgs(
        B, T, H_q, H_v, K, V, n_seq, n_slots, states.stride(0), q_row, k_row, v_row, q_batch, k_batch, v_batch,
        dtype, _lib.F32 if o is None else _DT[o.dtype], K ** -0.5 if scale is None else float(scale), qp, kp, vp, g.data_ptr(),
        beta.data_ptr(), None if cu is None else cu.data_ptr(), None if sl is None else sl.data_ptr(),
        None if pa is None else pa.data_ptr(), None if ac is None else ac.data_ptr(), states.data_ptr(),
        None if o is None else o.data_ptr())
    written = [states] if parents is None or accepted is not None else []
    if out is not None:
        written.append(out)
    _launch(call, args, dev, written)
    return o


def recurrent_gated_delta_rule(q, k, v, g, beta, states, scale=None, cu_seqlens=None, *, slots=None,
                               output_dtype=torch.float32, out=None):
    """The recurrent form: every sequence's tokens are taken into its state, in place.
    Returns ``o`` [B,T,H_v,V].

    q, k [B,T,H_q,K], v [B,T,H_v,V], g and beta [B,T,H_v] as for
    :func:`chunk_gated_delta_rule`, with B sequences of T tokens, or packed sequences
    with ``cu_seqlens``; the result is that of the chunked operator with the states as
    initial states and the final states written over them.  Meant for one token per
    sequence or a few (the state is read and written once a call, and the tokens are
    taken one after the other).  q, k and v may be slices of a wider projection: they
    are read in place where a token's heads are contiguous.

    ``states`` float32 [n_slots,H_v,K,V], the slots any distance apart; ``slots`` int32
    [N] names each sequence's slot (default: slot j for sequence j).  A sequence whose
    slot is negative (the padding of a batch) is skipped and its rows of ``o`` are
    zero; so is a sequence that names a slot which an earlier one has.  ``out``: a
    contiguous tensor to write; rows that belong to no sequence are left as they are.
    """
    return _run(_lib.step, q, k, v, g, beta, None, None, states, scale, cu_seqlens, slots, output_dtype, out)


def tree_gated_delta_rule(q, k, v, g, beta, parents, states, scale=None, cu_seqlens=None, *, slots=None,
                          output_dtype=torch.float32, out=None):
    """Trees of drafted tokens over the cached states, which are only read.  Returns
    ``o`` [B,T,H_v,V]: of every node, what :func:`recurrent_gated_delta_rule` would
    give for it after the nodes on its path.

    A sequence is one tree of at most 64 nodes: B trees of T nodes, or packed trees
    with ``cu_seqlens``.  ``parents`` int32 [B,T] holds the place of a node's parent
    among its tree's nodes, which come after their parents, or -1 for a child of the
    cached state; an entry that is no earlier node counts as -1.  A node influences
    its own row and its descendants', whatever its values.  Several trees may name one
    slot; a tree whose slot is negative gets rows of zeros, and a packed tree of more
    than 64 nodes rows of NaN.  The other arguments are those of
    :func:`recurrent_gated_delta_rule`.
    """
    return _run(_lib.tree, q, k, v, g, beta, parents, None, states, scale, cu_seqlens, slots, output_dtype, out)


def tree_gated_delta_rule_accept(k, v, g, beta, parents, accepted, states, cu_seqlens=None, *, slots=None):
    """Takes the tokens on the path to an accepted node into each sequence's state, in
    place, with the very results of :func:`recurrent_gated_delta_rule` on those tokens.
    Returns ``states``.

    k, v, g, beta, parents, cu_seqlens and slots as given to
    :func:`tree_gated_delta_rule`; ``accepted`` int32 [N] is the last accepted node of
    each tree, or -1 for none (the state then stays as it is).  A sequence that names
    a slot which an earlier one has is skipped.
    """
    _run(_lib.tree_accept, None, k, v, g, beta, parents, accepted, states, 1.0, cu_seqlens, slots, None, None)
    return states


def _check_pool(x, name):
    """One layer's pool, or [layers, ...] of them."""
    if x.dtype != torch.float32 or x.dim() not in (4, 5):
        raise ValueError("%s must be float32 [n_slots,H_v,K,V] or [layers,n_slots,H_v,K,V]" % name)
    if x.dim() == 5:
        n, inner = x.shape[0], x.shape[2] * x.shape[3] * x.shape[4]
        if n > 1 and (x.stride(0) % 4 or x.stride(0) < inner):
            raise ValueError("a slot of %s must be contiguous and 16-byte aligned" % name)
        if n > 0:
            _check_states(x[0], name)
    else:
        _check_states(x, name)


def copy_states(states, dst, src, source=None):
    """For every entry i, slot ``dst[i]`` of ``states`` becomes what slot ``src[i]`` of
    ``source`` (default: ``states``) was before the call, or zero where ``src[i]`` is
    -1.  Returns ``states``.

    One list of up to 4096 entries may thus fork a state (a source named several
    times), move, swap or reorder states within a pool, and clear slots for new
    sequences.  Entries with ``dst`` -1 are skipped; of entries with the same ``dst``
    the last one stands.  On the device, entries past either pool are skipped too.

    ``states`` and ``source``: float32 [n_slots,H_v,K,V], or [layers,n_slots,H_v,K,V]
    for the pools of several layers copied by the same list; ``dst``, ``src``: int32
    [n].  ``source`` may be another pool, such as the final states of a prefill; it
    must not overlap ``states`` in memory, unless it is the same pool.
    """
    _check_pool(states, "states")
    if source is None or source is states:
        source = states
    else:
        _check_pool(source, "source")
        if source.dim() != states.dim() or source.shape[-3:] != states.shape[-3:] or \
                (states.dim() == 5 and source.shape[0] != states.shape[0]):
            raise ValueError("states and source must hold states of one shape and as many layers")
        same = source.data_ptr() == states.data_ptr() and source.shape == states.shape and \
            source.stride() == states.stride()
        if not same and _overlap(states, source):
            raise ValueError("source overlaps states")
    n, n_dst, n_src = dst.numel(), states.shape[-4], source.shape[-4]
    if n > _lib.COPY_MAX:
        raise ValueError("at most %d entries" % _lib.COPY_MAX)
    _indices(dst, n, "dst", -1, n_dst)
    _indices(src, n, "src", -1, n_src)
    if torch.is_grad_enabled() and (states.requires_grad or source.requires_grad):
        _refuse_gradients()
    dev = states.device
    if dev.type != "cuda":
        raise ValueError("inputs must be on the GPU")
    if source.device != dev:
        raise ValueError("all tensors must be on one GPU")
    dst, src = _on(dst, dev), _on(src, dev)
    H, K, V = states.shape[-3:]
    layers, layer, source_layer = 1, 0, 0
    if states.dim() == 5:
        layers, layer, source_layer = states.shape[0], 4 * states.stride(0), 4 * source.stride(0)
    args = _lib.CopyArgs(n, n_dst, n_src, 4 * H * K * V, 4 * states.stride(-4), 4 * source.stride(-4), layers, layer,
                         source_layer, dst.data_ptr(), src.data_ptr(), states.data_ptr(), source.data_ptr())
    _launch(_lib.copy_states, args, dev, [states])
    return states
