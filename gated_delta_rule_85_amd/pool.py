"""Serving operators of the gated delta rule and of linear attention on a pool of recurrent states.

A serving program keeps one K x V state (fp32) per (sequence, v head) in a pool
``states [n_slots, H_v, K, V]``, the layout of the chunked operator's initial and
final states, and names a sequence's state by its slot:

- :func:`recurrent_gated_delta_rule` takes every sequence's next token (or few
  tokens) into its state, in place;
- :func:`tree_gated_delta_rule` evaluates trees of drafted tokens against the
  states, which stay as they are, and :func:`tree_gated_delta_rule_accept` takes the
  accepted path into them;
- :func:`recurrent_linear_attention` is the first of these for linear attention with a
  decay for each head;
- :func:`copy_states` copies, forks, moves and clears states.

They are inference operators: no gradients (the chunked operator has them), no
workspace, and all of them may be captured into a graph.  ``slots``, ``parents``,
``accepted``, ``cu_seqlens``, ``dst`` and ``src`` are int32.  On the device nothing
waits for them: the library clamps or skips what is out of range (reading them here
would synchronise the stream).  On the host their values are checked, and the copy to
the device waits for the stream's earlier work and cannot be captured.
"""
import torch

from . import _lib


class _NotBuilt:
    """Stands for the compiled binding where it cannot be imported: the chunked operator does
    not need it, and the operators here raise ImportError when they are called."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError("_gdr_torch.so is not built for this interpreter and torch (%s); run `python "
                          "gated_delta_rule_85_amd/build.py` or __graft_entry__.build() first" % self._why)


# the functions below are called once per layer and token: their checks are in csrc/gdr_torch.cpp
try:
    from . import _gdr_torch
    _gdr_torch.connect(_lib.GdrError, torch._C._cuda_getCurrentRawStream)
except (ImportError, AttributeError) as e:  # (a torch without that function)
    _gdr_torch = _NotBuilt(e)


def recurrent_gated_delta_rule(q, k, v, g, beta, states, scale=None, cu_seqlens=None, *, slots=None,
                               output_dtype=torch.float32, out=None):
    """The recurrent form: every sequence's tokens are taken into its state, in place.
    Returns ``o`` [B,T,H_v,V].

    q, k [B,T,H_q,K], v [B,T,H_v,V], g and beta [B,T,H_v] as for
    :func:`chunk_gated_delta_rule`, with B sequences of T tokens, or packed sequences
    with ``cu_seqlens``; the result is that of the chunked operator with the states as
    initial states and the final states written over them.  Meant for one token per
    sequence or a few: the state is read and written once a call and the tokens are
    taken one after the other, which is faster than the chunked operator up to about 16
    tokens a sequence.  q, k and v may be slices of a wider projection: they
    are read in place where a token's heads are contiguous.

    ``states`` float32 [n_slots,H_v,K,V], the slots any distance apart; ``slots`` int32
    [N] names each sequence's slot (default: slot j for sequence j).  A sequence whose
    slot is negative (the padding of a batch) is skipped and its rows of ``o`` are
    zero; so is a sequence that names a slot which an earlier one has (every sequence
    looks through the slots before its own, which shows from about ten thousand on: 32768
    sequences of two 64 x 64 heads take 540 us a step, 368 without ``slots``).  ``out``: a
    contiguous tensor to write; rows that belong to no sequence are left as they are.
    """
    return _gdr_torch.step(q, k, v, g, beta, states, scale, cu_seqlens, slots, output_dtype, out)


def recurrent_linear_attention(q, k, v, g, states, scale=None, cu_seqlens=None, *, slots=None,
                               output_dtype=torch.float32, out=None):
    """The recurrent form of :func:`chunk_linear_attention`: every sequence's tokens are taken
    into its state, in place.  Returns ``o`` [B,T,H_v,V].

    g is [B,T,H_v] or, fixed for each v head, [H_v]; there is no beta.  The other arguments,
    and what happens to sequences without a slot, are those of
    :func:`recurrent_gated_delta_rule`.
    """
    return _gdr_torch.la_step(q, k, v, g, states, scale, cu_seqlens, slots, output_dtype, out)


def tree_gated_delta_rule(q, k, v, g, beta, parents, states, scale=None, cu_seqlens=None, *, slots=None,
                          output_dtype=torch.float32, out=None):
    """Trees of drafted tokens over the cached states, which are only read.  Returns
    ``o`` [B,T,H_v,V]: of every node, what :func:`recurrent_gated_delta_rule` would
    give for it after the nodes on its path.

    A sequence is one tree of at most 64 nodes: B trees of T nodes, or packed trees
    with ``cu_seqlens``.  ``parents`` int32 [B,T] holds the place of a node's parent
    among its tree's nodes, which come after their parents, or -1 for a child of the
    cached state; an entry that is no earlier node counts as -1.  A node influences
    its own row and its descendants' only, whatever its values; where a value on a node's
    path is not finite, or a product of values on it (of q and keys, or the e^g from the
    state or an ancestor to the node: gates that add up to more than 88) passes 1.6e38,
    the node's row may be NaN (values of q, k and the state past bfloat16's 3.39e38 count
    as infinite).  Several trees may name one slot; a tree whose slot is negative gets
    rows of zeros, and a packed tree of more than 64 nodes rows of NaN.  The other arguments are those of
    :func:`recurrent_gated_delta_rule`.
    """
    return _gdr_torch.tree(q, k, v, g, beta, parents, states, scale, cu_seqlens, slots, output_dtype, out)


def tree_gated_delta_rule_accept(k, v, g, beta, parents, accepted, states, cu_seqlens=None, *, slots=None):
    """Takes the tokens on the path to an accepted node into each sequence's state, in
    place, with the very results of :func:`recurrent_gated_delta_rule` on those tokens.
    Returns ``states``.

    k, v, g, beta, parents, cu_seqlens and slots as given to
    :func:`tree_gated_delta_rule`; ``accepted`` int32 [N] is the last accepted node of
    each tree, or -1 for none (the state then stays as it is).  A sequence that names
    a slot which an earlier one has is skipped.
    """
    return _gdr_torch.accept(k, v, g, beta, parents, accepted, states, cu_seqlens, slots)


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
    must not overlap ``states`` in memory, unless it is the same pool; the states of two
    pools of equal strides may lie between each other's.
    """
    return _gdr_torch.copy(states, dst, src, source)
