"""MI355X (gfx950) gated delta rule: chunked prefill with its backward, and the
recurrent operators that serve from its states.

The operator (FlashQLA's GDN chunked prefill) runs in libgdr.so, hand-written
HIP kernels behind the C ABI of include/gdr.h; this package is a thin
PyTorch-facing binding of it (ctypes, and compiled for the calls of a decode
step).
"""
from .api import (SavedForBackward, chunk_bound, chunk_gated_delta_rule, chunk_gated_delta_rule_bwd,
                  chunk_gated_delta_rule_fwd, num_chunks)
from .pool import (copy_states, recurrent_gated_delta_rule, tree_gated_delta_rule,
                   tree_gated_delta_rule_accept)

__all__ = ["chunk_gated_delta_rule", "chunk_gated_delta_rule_fwd", "chunk_gated_delta_rule_bwd",
           "num_chunks", "chunk_bound", "SavedForBackward", "recurrent_gated_delta_rule",
           "tree_gated_delta_rule", "tree_gated_delta_rule_accept", "copy_states"]
