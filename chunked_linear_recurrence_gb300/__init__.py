"""GB300-native chunk-parallel gated delta rule with boundary-state passing.

The computation lives in ``libsf_gdn.so`` (hand-written sm_103a CUDA behind the
C ABI in ``include/sf_gdn.h``); this package is its thin ctypes binding, with
the same entry-point names:

* ``sf_gdn_chunk_fwd``        -- chunk_gdn forward (output + final state)
* ``sf_gdn_paged_chunk_fwd``  -- the forward advancing a paged state cache in place
* ``sf_gdn_segment_summary``  -- affine map S_out = S_in @ P + S_ext of token ranges
* ``sf_state_scan``           -- exclusive scan of segment maps -> entry states
* ``sf_gdn_chunk_bwd``        -- gradients w.r.t. q, k, v, gate, beta, initial state
* ``sf_gdn_segment_reverse_summary`` -- cotangent map dS_entry = dS_exit @ P^T + C of segments
* ``sf_state_scan_reverse``   -- reverse scan of cotangent maps -> segment exit cotangents

and, for the layers around it (``include/sf_linattn.h``),

* ``sf_linattn_chunk_fwd``, ``sf_linattn_paged_chunk_fwd``, ``sf_linattn_chunk_bwd``
                              -- linear attention with a decay for each head
* ``sf_linattn_step``, ``sf_gdn_step`` -- one token of every sequence on the paged state pool
* ``sf_qk_norm_rope_fwd``, ``sf_qk_norm_rope_bwd`` -- norm of each query/key head and the
                              position rotation (one or several axes) in one pass

and, for decoding several tokens at a time on that pool (``include/sf_decode.h``),

* ``sf_gdn_draft_step``, ``sf_linattn_draft_step`` -- outputs of drafted tokens, after the pool
                              has been advanced by the tokens accepted before
* ``sf_gdn_commit``, ``sf_linattn_commit`` -- that advance alone
* ``sf_draft_verify``         -- drafted tokens against the target's probabilities
* ``sf_state_copy``, ``sf_state_fork``, ``sf_state_compact`` -- the pool's slots copied, forked and
                              moved together

Build the library with ``python -m chunked_linear_recurrence_gb300.build``.
"""
from ._native import (SfError, load, sf_gdn_chunk_bwd, sf_gdn_chunk_fwd,  # noqa: F401
                      sf_gdn_paged_chunk_fwd, sf_gdn_segment_reverse_summary, sf_gdn_segment_summary, sf_state_scan,
                      sf_state_scan_reverse, sf_validate_cu_seqlens, sf_workspace_status)
from ._decode import (sf_draft_verify, sf_gdn_commit, sf_gdn_draft_step,  # noqa: F401
                      sf_linattn_commit, sf_linattn_draft_step, sf_state_compact, sf_state_copy,
                      sf_state_fork, sf_state_workspace)
from ._linattn import (sf_gdn_step, sf_linattn_bwd_workspace, sf_linattn_chunk_bwd,  # noqa: F401
                       sf_linattn_chunk_fwd, sf_linattn_fwd_workspace,
                       sf_linattn_paged_chunk_fwd, sf_linattn_step, sf_qk_norm_rope_bwd,
                       sf_qk_norm_rope_bwd_workspace, sf_qk_norm_rope_fwd)

__all__ = ["SfError", "load", "sf_gdn_chunk_fwd", "sf_gdn_paged_chunk_fwd",
           "sf_gdn_segment_summary", "sf_state_scan",
           "sf_gdn_chunk_bwd", "sf_gdn_segment_reverse_summary", "sf_state_scan_reverse",
           "sf_validate_cu_seqlens", "sf_workspace_status",
           "sf_linattn_chunk_fwd", "sf_linattn_paged_chunk_fwd", "sf_linattn_chunk_bwd",
           "sf_linattn_step", "sf_gdn_step", "sf_qk_norm_rope_fwd", "sf_qk_norm_rope_bwd",
           "sf_linattn_fwd_workspace", "sf_linattn_bwd_workspace",
           "sf_qk_norm_rope_bwd_workspace",
           "sf_gdn_draft_step", "sf_linattn_draft_step", "sf_gdn_commit", "sf_linattn_commit",
           "sf_draft_verify", "sf_state_copy", "sf_state_fork", "sf_state_compact",
           "sf_state_workspace"]
