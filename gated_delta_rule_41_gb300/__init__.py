"""GB300-native Kimi Delta Attention (KDA) chunk scan and decode step, the
paged key-value cache of the softmax-attention layers of a KDA:GQA hybrid, and
what stands around a mixing layer (gated recurrence, norms, 8-bit activations).

The compute lives in ``libkda.so`` (hand-written CUDA for sm_103a behind a C
ABI declared in ``include/kda.h``).  ``gated_delta_rule_41_gb300.kda``,
``.paged`` and ``.block`` are the thin Python binding: they marshal torch tensors
into the C calls and nothing else.  The library is loaded on first use; if it is missing, every call
raises instead of falling back to another implementation.
"""
from .kda import (  # noqa: F401
    KdaError, SavedForward, chunk_kda_fwd, chunk_kda_bwd, chunk_kda_fwd_varlen,
    chunk_kda_bwd_varlen, recurrent_step, workspace_bytes,
    library_path,
    load_library, check, timing_enable, timing_read,
)
from .paged import (  # noqa: F401
    KVPages, PageBook, paged_append, paged_decode, paged_decode_workspace, paged_prefill,
    paged_prefill_workspace, pages_copy,
)
from .block import (  # noqa: F401
    Packed8, add_norm_bwd, add_norm_fwd, gated_norm_bwd, gated_norm_fwd, gated_scan_bwd,
    gated_scan_fwd, gated_scan_step, pack8, unpack8,
)
