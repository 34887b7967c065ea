"""GB300-native (sm_103a) DSA sparse decode attention over a paged KV cache.

The compute lives in libsdattn.so (CUDA kernels behind the C ABI of
include/sdattn.h); this package is its thin ctypes binding plus the seeded
synthetic workload generators (``inputs``).  Importing the package does not
load the library; the first call does, and raises if it is not built.
"""
from ._binding import (  # noqa: F401
    FLAG_BOUNDS,
    FLAG_FULL,
    FLAG_NONFINITE,
    FLAG_TIMEOUT,
    SdaError,
    declared_functions,
    default_workspace,
    load,
    no_alloc_read_errors,
    paged_workspace_bytes,
    quantised_workspace_bytes,
    read_errors,
    set_wait_limit_ns,
    sparse_decode_attention,
    sparse_decode_attention_no_alloc,
    sparse_decode_paged_attention,
    sparse_decode_plan_step,
    sparse_decode_quantised_append,
    sparse_decode_quantised_attention,
    sparse_decode_quantised_paged_attention,
    sparse_decode_quantised_read,
    sparse_decode_rope_append,
    sparse_decode_select_regions,
    sparse_decode_splits,
    sparse_decode_summary_scores,
    sparse_decode_swa_attention,
    sparse_decode_swa_splits,
    status_string,
    step_workspace,
    timeline_buffer,
    use_library,
    workspace_bytes,
)
