"""GB300-native (sm_103a) chunked forward pass of Kimi Delta Attention (KDA), and the
operators that serve a model around it: the single-token KDA step, linear attention with
one decay per head (chunked and single-token), and the norms of a layer.

The compute lives in libkda.so (hand-written CUDA behind the C ABI of
include/kda.h); this package is its thin Python binding plus the seeded
synthetic workloads. Importing the package does not load the library: the
first call does, and fails loudly if libkda.so has not been built.
"""
from .kda import (fwd, fwd_noalloc, NOALLOC_MAX_SCRATCH, workspace_size, debug_chunk_matrices, device_status,  # noqa: F401
                  max_chunks, plan, CP_OFF, CP_SEGMENTS)
from .serving import add_norm, la_fwd, la_step, la_workspace_size, norm_gate, step  # noqa: F401

__version__ = "0.1.0"
