"""GB300 (sm_103a) Kimi Delta Attention prefill / MTP verify.

The compute lives in libkda.so (C ABI, include/kda.h); ``kda`` is its ctypes
binding, and ``ops`` that of the operators around KDA (include/kda_ops.h): the
short causal convolution, the query / key norm with rotation, the attention of
prompts and of drafted tokens over a paged cache, the residual stream's norm, and the
moves in caches and pools that verified trees and forked requests need.  Importing
this package loads nothing; the library is loaded on the first call and its absence
is an error, never a fallback.
"""
from .kda import (CHUNK, HEAD_DIM, KdaError, host_staging_size, kda_prefill,  # noqa: F401
                  overrides, prefill_schedule,
                  kda_prefill_host, kda_verify, lib, status_string, workspace_layout,
                  workspace_size)
from .ops import (chunk_attention_schedule, kda_cache_commit, kda_chunk_attention, kda_pool_copy,  # noqa: F401
                  kda_qk_norm_rope, kda_residual_norm, kda_short_conv, kda_tree_attention,
                  rope_frequencies, tree_attention_schedule, tree_mask)
