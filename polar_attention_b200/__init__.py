"""B200 (sm_100a) Polar Attention: fused causal prefill, GQA paged decode (single
tokens, chunks, drafted trees, selected pages), the paged KV cache's own
operations and the gated-delta memory channel.

The computation lives in libpolar_attn.so (hand-written CUDA for sm_100a behind
the C ABI of include/polar_attn.h, include/polar_cache.h and
include/polar_gdelta.h); ``native`` is its thin ctypes binding and ``workloads``
the seeded synthetic inputs.  The library is loaded on first use, and a missing
build raises: there is no CPU or PyTorch fallback.
"""
from .native import (bwd, bwd_from_state, bwd_workspace_size,  # noqa: F401
                     cache_append, cache_compact, cache_fork, cache_free, cache_reserve,
                     cache_workspace_size, decode_chunk_workspace_size,
                     decode_paged, decode_paged_chunk,
                     decode_paged_host, decode_paged_sparse, decode_paged_tree,
                     decode_sparse_workspace_size, decode_staging_size,
                     decode_tree_workspace_size, decode_workspace_size, fwd, fwd_host,
                     fwd_staging_size, fwd_state_size, fwd_train, fwd_workspace_size,
                     gdelta_prefill, gdelta_step,
                     gdelta_workspace_size, get_status,
                     launch_count, PageCache, PolarError)

__all__ = ["fwd", "bwd", "bwd_workspace_size", "fwd_train", "bwd_from_state", "fwd_state_size",
           "fwd_host", "fwd_staging_size", "fwd_workspace_size", "decode_paged",
           "decode_paged_chunk", "decode_chunk_workspace_size", "decode_paged_host",
           "decode_staging_size", "decode_workspace_size", "gdelta_prefill", "gdelta_step",
           "gdelta_workspace_size", "get_status", "launch_count",
           "decode_paged_tree", "decode_tree_workspace_size", "decode_paged_sparse",
           "decode_sparse_workspace_size", "PageCache", "cache_reserve", "cache_append",
           "cache_fork", "cache_free", "cache_compact", "cache_workspace_size",
           "PolarError"]
