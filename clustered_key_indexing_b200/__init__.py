"""B200 (sm_100a) Latent Sparse Attention: indexer + attention path.

Thin PyTorch-facing binding of liblsa.so (include/lsa.h).  PyTorch only
allocates device memory and provides streams; every step runs in the
library's CUDA kernels.  See `api` for the calls.
"""
from .api import (Cache, Config, Decode, KernelTimer, KV8, Tree, attn_backward, build_buckets, build_tree, check_device_error,
                  fit_pca, kv8_attn, kv8_attn_workspace_bytes, kv8_copy_pages, kv8_sparse_attn,
                  kv8_sparse_attn_workspace_bytes, kv8_write, lse_combine, prefill, prefill_chunk, prefill_host, prefill_workspace_bytes, query_latent,
                  select, select_attn, select_attn_workspace_bytes, select_workspace_bytes, shard_build_buckets,
                  shard_cand_cap, shard_candidates, shard_merge, sparse_attn, sparse_attn_partial)
from .pages import KV8Pages

__all__ = ["Cache", "Config", "Decode", "KernelTimer", "KV8", "KV8Pages", "Tree", "attn_backward", "build_buckets", "build_tree", "check_device_error",
           "fit_pca", "kv8_attn", "kv8_attn_workspace_bytes", "kv8_copy_pages", "kv8_sparse_attn",
           "kv8_sparse_attn_workspace_bytes", "kv8_write", "lse_combine", "prefill", "prefill_chunk", "prefill_host", "prefill_workspace_bytes",
           "query_latent", "select", "select_attn", "select_attn_workspace_bytes", "select_workspace_bytes",
           "shard_build_buckets", "shard_cand_cap", "shard_candidates", "shard_merge", "sparse_attn",
           "sparse_attn_partial"]
