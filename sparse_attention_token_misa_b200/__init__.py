"""B200-native (sm_100a) MISA / MISA-dagger / HISA token indexer, and the
sparse attention over the tokens it selects.

The compute path is libmisa.so (C ABI in include/misa.h, CUDA kernels under
csrc/); this package is its Python binding: the same entry points taking torch
device tensors (`_native`), the four indexers as preallocated call sequences
(`indexer`), and the latent cache in 16, 8 or 4 bits with the attention that
reads it (`latent`).
"""
from . import _native
from ._native import (MisaError, alloc_workspace, append_keys, block_stats, error_query, error_reset,  # noqa: F401
                      gather_candidates, hier_rerank, hisa_block_filter, index_decode, index_score, index_score_blocks, lib, num_windows,
                      route_heads,
                      shard_prefix, sparse_mla, topk, workspace_bytes)
from .indexer import DenseIndexer, HisaIndexer, MisaDaggerIndexer, MisaIndexer  # noqa: F401
from ._native import OP_APPEND_KV, OP_PREFIX_MLA, OP_READ_KV, OP_SPARSE_MLA_Q  # noqa: F401
from .latent import (LatentCache, alloc_kv_cache, append_kv, kv_row_bytes, prefix_mla, read_kv,  # noqa: F401
                     sparse_mla_q)
from .sharded import ShardedMisaIndexer, TorchShardComm, shard_bounds  # noqa: F401

__all__ = [
    "MisaError", "alloc_workspace", "append_keys", "block_stats", "error_query", "error_reset",
    "gather_candidates", "hier_rerank", "shard_prefix", "ShardedMisaIndexer", "TorchShardComm", "shard_bounds",
    "hisa_block_filter", "index_decode", "index_score", "index_score_blocks", "lib", "num_windows", "route_heads", "sparse_mla", "topk", "workspace_bytes",
    "LatentCache", "alloc_kv_cache", "append_kv", "kv_row_bytes", "prefix_mla", "read_kv", "sparse_mla_q",
    "OP_APPEND_KV", "OP_PREFIX_MLA", "OP_READ_KV", "OP_SPARSE_MLA_Q",
    "DenseIndexer", "HisaIndexer", "MisaDaggerIndexer", "MisaIndexer",
]
