"""Top-k sparse decode attention over a paged KV cache, for NVIDIA B200 (sm_100a).

The computation lives in ``libsd.so`` (hand-written CUDA kernels behind the C
ABI of ``include/sd_api.h``); this package is a thin ctypes binding over it
plus the seeded synthetic-input generator used by tests and benchmarks.
"""
from .api import (  # noqa: F401
    EXPORTED,
    KvCache,
    NOALLOC_MAX_SCORES,
    SD_DEVERR_INDEX,
    SD_DEVERR_PAGE,
    SD_DEVERR_SEQLEN,
    SD_DEVERR_TIMEOUT,
    SD_KV_BF16,
    SD_KV_E4M3,
    SD_KV_INT8,
    SdError,
    TRI_PER_HEAD,
    TRI_PER_LAYER_PER_HEAD,
    TRI_UNION,
    StageTimer,
    alloc_block_step_workspace,
    alloc_block_topk_workspace,
    alloc_kv_attn_workspace,
    alloc_kv_cache,
    alloc_workspace,
    device_errors,
    last_launch_count,
    load_library,
    sd_block_topk,
    sd_decode_step,
    sd_decode_step_hinted,
    sd_indexer_topk,
    sd_indexer_topk_hinted,
    sd_indexer_topk_noalloc,
    sd_kv_attn,
    sd_kv_block_step,
    sd_kv_load,
    sd_kv_store,
    sd_sparse_attn,
    sd_sparse_attn_csr,
    sd_sparse_attn_layers,
    sd_tri_compact,
    sd_tri_compact_layers,
    set_wait_limit,
    workspace_size,
)

__all__ = [
    "sd_indexer_topk", "sd_indexer_topk_hinted", "sd_indexer_topk_noalloc", "sd_decode_step_hinted", "sd_sparse_attn", "sd_sparse_attn_layers", "sd_sparse_attn_csr",
    "sd_decode_step", "sd_tri_compact", "sd_tri_compact_layers", "TRI_UNION", "TRI_PER_HEAD",
    "TRI_PER_LAYER_PER_HEAD", "KvCache", "alloc_kv_cache", "sd_kv_store", "sd_kv_load", "sd_kv_attn", "sd_block_topk",
    "sd_kv_block_step", "alloc_kv_attn_workspace", "alloc_block_topk_workspace", "alloc_block_step_workspace",
    "SD_KV_BF16", "SD_KV_INT8", "SD_KV_E4M3",
    "workspace_size", "alloc_workspace", "device_errors", "set_wait_limit", "load_library", "SdError", "StageTimer",
]
