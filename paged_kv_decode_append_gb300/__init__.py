"""Paged KV-cache decode + append attention for GB300 (sm_103a).

The product is the C-ABI library ``libpkv.so`` (``include/pkv.h``); this
package holds its CUDA sources (``csrc/``), the build step, the thin ctypes
binding (``api``) and the seeded synthetic workload generators
(``workloads``).
"""
from .api import (  # noqa: F401
    HND,
    ROPE_HALF,
    ROPE_INTERLEAVED,
    DecodeStep,
    LayerCaches,
    NHD,
    PagePool,
    PkvError,
    cache_desc,
    decode_workspace,
    device_pool,
    default_decode_max_qlen,
    mass_workspace,
    mixed_workspace,
    pkv_append,
    pkv_attn_mass,
    pkv_decode_bucket,
    pkv_decode_attn,
    pkv_decode_workspace_size,
    pkv_evict_apply,
    pkv_evict_plan,
    pkv_mass_workspace_size,
    pkv_mixed_attn,
    pkv_mixed_workspace_size,
    pkv_pool_bytes,
    pkv_prefill_attn,
    pkv_prefill_workspace_size,
    pkv_rope,
    pkv_rope_append,
    pkv_table_update,
    pkv_tree_accept,
    pkv_tree_attn,
    pkv_tree_build,
    pkv_tree_commit,
    pkv_tree_workspace_size,
    prefill_workspace,
    pkv_validate_host,
    rope_freqs,
    tree_workspace,
)
