"""Hybrid-SWA dual-KV-pool attention for GB300 (sm_103a).

The library is ``_build/libhsa.so`` with the C ABI of ``include/hsa.h``; this
package is its thin Python binding.  Build it with ``__graft_entry__.build()``
(or ``python -m full_attention_kv_gb300.build``).
"""
from .binding import (  # noqa: F401
    EXPORTS, HSA_CUDA_ERROR, HSA_DECODE_APPEND, HSA_DECODE_EARLY_POOL_READ, HSA_DEVERR_BAD_BLOCK,
    HSA_DEVERR_BAD_LEN, HSA_DEVERR_BAD_PAGE, HSA_DEVERR_BAD_RING, HSA_DEVERR_BAD_SEQ,
    HSA_DEVERR_TIMEOUT, HSA_INVALID_ARG, HSA_KV_E4M3, HSA_KV_E5M2, HSA_OK, HSA_OUT_OF_RANGE,
    HSA_UNSUPPORTED_SHAPE, TREE_EXPORTS, DualPool, HsaError, HsaPools, HsaRopeParams, PrefixTree,
    Rope, decode_shared_workspace, decode_workspace, hsa_decode_attn, hsa_decode_attn_shared,
    hsa_decode_shared_workspace_bytes,
    fp8_code, hsa_decode_attn_append, hsa_decode_attn_noalloc, hsa_decode_workspace_bytes,
    hsa_kv_append, hsa_kv_compact, hsa_kv_select, decode_weights_workspace, hsa_decode_attn_weights,
    hsa_decode_weights_workspace_bytes, hsa_prefill_weights, hsa_prefill_weights_workspace_bytes,
    prefill_weights_workspace,
    hsa_prefill_attn, hsa_rope, hsa_rope_kv_append, hsa_swa_prefetch, hsa_window_safe_len, hsa_window_safe_len_bitmap, lib,
    status_string)
