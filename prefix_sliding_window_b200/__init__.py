"""Prefix Sliding attention hot path for NVIDIA B200 (sm_100a).

The compute lives in libps.so (C ABI, include/ps.h): the KV append with Continue-PE RoPE,
the split-K decode over the pinned prefix plus the W-slot ring, the full-attention
comparator, the masked (two-level filtered) prefill, the per-head norm with rotary positions
(forward and backward) and the 4-bit store with its decode.  ``binding`` is the thin ctypes
layer over it; ``cache`` allocates the caller-owned buffers with PyTorch.
"""
from . import binding  # noqa: F401
from .binding import (  # noqa: F401
    PsError,
    make_cache,
    make_cache_q4,
    make_norm,
    make_params,
    make_rope,
    ps_decode_attn,
    ps_decode_attn_q4,
    ps_decode_q4_workspace_bytes,
    ps_decode_visible_ranges,
    ps_decode_workspace_bytes,
    ps_full_attn_ref,
    ps_full_attn_workspace_bytes,
    ps_kv_append_norm_rope,
    ps_kv_append_norm_rope_paged,
    ps_kv_append_norm_rope_q4,
    ps_kv_append_rope,
    ps_kv_read_q4,
    ps_masked_prefill_attn,
    ps_prefill_plan_tiles,
    ps_prefill_tile_geometry,
    ps_prefill_workspace_bytes,
    ps_qk_norm_rope,
    ps_qk_norm_rope_bwd,
    ps_qk_norm_rope_bwd_workspace_bytes,
    ps_version,
)
