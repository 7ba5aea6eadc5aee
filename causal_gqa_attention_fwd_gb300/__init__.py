"""Causal grouped-query attention (forward and backward) for GB300 (sm_103a).

The public entry points mirror the C ABI of include/gqa_attn.h and take
PyTorch CUDA tensors (PyTorch supplies device memory and the stream):

    attn_fwd(q, k, v, causal=True, scale=None) -> (o, lse)
    attn_fwd_rope(q, k, v, rope_cos_sin, causal=True, scale=None) -> (o, lse), q and k rotated
    attn_varlen_fwd_rope(q, k, v, cu_seqlens, max_seqlen, rope_cos_sin, ...) -> (o, lse)
    attn_bwd(q, k, v, o, lse, dout, causal=True, scale=None) -> (dq, dk, dv)
    attn_bwd_rope(q, k, v, o, lse, dout, rope_cos_sin, ...) -> (dq, dk, dv), the backward of attn_fwd_rope
    attn_varlen_bwd_rope(q, k, v, o, lse, dout, cu_seqlens, max_seqlen, rope_cos_sin, ...) -> (dq, dk, dv)
    attn_varlen_fwd(q, k, v, cu_seqlens, max_seqlen, ...) -> (o, lse)
    attn_varlen_bwd(q, k, v, o, lse, dout, cu_seqlens, max_seqlen, ...) -> (dq, dk, dv)
    attn_decode_fwd(q, k_cache, v_cache, cache_lens, scale=None) -> (o, lse)
    attn_decode_paged_fwd(q, k_pages, v_pages, block_table, cache_lens, scale=None) -> (o, lse)
    attn_decode_fp8_fwd / attn_decode_paged_fp8_fwd: the same over E4M3 caches with per-tensor scales
    attn_decode_q4_fwd / attn_decode_paged_q4_fwd: the same over 4-bit caches (E2M1, a scale per 16 features)
    attn_cache_plan(cache_lens, new_lens, block_table, page_size, free_pages, cursor, total_tokens)
        -> (slots, positions, cu_seqlens, lens_out, cursor_out), block_table extended in place
    attn_rope(q, k, positions, rope_cos_sin, interleaved=False) -> (q_out, k_out)
    attn_rope_bwd(dq_out, dk_out, positions, rope_cos_sin, interleaved=False) -> (dq, dk)
    attn_rope_table(n, rotary_dim, base=10000.0, factor=1.0, ...) -> rope_cos_sin, scaled for long contexts
    attn_cache_append / attn_cache_append_fp8 / attn_cache_append_q4: k and v (k rotated, if asked) into cache slots
    attn_cache_gather_q4(slots, k4, k4_sf, v4, v4_sf, k_scale, v_scale) -> (k, v) bf16
    attn_decode_prefix_fwd(q, k_prefix, v_prefix, prefix_lens, k_cache, v_cache, cache_lens, scale=None) -> (o, lse):
        cached attention of rows that share prefixes; attn_decode_paged_prefix_fwd: over one pool of pages
    attn_cache_weights / attn_cache_weights_fp8 / attn_cache_weights_q4: the attention weight cached keys receive, added up
    attn_cache_evict(weights, caches, cache_lens, budget, recent=0, first=0, ...) -> (kept, lens_out), caches cut in place

All arithmetic runs in the library's hand-written sm_103a kernels; a call
raises if the library is not built.
"""
from ._binding import (  # noqa: F401
    LIB_PATH,
    AttnError,
    attn_bwd,
    attn_bwd_noalloc,
    attn_bwd_rope,
    attn_bwd_rope_workspace_size,
    attn_bwd_workspace_size,
    attn_decode_fp8_fwd,
    attn_decode_fwd,
    attn_decode_paged_fp8_fwd,
    attn_decode_paged_fwd,
    attn_decode_workspace_size,
    attn_fwd,
    attn_fwd_rope,
    attn_fwd_rope_workspace_size,
    attn_varlen_fwd_rope,
    attn_varlen_fwd_rope_workspace_size,
    attn_varlen_bwd,
    attn_varlen_bwd_rope,
    attn_varlen_bwd_rope_workspace_size,
    attn_varlen_bwd_workspace_size,
    attn_varlen_fwd,
    get_check_line,
    get_device_status,
    lib,
    profile_enable,
    profile_read,
    profile_reset,
    status_string,
)
from ._cache import (  # noqa: F401
    attn_cache_append,
    attn_cache_append_fp8,
    attn_cache_append_q4,
    attn_cache_evict,
    attn_cache_gather_q4,
    attn_cache_plan,
    attn_cache_weights,
    attn_cache_weights_fp8,
    attn_cache_weights_q4,
    attn_decode_paged_prefix_fwd,
    attn_decode_paged_q4_fwd,
    attn_decode_prefix_fwd,
    attn_decode_prefix_workspace_size,
    attn_decode_q4_fwd,
    attn_decode_q4_workspace_size,
    attn_rope,
    attn_rope_bwd,
    attn_rope_table,
)
