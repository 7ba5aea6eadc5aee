"""The cache operators of include/gqa_attn.h on PyTorch CUDA tensors: the cache
plan, rotary positions, appending to and gathering from caches, and attention
over 4-bit caches.

All tensors of a call are on one device, which need not be the current one; the
kernels run on ``stream`` (a torch.cuda.Stream or a handle), or on that device's
current stream, and so is allocated what the call allocates: an output used on
another stream afterwards needs Tensor.record_stream, as ever.  A torch.cuda.Stream
of another device is refused; a handle is taken for one of the tensors' device.  Checks, output
allocation and the C calls are native (csrc/cache_binding.cpp): a decode step's
calls take a few microseconds each.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding

_bound = None   # the library handle whose functions _cache_ext calls
_mod = None


def _ext():
    """The native module, bound to the loaded library."""
    global _bound, _mod
    if _bound is not None and _binding._lib is _bound:
        return _mod
    handle = _binding.lib()
    if _mod is None:
        try:
            from . import _cache_ext
        except ImportError as e:
            raise RuntimeError("the _cache_ext module is missing or was built for another PyTorch: build it with "
                               "causal_gqa_attention_fwd_gb300.build.build(). There is no fallback implementation.") from e
        _mod = _cache_ext
    names = [n for n in _binding.SIGNATURES if n.startswith(("attn_cache_", "attn_rope")) or "_q4_" in n]
    _mod.bind({n: ctypes.cast(getattr(handle, n), ctypes.c_void_p).value for n in names}, _binding._check,
              getattr(torch._C, "_cuda_getCurrentRawStream", None))
    _bound = handle
    return _mod


def _run(stream, f, *args, device=None):
    """f(*args) on `stream`: made the current one, so that what the call allocates belongs to it.  device: the call's,
    where no tensor among args tells it (None: the stream's, or for a handle the current one)."""
    if stream is None:
        return f(*args)
    device = next((t.device for t in args if isinstance(t, torch.Tensor) and t.is_cuda), device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif device is not None and stream.device != device:
        raise ValueError(f"the stream is one of {stream.device}, the call's tensors are on {device}")
    with torch.cuda.stream(stream):
        return f(*args)


def attn_cache_plan(cache_lens, new_lens, block_table, page_size: int, free_pages, cursor=None, total_tokens=None,
                    slots=None, positions=None, cu_seqlens=None, lens_out=None, cursor_out=None, stream=None):
    """Block table, slots and positions of the tokens new_lens [B] adds to requests of cache_lens [B] keys.

    Each request gets the pages it lacks from free_pages, from index cursor (int32 [1], None: 0) on; they are written
    into block_table [B, max_pages] in place.  total_tokens: length of slots and positions (default: that of slots), which
    are packed in request order: request b's from entry cu_seqlens[b] on, none without new tokens; the entries past the last
    new token are -1 and 0.  All tensors int32 on the device
    -> (slots [total_tokens], positions [total_tokens], cu_seqlens [B+1], lens_out [B], cursor_out [1])."""
    return _run(stream, _ext().plan, cache_lens, new_lens, block_table, page_size, free_pages, cursor, total_tokens, slots,
                positions, cu_seqlens, lens_out, cursor_out)


def attn_rope_table(n: int, rotary_dim: int, base: float = 10000.0, factor: float = 1.0, original_positions: int = 0,
                    low_turns: float = 1.0, high_turns: float = 32.0, mscale: float = 1.0, out=None, device=None,
                    stream=None):
    """Rotary table float32 [n, rotary_dim] (cosines, then sines) of positions 0..n-1, frequencies
    base^(-2i/rotary_dim): divided by factor, or with original_positions > 0 only those that make few turns over the
    original context (all below low_turns, none above high_turns, in between blended linearly over the turns, not over the
    pair index as some released models' tables are); entries times mscale."""
    on = None                                       # out's
    if out is None:
        if device is None and isinstance(stream, torch.cuda.Stream):
            device = stream.device
        on = torch.device("cuda", device) if isinstance(device, int) else torch.device(device or "cuda")
        if on.type == "cuda" and on.index is None:
            on = torch.device("cuda", torch.cuda.current_device())

    def make(out):
        if out is None:
            out = torch.empty(n, rotary_dim, dtype=torch.float32, device=on)
        return _ext().rope_table(out, n, rotary_dim, base, factor, original_positions, low_turns, high_turns, mscale)
    return _run(stream, make, out, device=on)


def attn_rope(q, k, positions, rope_cos_sin, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """q and k (None: q alone) rotated at their positions.  [total,H,D] with positions [total], or [B,H,T,D] with
    [B,T] or [T]; bf16, views whose last dimension is contiguous are taken as they are.  rope_cos_sin float32
    [n, rotary_dim]: the first rotary_dim features are rotated, in pairs (i, i + rotary_dim/2), or (2i, 2i + 1) if
    interleaved.  An output may be its input -> (q_out, k_out)."""
    return _run(stream, _ext().rope, False, q, k, positions, rope_cos_sin, interleaved, q_out, k_out)


def attn_rope_bwd(dq_out, dk_out, positions, rope_cos_sin, interleaved: bool = False, dq=None, dk=None, stream=None):
    """Backward of attn_rope: the gradients of its inputs from those of its outputs -> (dq, dk)."""
    return _run(stream, _ext().rope, True, dq_out, dk_out, positions, rope_cos_sin, interleaved, dq, dk)


def attn_cache_append(k, v, slots, k_cache, v_cache, positions=None, rope_cos_sin=None, interleaved: bool = False,
                      stream=None):
    """Writes k, v ([total,Hkv,D] or [B,Hkv,T,D] bf16, views as attn_rope) into the slots (int32, one a token, -1:
    nowhere) of bf16 caches [pages,Hkv,page_size,D] ([B,Hkv,S,D]: slot b*S + j).  With rope_cos_sin k is rotated at
    positions (int32, one a token) on the way.  The slots of a call differ from one another."""
    _run(stream, _ext().append, k, v, slots, (k_cache, v_cache), (), positions, rope_cos_sin, interleaved)


def attn_cache_append_fp8(k, v, slots, k8, v8, k_scale: float, v_scale: float, positions=None, rope_cos_sin=None,
                          interleaved: bool = False, stream=None):
    """attn_cache_append into E4M3 caches (uint8 codes of x / scale, saturating at +-448)."""
    _run(stream, _ext().append, k, v, slots, (k8, v8), (k_scale, v_scale), positions, rope_cos_sin, interleaved)


def attn_cache_append_q4(k, v, slots, k4, k4_sf, v4, v4_sf, k_scale: float, v_scale: float, positions=None,
                         rope_cos_sin=None, interleaved: bool = False, stream=None):
    """attn_cache_append into 4-bit caches: uint8 codes [pages,Hkv,page_size,D/2] (two E2M1 a byte) and block scales
    [pages,Hkv,page_size,D/16] (E4M3); value = e2m1 * e4m3 * scale."""
    _run(stream, _ext().append, k, v, slots, (k4, k4_sf, v4, v4_sf), (k_scale, v_scale), positions, rope_cos_sin, interleaved)


def attn_cache_gather_q4(slots, k4, k4_sf, v4, v4_sf, k_scale: float, v_scale: float, k=None, v=None, stream=None):
    """Slots of 4-bit caches read back as bf16 values (slot -1: zeros) -> (k, v [tokens, Hkv, D])."""
    return _run(stream, _ext().gather, slots, k4, k4_sf, v4, v4_sf, k_scale, v_scale, k, v)


def attn_decode_q4_workspace_size(B, Hq, Hkv, Tq, S, D) -> int:
    return int(_binding.lib().attn_decode_q4_workspace_size(B, Hq, Hkv, Tq, S, D))


def attn_decode_q4_fwd(q, k4, k4_sf, v4, v4_sf, k_scale: float, v_scale: float, cache_lens, scale=None, o=None,
                       lse=None, workspace=None, stream=None, rope_cos_sin=None):
    """Cached attention over 4-bit caches: k4, v4 uint8 [B,Hkv,S,D/2], k4_sf, v4_sf uint8 [B,Hkv,S,D/16] as
    attn_cache_append_q4 writes them; everything else as attn_decode_fwd, but that a row may hold fewer keys than
    queries, or none (a query that sees no key gives o = 0, lse = -inf)."""
    return _run(stream, _ext().decode, q, k4, k4_sf, v4, v4_sf, k_scale, v_scale, None, cache_lens, scale, o, lse, workspace,
                rope_cos_sin)


def attn_decode_paged_q4_fwd(q, k4_pages, k4_sf_pages, v4_pages, v4_sf_pages, k_scale: float, v_scale: float,
                             block_table, cache_lens, scale=None, o=None, lse=None, workspace=None, stream=None,
                             rope_cos_sin=None):
    """attn_decode_q4_fwd over paged caches [num_pages,Hkv,page_size,...] through block_table [B, max_pages]."""
    if block_table is None:
        raise TypeError("block_table must be a torch.Tensor")
    return _run(stream, _ext().decode, q, k4_pages, k4_sf_pages, v4_pages, v4_sf_pages, k_scale, v_scale, block_table,
                cache_lens, scale, o, lse, workspace, rope_cos_sin)
