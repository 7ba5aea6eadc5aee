"""The cache operators of include/gqa_attn.h on PyTorch CUDA tensors: the cache
plan, rotary positions, appending to and gathering from caches, and attention
over 4-bit caches.

Argument marshalling only, as in ``_binding``.  All tensors of a call are on
one device, which need not be the current one; the kernels run on ``stream``,
or on that device's current stream.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import _check, _scale, lib

_Strides6 = ctypes.c_longlong * 6
_Strides12 = ctypes.c_longlong * 12


def _at(t, name, dtype, dev, contiguous=True):
    """Address of a tensor of the call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call's first tensor on cuda:{dev}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _call(name, dev, stream, *args):
    """The C call on `stream` (None: the device's current one), with the tensors' device current."""
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    fn = getattr(lib(), name)
    if dev == torch.cuda.current_device():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st:
        _check(st, name)


def _scratch(n, dev, stream):
    """A workspace that the stream which uses it owns, so that its memory is not handed to another one meanwhile."""
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device=dev)


def _tokens(x, name):
    """(B, T, H, D) of a [total,H,D] or [B,H,T,D] tensor."""
    if x.dim() == 3:
        return 1, x.shape[0], x.shape[1], x.shape[2]
    if x.dim() == 4:
        return x.shape[0], x.shape[2], x.shape[1], x.shape[3]
    raise ValueError(f"{name} must be [total, H, D] or [B, H, T, D]")


def _strides(x, name, out=False):
    """(batch, token, head) strides in elements; those of single entries are 0."""
    s, n = x.stride(), x.shape
    if n[-1] > 1 and s[-1] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if out and any(s[i] == 0 and n[i] > 1 for i in range(len(n))):
        raise ValueError(f"{name} must not repeat its memory")
    if len(n) == 3:
        return 0, s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0
    return s[0] if n[0] > 1 else 0, s[2] if n[2] > 1 else 0, s[1] if n[1] > 1 else 0


def _table(t, dev):
    """(address, positions, rotary_dim) of a rotary table."""
    if t is None:
        return None, 0, 0
    if t.dim() != 2:
        raise ValueError("rope_cos_sin must be [positions, rotary_dim]")
    return _at(t, "rope_cos_sin", torch.float32, dev), t.shape[0], t.shape[1]


def attn_cache_plan(cache_lens, new_lens, block_table, page_size: int, free_pages, cursor=None, total_tokens=None,
                    slots=None, positions=None, cu_seqlens=None, lens_out=None, cursor_out=None, stream=None):
    """Block table, slots and positions of the tokens new_lens [B] adds to requests of cache_lens [B] keys.

    Each request gets the pages it lacks from free_pages, from index cursor (int32 [1], None: 0) on; they are written
    into block_table [B, max_pages] in place.  total_tokens: length of slots and positions (default: that of slots); the
    entries past the last new token are -1 and 0.  All tensors int32 on the device
    -> (slots [total_tokens], positions [total_tokens], cu_seqlens [B+1], lens_out [B], cursor_out [1])."""
    dev = _device(cache_lens, "cache_lens")
    B = cache_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B or new_lens.numel() != B:
        raise ValueError("cache_lens and new_lens must be [B], block_table [B, max_pages]")
    if total_tokens is None:
        if slots is None:
            raise ValueError("total_tokens (or slots) is needed: the lengths are not read on the host")
        total_tokens = slots.numel()
    n = int(total_tokens)
    made = []
    want = ((slots, n), (positions, n), (cu_seqlens, B + 1), (lens_out, B), (cursor_out, 1))
    if any(t is None for t, _ in want):
        made = torch.empty(2 * n + 2 * B + 2, dtype=torch.int32, device=cache_lens.device).split([m for _, m in want])
    out, ptrs = [], []
    for i, (name, (t, m)) in enumerate(zip(("slots", "positions", "cu_seqlens", "lens_out", "cursor_out"), want)):
        t = made[i] if t is None else t
        p = _at(t, name, torch.int32, dev)
        if t.numel() != m:
            raise ValueError(f"{name} must have {m} entries, got {t.numel()}")
        out.append(t)
        ptrs.append(p if m else None)
    if cursor is not None and cursor.numel() != 1:
        raise ValueError("cursor must have one entry")
    i32 = torch.int32
    _call("attn_cache_plan", dev, stream, _at(cache_lens, "cache_lens", i32, dev), _at(new_lens, "new_lens", i32, dev),
          _at(block_table, "block_table", i32, dev), _at(free_pages, "free_pages", i32, dev),
          None if cursor is None else _at(cursor, "cursor", i32, dev), *ptrs, B, page_size, block_table.shape[1],
          free_pages.numel(), n)
    return tuple(out)


def attn_rope_table(n: int, rotary_dim: int, base: float = 10000.0, factor: float = 1.0, original_positions: int = 0,
                    low_turns: float = 1.0, high_turns: float = 32.0, mscale: float = 1.0, out=None, device=None,
                    stream=None):
    """Rotary table float32 [n, rotary_dim] (cosines, then sines) of positions 0..n-1, frequencies
    base^(-2i/rotary_dim): divided by factor, or with original_positions > 0 only those that make few turns over the
    original context (all below low_turns, none above high_turns, in between blended); entries times mscale."""
    if out is None:
        out = torch.empty(n, rotary_dim, dtype=torch.float32, device=device or "cuda")
    elif tuple(out.shape) != (n, rotary_dim):
        raise ValueError(f"out must be [{n}, {rotary_dim}]")
    dev = _device(out, "out")
    _call("attn_rope_table", dev, stream, _at(out, "out", torch.float32, dev), n, rotary_dim, base, factor,
          original_positions, low_turns, high_turns, mscale)
    return out


def _rope_call(name, q, k, positions, rope_cos_sin, interleaved, q_out, k_out, stream):
    dev = _device(q, "q")
    B, T, Hq, D = _tokens(q, "q")
    Hkv = 0
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
    kp = kop = None
    ks = kos = (0, 0, 0)
    if k is not None:
        if k.dim() != q.dim() or _tokens(k, "k")[:2] != (B, T) or k.shape[-1] != D:
            raise ValueError("k must have q's tokens and head dimension")
        Hkv = _tokens(k, "k")[2]
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device) if k_out is None else k_out
        kp, kop = (_at(t, n, torch.bfloat16, dev, False) for t, n in ((k, "k"), (k_out, "k_out")))
        ks, kos = _strides(k, "k"), _strides(k_out, "k_out", True)
        if k_out.shape != k.shape:
            raise ValueError("k_out must have k's shape")
    elif k_out is not None:
        raise ValueError("k_out without k")
    if q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    if positions.numel() == B * T and (positions.dim() == 1 or tuple(positions.shape) == (B, T)):
        stride = T
    elif tuple(positions.shape) == (T,):
        stride = 0
    else:
        raise ValueError("positions must hold one entry a token ([total], [B, T], or [T] for every batch row)")
    tab, n, R = _table(rope_cos_sin, dev)
    if tab is None:
        raise TypeError("rope_cos_sin must be a torch.Tensor")
    st = _Strides12(*_strides(q, "q"), *ks, *_strides(q_out, "q_out", True), *kos)
    _call(name, dev, stream, _at(q, "q", torch.bfloat16, dev, False), kp,
          _at(q_out, "q_out", torch.bfloat16, dev, False), kop, _at(positions, "positions", torch.int32, dev), stride,
          tab, n, B, T, Hq, Hkv, D, R, int(interleaved), st)
    return q_out, k_out


def attn_rope(q, k, positions, rope_cos_sin, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """q and k (None: q alone) rotated at their positions.  [total,H,D] with positions [total], or [B,H,T,D] with
    [B,T] or [T]; bf16, views whose last dimension is contiguous are taken as they are.  rope_cos_sin float32
    [n, rotary_dim]: the first rotary_dim features are rotated, in pairs (i, i + rotary_dim/2), or (2i, 2i + 1) if
    interleaved.  An output may be its input -> (q_out, k_out)."""
    return _rope_call("attn_rope", q, k, positions, rope_cos_sin, interleaved, q_out, k_out, stream)


def attn_rope_bwd(dq_out, dk_out, positions, rope_cos_sin, interleaved: bool = False, dq=None, dk=None, stream=None):
    """Backward of attn_rope: the gradients of its inputs from those of its outputs -> (dq, dk)."""
    return _rope_call("attn_rope_bwd", dq_out, dk_out, positions, rope_cos_sin, interleaved, dq, dk, stream)


def _append(name, k, v, slots, caches, scales, dtype, per_byte, positions, rope_cos_sin, interleaved, stream):
    dev = _device(k, "k")
    B, T, H, D = _tokens(k, "k")
    if v.shape != k.shape:
        raise ValueError("v must have k's shape")
    c = caches[0][1]
    if c.dim() != 4:
        raise ValueError(f"{caches[0][0]} must be [pages, Hkv, page_size, ...]")
    pages, page_size = c.shape[0], c.shape[2]
    ptrs = []
    for (cname, t), div in zip(caches, per_byte):
        if tuple(t.shape) != (pages, H, page_size, D // div):
            raise ValueError(f"{cname} must be [pages, Hkv, page_size, {D // div}] with k's heads")
        ptrs.append(_at(t, cname, dtype, dev))
    if slots.numel() != B * T:
        raise ValueError("slots must hold one entry a token")
    tab, n, R = _table(rope_cos_sin, dev)
    pos = None
    if tab is not None:
        if positions is None or positions.numel() != B * T:
            raise ValueError("positions must hold one entry a token")
        pos = _at(positions, "positions", torch.int32, dev)
    elif positions is not None:
        raise ValueError("positions without rope_cos_sin")
    st = _Strides6(*_strides(k, "k"), *_strides(v, "v"))
    _call(name, dev, stream, _at(k, "k", torch.bfloat16, dev, False), _at(v, "v", torch.bfloat16, dev, False),
          _at(slots, "slots", torch.int32, dev), pos, tab, n, R, int(interleaved), *ptrs, *scales, B, T, H, D,
          page_size, pages, st)


def attn_cache_append(k, v, slots, k_cache, v_cache, positions=None, rope_cos_sin=None, interleaved: bool = False,
                      stream=None):
    """Writes k, v ([total,Hkv,D] or [B,Hkv,T,D] bf16, views as attn_rope) into the slots (int32, one a token, -1:
    nowhere) of bf16 caches [pages,Hkv,page_size,D] ([B,Hkv,S,D]: slot b*S + j).  With rope_cos_sin k is rotated at
    positions (int32, one a token) on the way.  The slots of a call differ from one another."""
    _append("attn_cache_append", k, v, slots, (("k_cache", k_cache), ("v_cache", v_cache)), (), torch.bfloat16, (1, 1),
            positions, rope_cos_sin, interleaved, stream)


def attn_cache_append_fp8(k, v, slots, k8, v8, k_scale: float, v_scale: float, positions=None, rope_cos_sin=None,
                          interleaved: bool = False, stream=None):
    """attn_cache_append into E4M3 caches (uint8 codes of x / scale, saturating at +-448)."""
    _append("attn_cache_append_fp8", k, v, slots, (("k8", k8), ("v8", v8)), (float(k_scale), float(v_scale)),
            torch.uint8, (1, 1), positions, rope_cos_sin, interleaved, stream)


def attn_cache_append_q4(k, v, slots, k4, k4_sf, v4, v4_sf, k_scale: float, v_scale: float, positions=None,
                         rope_cos_sin=None, interleaved: bool = False, stream=None):
    """attn_cache_append into 4-bit caches: uint8 codes [pages,Hkv,page_size,D/2] (two E2M1 a byte) and block scales
    [pages,Hkv,page_size,D/16] (E4M3); value = e2m1 * e4m3 * scale."""
    _append("attn_cache_append_q4", k, v, slots, (("k4", k4), ("k4_sf", k4_sf), ("v4", v4), ("v4_sf", v4_sf)),
            (float(k_scale), float(v_scale)), torch.uint8, (2, 16, 2, 16), positions, rope_cos_sin, interleaved, stream)


def _q4_cache(k4, k4_sf, v4, v4_sf, dev, names):
    """Addresses of a 4-bit cache's tensors, checked against k4's shape."""
    if k4.dim() != 4:
        raise ValueError(f"{names[0]} must be [pages, Hkv, page_size, D/2]")
    n, h, p, w = k4.shape
    if v4.shape != k4.shape or tuple(k4_sf.shape) != (n, h, p, w // 8) or v4_sf.shape != k4_sf.shape:
        raise ValueError(f"{names[0]} and {names[2]} must be [pages, Hkv, page_size, D/2], {names[1]} and {names[3]} "
                         "[pages, Hkv, page_size, D/16]")
    return [_at(t, m, torch.uint8, dev) for t, m in zip((k4, k4_sf, v4, v4_sf), names)]


def attn_cache_gather_q4(slots, k4, k4_sf, v4, v4_sf, k_scale: float, v_scale: float, k=None, v=None, stream=None):
    """Slots of 4-bit caches read back as bf16 values (slot -1: zeros) -> (k, v [tokens, Hkv, D])."""
    dev = _device(slots, "slots")
    ptrs = _q4_cache(k4, k4_sf, v4, v4_sf, dev, ("k4", "k4_sf", "v4", "v4_sf"))
    n, (pages, H, page_size, w) = slots.numel(), k4.shape
    k, v = (torch.empty(n, H, 2 * w, dtype=torch.bfloat16, device=k4.device) if t is None else t for t in (k, v))
    if tuple(k.shape) != (n, H, 2 * w) or v.shape != k.shape:
        raise ValueError("k, v must be [tokens, Hkv, D]")
    _call("attn_cache_gather_q4", dev, stream, _at(slots, "slots", torch.int32, dev), *ptrs, float(k_scale),
          float(v_scale), _at(k, "k", torch.bfloat16, dev), _at(v, "v", torch.bfloat16, dev), n, H, 2 * w, page_size,
          pages)
    return k, v


def attn_decode_q4_workspace_size(B, Hq, Hkv, Tq, S, D) -> int:
    return int(lib().attn_decode_q4_workspace_size(B, Hq, Hkv, Tq, S, D))


def _decode_q4(name, q, ptrs, k_scale, v_scale, block_table, cache_lens, scale, o, lse, workspace, stream,
               rope_cos_sin, Hkv, S, sizes, dev):
    B, Hq, Tq, D = q.shape
    if cache_lens.shape != (B,):
        raise ValueError("cache_lens must be [B]")
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device) if lse is None else lse
    if o.shape != q.shape or lse.shape != q.shape[:3]:
        raise ValueError("o must be [B, Hq, Tq, D], lse [B, Hq, Tq]")
    if workspace is None:
        need = attn_decode_q4_workspace_size(B, Hq, Hkv, Tq, S, D)
        workspace = _scratch(need, dev, stream) if need else None
    ws, ws_len = (None, 0) if workspace is None else (_at(workspace, "workspace", torch.uint8, dev), workspace.numel())
    tab, n, R = _table(rope_cos_sin, dev)
    if tab is not None and R != D:
        raise ValueError("rope_cos_sin must be [positions, D]")
    bf = torch.bfloat16
    _call(name, dev, stream, _at(q, "q", bf, dev), *ptrs, float(k_scale), float(v_scale),
          *(() if block_table is None else (_at(block_table, "block_table", torch.int32, dev),)),
          _at(cache_lens, "cache_lens", torch.int32, dev), _at(o, "o", bf, dev), _at(lse, "lse", torch.float32, dev), ws,
          ws_len, B, Hq, Hkv, Tq, *sizes, D, _scale(scale, D), tab, n)
    return o, lse


def attn_decode_q4_fwd(q, k4, k4_sf, v4, v4_sf, k_scale: float, v_scale: float, cache_lens, scale=None, o=None,
                       lse=None, workspace=None, stream=None, rope_cos_sin=None):
    """Cached attention over 4-bit caches: k4, v4 uint8 [B,Hkv,S,D/2], k4_sf, v4_sf uint8 [B,Hkv,S,D/16] as
    attn_cache_append_q4 writes them; everything else as attn_decode_fwd, but that a row may hold fewer keys than
    queries, or none (a query that sees no key gives o = 0, lse = -inf)."""
    dev = _device(q, "q")
    ptrs = _q4_cache(k4, k4_sf, v4, v4_sf, dev, ("k4", "k4_sf", "v4", "v4_sf"))
    B, D = q.shape[0], q.shape[-1]
    if k4.shape[0] != B or 2 * k4.shape[3] != D:
        raise ValueError("k4, v4 must be [B, Hkv, S, D/2] matching q")
    Hkv, S = k4.shape[1], k4.shape[2]
    return _decode_q4("attn_decode_q4_fwd", q, ptrs, k_scale, v_scale, None, cache_lens, scale, o, lse, workspace,
                      stream, rope_cos_sin, Hkv, S, (S,), dev)


def attn_decode_paged_q4_fwd(q, k4_pages, k4_sf_pages, v4_pages, v4_sf_pages, k_scale: float, v_scale: float,
                             block_table, cache_lens, scale=None, o=None, lse=None, workspace=None, stream=None,
                             rope_cos_sin=None):
    """attn_decode_q4_fwd over paged caches [num_pages,Hkv,page_size,...] through block_table [B, max_pages]."""
    dev = _device(q, "q")
    ptrs = _q4_cache(k4_pages, k4_sf_pages, v4_pages, v4_sf_pages, dev,
                     ("k4_pages", "k4_sf_pages", "v4_pages", "v4_sf_pages"))
    B, D = q.shape[0], q.shape[-1]
    num_pages, Hkv, page_size, w = k4_pages.shape
    if 2 * w != D or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("k4_pages must match q's head dimension, block_table be [B, max_pages]")
    max_pages = block_table.shape[1]
    return _decode_q4("attn_decode_paged_q4_fwd", q, ptrs, k_scale, v_scale, block_table, cache_lens, scale, o, lse,
                      workspace, stream, rope_cos_sin, Hkv, page_size * max_pages, (page_size, num_pages, max_pages),
                      dev)
