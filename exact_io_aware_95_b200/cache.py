"""8-bit key/value cache: e4m3 codes [B, Nk, Hkv, d] with one power-of-two scale
per (token, key head), kept as an exponent byte [B, Hkv, Nk] (uint8; a byte e
stands for 2^(e - 127)).

``cache_append`` quantises new keys and values into it, ``cache_read`` reads it
back as bf16 (exactly), ``cache_decode_fwd`` is the decode-shaped attention over
it.  Argument marshalling only: see include/fa.h for the definitions and limits.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _check, _need, _need_shape, _need_workspace, _on, _same_device, _scale, _stream_ptr, lib
from .modified import _slopes, _softcap, _window

__all__ = ["cache_append", "cache_read", "cache_decode_fwd", "cache_decode_workspace_size"]


def _need_cache(codes, exps, name: str, scale_name: str, shape=None):
    _need(codes, name, torch.float8_e4m3fn, 4)
    if shape is not None and codes.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(codes.shape)}")
    B, Nk, Hkv, _ = codes.shape
    _need_shape(exps, scale_name, torch.uint8, (B, Hkv, Nk))


def cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 k_scale: torch.Tensor, v_scale: torch.Tensor, start: torch.Tensor,
                 count: Optional[torch.Tensor] = None) -> None:
    """Quantise rows k, v (bf16 [B, T, Hkv, d]) into rows start[b] ..
    start[b] + count[b] - 1 of the caches, in place (start, count: int32 [B];
    count None: all T)."""
    _need(k, "k", torch.bfloat16, 4)
    _need_shape(v, "v", torch.bfloat16, k.shape)
    B, T, Hkv, d = k.shape
    _need(k_cache, "k_cache", torch.float8_e4m3fn, 4)
    Nk = k_cache.shape[1]
    _need_cache(k_cache, k_scale, "k_cache", "k_scale", (B, Nk, Hkv, d))
    _need_cache(v_cache, v_scale, "v_cache", "v_scale", (B, Nk, Hkv, d))
    _need_shape(start, "start", torch.int32, (B,))
    if count is not None:
        _need_shape(count, "count", torch.int32, (B,))
    _same_device(k, v, k_cache, v_cache, k_scale, v_scale, start, count)
    with _on(k):
        st = lib().fa_cache_append(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                   k_scale.data_ptr(), v_scale.data_ptr(), start.data_ptr(),
                                   None if count is None else count.data_ptr(), B, T, Nk, Hkv, d, _stream_ptr(k))
    _check(st, "fa_cache_append")


def cache_read(cache: torch.Tensor, scale: torch.Tensor, seqlens: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The cached values as bf16 [B, Nk, Hkv, d], exactly; zero in the rows from
    seqlens[b] (int32 [B]; None: all Nk rows are read) on."""
    _need_cache(cache, scale, "cache", "scale")
    B, Nk, Hkv, d = cache.shape
    if seqlens is not None:
        _need_shape(seqlens, "seqlens", torch.int32, (B,))
    o = cache.new_empty(cache.shape, dtype=torch.bfloat16) if out is None else out
    _need_shape(o, "out", torch.bfloat16, cache.shape)
    _same_device(cache, scale, o, seqlens)
    with _on(cache):
        st = lib().fa_cache_read(cache.data_ptr(), scale.data_ptr(), None if seqlens is None else seqlens.data_ptr(),
                                 o.data_ptr(), B, Nk, Hkv, d, _stream_ptr(cache))
    _check(st, "fa_cache_read")
    return o


def cache_decode_workspace_size(B: int, Nq: int, Nk: int, H: int, Hkv: int, d: int) -> int:
    return int(lib().fa_cache_decode_workspace_size(B, Nq, Nk, H, Hkv, d))


def cache_decode_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                     v_scale: torch.Tensor, seqlens_k: Optional[torch.Tensor] = None, causal: bool = False,
                     scale: Optional[float] = None, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                     window: int = 0, out=None, lse=None, workspace=None):
    """Decode-shaped forward from an 8-bit cache: q [B, Nq, H, d] (Nq <= 16)
    against the first seqlens_k[b] cached rows (int32 [B]; None: all).  Returns
    O bf16 [B, Nq, H, d] and LSE fp32 [B, H, Nq]."""
    _need(q, "q", torch.bfloat16, 4)
    B, Nq, H, d = q.shape
    _need_cache(k_cache, k_scale, "k_cache", "k_scale")
    Nk, Hkv = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Nk, Hkv, d) or Hkv < 1 or H % Hkv != 0:
        raise ValueError(f"k_cache must be [{B}, Nk, Hkv, {d}] with Hkv dividing {H}, got {tuple(k_cache.shape)}")
    _need_cache(v_cache, v_scale, "v_cache", "v_scale", k_cache.shape)
    if seqlens_k is not None:
        _need_shape(seqlens_k, "seqlens_k", torch.int32, (B,))
    softcap, window = _softcap(softcap), _window(window)
    _slopes(slopes, H)
    L = lib()
    need = L.fa_cache_decode_workspace_size(B, Nq, Nk, H, Hkv, d)
    if out is not None:
        _need_shape(out, "out", torch.bfloat16, q.shape)
    if lse is not None:
        _need_shape(lse, "lse", torch.float32, (B, H, Nq))
    if workspace is not None:
        _need_workspace(workspace, need)
    _same_device(q, k_cache, v_cache, k_scale, v_scale, seqlens_k, slopes, out, lse, workspace)
    o = torch.empty_like(q) if out is None else out
    l = q.new_empty((B, H, Nq), dtype=torch.float32) if lse is None else lse
    ws = q.new_empty(max(need, 256), dtype=torch.uint8) if workspace is None else workspace
    with _on(q):
        st = L.fa_cache_decode_fwd(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                       v_scale.data_ptr(), o.data_ptr(), l.data_ptr(),
                                       None if seqlens_k is None else seqlens_k.data_ptr(),
                                       None if slopes is None else slopes.data_ptr(), ws.data_ptr(),
                                       ws.nbytes, B, Nq, Nk, H, Hkv, d, _scale(scale, d), softcap,
                                       window, int(bool(causal)), _stream_ptr(q))
    _check(st, "fa_cache_decode_fwd")
    return o, l
