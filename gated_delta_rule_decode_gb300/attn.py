"""Thin Python binding of the softmax-attention entry points of libkda.so.

Attention over packed prompts (:func:`prefill`), an 8-bit paged key/value
cache (:class:`KVCache`, :func:`append`), attention over it for single tokens
and draft windows (:func:`decode`) and the eviction of its lightest pages
(:func:`evict`), as declared in ``include/kda_attn.h``.  As in :mod:`kda`,
functions check shapes, dtypes and devices, pass raw device pointers and the
current CUDA stream, and raise ``KdaError`` on a negative status; all
arithmetic runs in the library's kernels.

What a call allocates (results and scratch) comes from the memory of the stream
that it runs on, ``stream`` where that is given: use such results on another
stream as any tensor of that stream (wait for it, ``record_stream``).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .kda import KdaError, _check, _dtype_code, _empty, _need, lib  # noqa: F401

PAGE_TOKENS = 64
KDA_DEVERR_PAGE = 256
KDA_DEVERR_SCALE = 512

EXPORTED = ("kda_attn_prefill", "kda_cache_append", "kda_attn_decode", "kda_attn_decode_workspace_bytes",
            "kda_cache_evict")


class KdaAttnDims(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class KdaKvCache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64)]


class KVCache(NamedTuple):
    """The 8-bit cache: pages of 64 positions, one power-of-two scale per page and head."""
    k_pages: torch.Tensor  # [num_pages, Hkv, 64, d] float8_e4m3fn
    v_pages: torch.Tensor  # [num_pages, Hkv, d, 64] float8_e4m3fn
    k_scale: torch.Tensor  # [num_pages, Hkv] fp32
    v_scale: torch.Tensor  # [num_pages, Hkv] fp32


class Evicted(NamedTuple):
    seq_lens: torch.Tensor     # [B] int32
    block_table: torch.Tensor  # [B, max_pages] int32
    weight: torch.Tensor       # [B, max_pages] fp32
    freed: torch.Tensor        # [B, max_pages] int32, -1 past freed_count
    freed_count: torch.Tensor  # [B] int32


_VP, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_PD, _PC = ctypes.POINTER(KdaAttnDims), ctypes.POINTER(KdaKvCache)


def _declare(lib):
    lib.kda_attn_prefill.argtypes = [_PD, _I32, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP]
    lib.kda_cache_append.argtypes = [_PD, _PC, _I32, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _I32, _VP, _VP]
    lib.kda_attn_decode.argtypes = [_PD, _PC, _I32, _I32, _VP, _I64, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _SZ,
                                    _VP, _VP]
    lib.kda_attn_decode_workspace_bytes.argtypes = [_PD, _I32, _I32, _I32, _I32]
    lib.kda_cache_evict.argtypes = [_I32, _I32, _I32, _I32, _I32] + [_VP] * 10
    for name in EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    lib.kda_attn_decode_workspace_bytes.restype = _SZ
    return lib


_lib = _declare(lib())


_F32, _I32T, _F8 = torch.float32, torch.int32, torch.float8_e4m3fn
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def make_dims(q_heads: int, kv_heads: int, head_dim: int, dtype_code: int, scale: float | None = None) -> KdaAttnDims:
    return KdaAttnDims(int(q_heads), int(kv_heads), int(head_dim), int(dtype_code),
                       float(scale) if scale is not None else 0.0)


# A small call's time is the host's, so the checks below take their quick way
# first and look for what to say only when it fails.

def _gpu(t: torch.Tensor, name: str, stream) -> int:
    """The GPU of a call's first tensor, which the call's stream has to be of:
    the kernels run there, and every other tensor has to be there too."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    at = torch.cuda.current_device()
    if dev != at or (stream is not None and stream.device_index != dev):
        raise ValueError(f"{name} is on cuda:{dev}, the current GPU is cuda:{at}"
                         + (f", the stream is of cuda:{stream.device_index}" if stream is not None else ""))
    return dev


def _elsewhere(t: torch.Tensor, name: str, dev: int):
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call runs on cuda:{dev}")


def _ok(t: torch.Tensor, name: str, shape: tuple, dtype, dev: int):
    """Checks a contiguous tensor on GPU `dev`."""
    if not (t.get_device() == dev and t.shape == shape and t.dtype is dtype and t.is_contiguous()):
        _elsewhere(t, name, dev)
        _need(t, name, shape, dtype)


def _rows(t: torch.Tensor, name: str, shape: tuple, dtype, dev: int) -> int:
    """Checks a tensor of token rows that may lie apart (a slice of a fused
    projection) and returns the distance between tokens in elements."""
    H, d = shape[-2], shape[-1]
    if t.get_device() != dev:
        _elsewhere(t, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.is_contiguous():
        apart = H * d
    else:
        st = t.stride()
        apart = st[-3]
        if shape[-3] == 1:
            # the only token, or the only token of each sequence
            apart = st[0] if len(shape) == 4 and shape[0] > 1 else H * d
        ok = st[-1] == 1 and (H == 1 or st[-2] == d) and apart >= H * d
        if len(shape) == 4 and shape[0] > 1:
            ok = ok and st[0] == shape[1] * apart
        if not ok:
            raise ValueError(f"{name} must have contiguous [heads, d] rows at one distance")
    if (apart * t.element_size()) % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name}'s rows must start on 16-byte boundaries")
    return apart


def _ptr(t):
    return None if t is None else t.data_ptr()


def _flag(err_flag, dev: int):
    if err_flag is None:
        return None
    if err_flag.get_device() != dev or err_flag.dtype is not _I32T or err_flag.numel() < 1:
        raise ValueError(f"err_flag must be an int32 tensor on cuda:{dev}")
    return err_flag.data_ptr()


def _stream_handle(stream, dev: int):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream().cuda_stream


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """Memory like t's, of the call's stream (quicker than :func:`_empty`)."""
    return torch.empty_like(t) if stream is None else _empty(t.shape, t.dtype, t.device, stream)


def _check_cache(c: KVCache, dev: int):
    k, v, ks, vs = c
    N, Hkv, page, d = k.shape
    if page != PAGE_TOKENS:
        raise ValueError(f"k_pages has {page} positions per page, expected {PAGE_TOKENS}")
    _ok(k, "k_pages", (N, Hkv, PAGE_TOKENS, d), _F8, dev)
    _ok(v, "v_pages", (N, Hkv, d, PAGE_TOKENS), _F8, dev)
    _ok(ks, "k_scale", (N, Hkv), _F32, dev)
    _ok(vs, "v_scale", (N, Hkv), _F32, dev)
    return Hkv, d, KdaKvCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), N)


def alloc_cache(num_pages: int, kv_heads: int, head_dim: int, device="cuda") -> KVCache:
    """An empty cache of ``num_pages`` pages of 64 positions."""
    f8 = torch.float8_e4m3fn
    return KVCache(torch.zeros((num_pages, kv_heads, PAGE_TOKENS, head_dim), dtype=torch.uint8, device=device).view(f8),
                   torch.zeros((num_pages, kv_heads, head_dim, PAGE_TOKENS), dtype=torch.uint8, device=device).view(f8),
                   torch.ones((num_pages, kv_heads), dtype=torch.float32, device=device),
                   torch.ones((num_pages, kv_heads), dtype=torch.float32, device=device))


def prefill(q, k, v, cu_seqlens, out=None, *, lse=None, return_lse=False, scale=None, err_flag=None, stream=None):
    """Causal attention over packed prompts.

    q: [T, Hq, d]; k, v: [T, Hkv, d], Hq a multiple of Hkv (rows may lie apart,
    as slices of one projection); cu_seqlens: [n + 1] int32.  Returns out
    [T, Hq, d], with ``return_lse`` also lse [T, Hq] fp32 (natural log).
    """
    T, Hq, d = q.shape
    Hkv, dt = k.shape[1], q.dtype
    code = _dtype_code(q)
    dev = _gpu(q, "q", stream)
    flag = _flag(err_flag, dev)
    qs, ks, vs = (_rows(q, "q", (T, Hq, d), dt, dev), _rows(k, "k", (T, Hkv, d), dt, dev),
                  _rows(v, "v", (T, Hkv, d), dt, dev))
    n = cu_seqlens.shape[0] - 1
    _ok(cu_seqlens, "cu_seqlens", (n + 1,), _I32T, dev)
    if out is None:
        out = _empty((T, Hq, d), dt, q.device, stream)
    else:
        _ok(out, "out", (T, Hq, d), dt, dev)
    if lse is None:
        if return_lse:
            lse = _empty((T, Hq), _F32, q.device, stream)
    else:
        _ok(lse, "lse", (T, Hq), _F32, dev)
    dims = make_dims(Hq, Hkv, d, code, scale)
    _check(_lib.kda_attn_prefill(ctypes.byref(dims), n, _ptr(cu_seqlens), T, _ptr(q), qs, _ptr(k), ks, _ptr(v), vs,
                                 _ptr(out), _ptr(lse), flag, _stream_handle(stream, dev)), "kda_attn_prefill")
    return (out, lse) if return_lse else out


def append(cache: KVCache, k, v, cu_seqlens, start_pos, block_table, *, err_flag=None, stream=None):
    """Quantises packed new tokens into the cache, after the ``start_pos``
    positions that each sequence holds.

    k, v: [T, Hkv, d]; cu_seqlens: [n + 1] int32; start_pos: [n] int32;
    block_table: [n, max_pages] int32.
    """
    dev = _gpu(k, "k", stream)
    flag = _flag(err_flag, dev)
    Hkv, d, c = _check_cache(cache, dev)
    T, dt = k.shape[0], k.dtype
    code = _dtype_code(k)
    ks, vs = _rows(k, "k", (T, Hkv, d), dt, dev), _rows(v, "v", (T, Hkv, d), dt, dev)
    n, width = block_table.shape
    _ok(cu_seqlens, "cu_seqlens", (n + 1,), _I32T, dev)
    _ok(start_pos, "start_pos", (n,), _I32T, dev)
    _ok(block_table, "block_table", (n, width), _I32T, dev)
    dims = make_dims(Hkv, Hkv, d, code)
    _check(_lib.kda_cache_append(ctypes.byref(dims), ctypes.byref(c), n, _ptr(cu_seqlens), T, _ptr(k), ks, _ptr(v), vs,
                                 _ptr(start_pos), _ptr(block_table), width, flag, _stream_handle(stream, dev)),
           "kda_cache_append")


def decode_workspace_bytes(q_heads, kv_heads, head_dim, dtype_code, batch, draft_len, max_pages, with_weight) -> int:
    """Bytes of workspace that :func:`decode` needs."""
    dims = make_dims(q_heads, kv_heads, head_dim, dtype_code)
    return _lib.kda_attn_decode_workspace_bytes(ctypes.byref(dims), batch, draft_len, max_pages, 1 if with_weight else 0)


def decode(q, cache: KVCache, seq_lens, block_table, out=None, *, lse=None, return_lse=False, weight_in=None,
           weight_out=None, return_weight=False, workspace=None, scale=None, err_flag=None, stream=None):
    """Attention of each sequence's last D (1..16) tokens, which are in the
    cache already; token t sees the positions before seq_lens - D + 1 + t.

    q: [B, D, Hq, d]; seq_lens: [B] int32 (0: padding); block_table:
    [B, max_pages] int32.  Returns out [B, D, Hq, d], then with ``return_lse``
    lse [B, D, Hq] fp32, then with ``return_weight`` (or ``weight_out``) the
    page weights [B, max_pages] fp32: ``weight_in`` (zero without it) plus the
    attention weight that this call's rows gave to each page.
    """
    dev = _gpu(q, "q", stream)
    flag = _flag(err_flag, dev)
    Hkv, d, c = _check_cache(cache, dev)
    B, D, Hq, _ = q.shape
    dt = q.dtype
    code = _dtype_code(q)
    qs = _rows(q, "q", (B, D, Hq, d), dt, dev)
    width = block_table.shape[1]
    _ok(seq_lens, "seq_lens", (B,), _I32T, dev)
    _ok(block_table, "block_table", (B, width), _I32T, dev)
    if out is None:
        out = _empty((B, D, Hq, d), dt, q.device, stream)
    else:
        _ok(out, "out", (B, D, Hq, d), dt, dev)
    if lse is None:
        if return_lse:
            lse = _empty((B, D, Hq), _F32, q.device, stream)
    else:
        _ok(lse, "lse", (B, D, Hq), _F32, dev)
    if weight_in is not None:
        _ok(weight_in, "weight_in", (B, width), _F32, dev)
    if weight_out is not None:
        _ok(weight_out, "weight_out", (B, width), _F32, dev)
    elif return_weight or weight_in is not None:
        weight_out = _empty((B, width), _F32, q.device, stream)
    dims = make_dims(Hq, Hkv, d, code, scale)
    pd = ctypes.byref(dims)
    if workspace is None:
        need = _lib.kda_attn_decode_workspace_bytes(pd, B, D, width, 0 if weight_out is None else 1)
        workspace = _empty((need,), torch.uint8, q.device, stream)
    else:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
        need = workspace.numel() * workspace.element_size()
    _check(_lib.kda_attn_decode(pd, ctypes.byref(c), B, D, _ptr(q), qs, _ptr(seq_lens), _ptr(block_table), width,
                                _ptr(out), _ptr(lse), _ptr(weight_in), _ptr(weight_out), _ptr(workspace), need,
                                flag, _stream_handle(stream, dev)), "kda_attn_decode")
    got = (out,) + ((lse,) if return_lse else ()) + ((weight_out,) if weight_out is not None else ())
    return got if len(got) > 1 else out


def evict(seq_lens, block_table, weight, budget: int, sink: int = 1, recent: int = 1, *, in_place=False,
          err_flag=None, stream=None) -> Evicted:
    """Drops the lightest pages of sequences that hold more than ``budget``;
    the first ``sink`` and last ``recent`` pages stay.

    seq_lens: [B] int32; block_table: [B, max_pages] int32; weight:
    [B, max_pages] fp32.  With ``in_place`` these three are updated.
    """
    dev = _gpu(seq_lens, "seq_lens", stream)
    flag = _flag(err_flag, dev)
    B, width = block_table.shape
    _ok(seq_lens, "seq_lens", (B,), _I32T, dev)
    _ok(block_table, "block_table", (B, width), _I32T, dev)
    _ok(weight, "weight", (B, width), _F32, dev)
    if in_place:
        lens, table, w = seq_lens, block_table, weight
    else:
        lens, table, w = _like(seq_lens, stream), _like(block_table, stream), _like(weight, stream)
    freed, count = _like(block_table, stream), _like(seq_lens, stream)
    _check(_lib.kda_cache_evict(B, width, int(budget), int(sink), int(recent), _ptr(seq_lens), _ptr(block_table),
                                _ptr(weight), _ptr(lens), _ptr(table), _ptr(w), _ptr(freed), _ptr(count),
                                flag, _stream_handle(stream, dev)), "kda_cache_evict")
    return Evicted(lens, table, w, freed, count)
