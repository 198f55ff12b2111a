"""Thin Python binding of the softmax-attention entry points of libkda.so.

Attention over packed prompts (:func:`prefill`), an 8-bit paged key/value
cache (:class:`KVCache`, :func:`append`), attention over it for single tokens
and draft windows (:func:`decode`) and the eviction of its lightest pages
(:func:`evict`); in front of them the norm and rotation of queries and keys
(:class:`Rotary`, :func:`norm_rotate`); for long contexts attention of batches
that share prefixes (:func:`decode_shared`), and attention over the pages that
a cheap score selects (:class:`KeySummary`, :func:`summarise`, :func:`select`,
:func:`decode_selected`), as declared in ``include/kda_attn.h``.  As in :mod:`kda`,
functions check shapes, dtypes and devices, pass raw device pointers and the
current CUDA stream, and raise ``KdaError`` on a negative status; all
arithmetic runs in the library's kernels.

What a call allocates (results and scratch) comes from the memory of the stream
that it runs on, ``stream`` where that is given: use such results on another
stream as any tensor of that stream (wait for it, ``record_stream``).
"""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction
from typing import NamedTuple

import torch

from .kda import KdaError, _check, _dtype_code, _empty, _need, lib  # noqa: F401

PAGE_TOKENS = 64
KDA_DEVERR_PAGE = 256
KDA_DEVERR_SCALE = 512

EXPORTED = ("kda_attn_prefill", "kda_cache_append", "kda_attn_decode", "kda_attn_decode_workspace_bytes",
            "kda_cache_evict", "kda_norm_rotate", "kda_attn_decode_shared", "kda_attn_decode_shared_workspace_bytes",
            "kda_cache_summarise", "kda_cache_select", "kda_cache_select_workspace_bytes", "kda_attn_decode_selected")


class KdaAttnDims(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class KdaKvCache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64)]


class KdaKeySummary(ctypes.Structure):
    _fields_ = [("bounds", ctypes.c_void_p), ("unit", ctypes.c_void_p)]


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


class Rotary(NamedTuple):
    """The rotation of :func:`norm_rotate` (see :func:`rotary`)."""
    turns: torch.Tensor  # [rotary_dim / 2] int64: turns per position in units of 2^-64, modulo one
    interleaved: bool = False  # pairs (2 i, 2 i + 1), else (i, i + rotary_dim / 2)
    factor: float = 1.0  # of the rotated channels


class KeySummary(NamedTuple):
    """Per page, kv head and channel the largest and smallest key, in whole numbers of one unit."""
    bounds: torch.Tensor  # [num_pages, Hkv, 2, d] int8
    unit: torch.Tensor    # [num_pages, Hkv] fp32, a power of two


class Selected(NamedTuple):
    """The pages that :func:`select` chose for each kv head."""
    seq_lens: torch.Tensor     # [B] int32: positions of the selected pages
    block_table: torch.Tensor  # [B, Hkv, budget] int32, -1 behind the last
    index: torch.Tensor        # [B, Hkv, budget] int32: places in the sequence's row, -1 behind the last


_VP, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_F = ctypes.c_float
_PD, _PC, _PS = ctypes.POINTER(KdaAttnDims), ctypes.POINTER(KdaKvCache), ctypes.POINTER(KdaKeySummary)


def _declare(lib):
    lib.kda_attn_prefill.argtypes = [_PD, _I32, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP]
    lib.kda_cache_append.argtypes = [_PD, _PC, _I32, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _I32, _VP, _VP]
    lib.kda_attn_decode.argtypes = [_PD, _PC, _I32, _I32, _VP, _I64, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _SZ,
                                    _VP, _VP]
    lib.kda_attn_decode_workspace_bytes.argtypes = [_PD, _I32, _I32, _I32, _I32]
    lib.kda_cache_evict.argtypes = [_I32, _I32, _I32, _I32, _I32] + [_VP] * 10
    lib.kda_norm_rotate.argtypes = [_PD, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _I32, _I32, _F, _VP, _VP, _F, _VP, _I64, _VP,
                                    _I64, _VP]
    lib.kda_attn_decode_shared.argtypes = [_PD, _PC, _I32, _I32, _VP, _I64, _VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _VP,
                                           _SZ, _VP, _VP]
    lib.kda_attn_decode_shared_workspace_bytes.argtypes = [_PD, _I32, _I32, _I32, _I32]
    lib.kda_cache_summarise.argtypes = [_PD, _PC, _PS, _I32, _VP, _I64, _VP, _VP, _I32, _VP, _VP]
    lib.kda_cache_select.argtypes = [_PD, _PS, _I64, _I32, _I32, _VP, _I64, _VP, _VP, _I32, _I32, _I32, _I32, _VP, _VP, _VP,
                                     _VP, _SZ, _VP, _VP]
    lib.kda_cache_select_workspace_bytes.argtypes = [_PD, _I32, _I32]
    lib.kda_attn_decode_selected.argtypes = [_PD, _PC, _I32, _I32, _VP, _I64, _VP, _VP, _I32, _VP, _VP, _VP, _SZ, _VP, _VP]
    for name in EXPORTED:
        getattr(lib, name).restype = _SZ if name.endswith("_bytes") else ctypes.c_int
    return lib


_lib = _declare(lib())


_F32, _I32T, _F8, _I8, _I64T = torch.float32, torch.int32, torch.float8_e4m3fn, torch.int8, torch.int64
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


def _check_summary(s: KeySummary, pages: int, Hkv: int, d: int, dev: int):
    _ok(s.bounds, "bounds", (pages, Hkv, 2, d), _I8, dev)
    _ok(s.unit, "unit", (pages, Hkv), _F32, dev)
    return KdaKeySummary(s.bounds.data_ptr(), s.unit.data_ptr())


def _workspace(workspace, size, like: torch.Tensor, dev: int, stream):
    """(the caller's workspace, or one of the call's stream of size() bytes; its bytes)"""
    if workspace is None:
        need = size()
        return _empty((need,), torch.uint8, like.device, stream), need
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return workspace, workspace.numel() * workspace.element_size()


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


# 2^192 / (2 pi), rounded
_TURN = 999031769477504631556283515717616693813654938713089696784


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, stretch: float = 1.0, trained: int | None = None,
                       slow: float = 1.0, fast: float = 32.0) -> torch.Tensor:
    """Angles per position, base^(-2 i / rotary_dim) for i < rotary_dim / 2, fp64 on the host.

    ``stretch`` > 1 adapts them to a context that many times longer than the one
    of the training: all are divided by it, or, where that one's length
    ``trained`` is given, only those that turn less than ``slow`` times in it;
    those that turn more than ``fast`` times stay, and between the two the share
    that is divided falls linearly with the number of turns.  (Models trained with
    a share that falls with the channel's index instead differ by up to 0.38 of it
    at 128 channels; :func:`rotary` takes any frequencies.)
    """
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even, not {rotary_dim}")
    if not (base > 0 and stretch > 0):
        raise ValueError("base and stretch must be positive")
    f = torch.tensor([float(base) ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)], dtype=torch.float64)
    if stretch == 1.0:
        return f
    if trained is None:
        return f / stretch
    if not 0 <= slow < fast:
        raise ValueError("slow must be below fast")
    keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
    return f * keep + f / stretch * (1 - keep)


def rotary(frequencies, *, interleaved: bool = False, factor: float = 1.0, device="cuda") -> Rotary:
    """Lays out the rotation by ``frequencies`` (angles per position, one per pair of channels, on the host)."""
    fixed = []
    for f in torch.as_tensor(frequencies, dtype=torch.float64).tolist():
        if not math.isfinite(f):
            raise ValueError(f"frequency {f}")
        whole = round(Fraction(f) * _TURN / (1 << 128)) % (1 << 64)
        fixed.append(whole - (1 << 64) if whole >> 63 else whole)
    return Rotary(torch.tensor(fixed, dtype=torch.int64, device=device), bool(interleaved), float(factor))


def norm_rotate(q, k, positions, rotary: Rotary, q_out=None, k_out=None, *, q_weight=None, k_weight=None, eps=1e-6,
                stream=None):
    """Norm of each query and key head (where its weight is given), then the rotation by ``positions``.

    q: [T, Hq, d]; k: [T, Hkv, d] (rows may lie apart, as slices of one
    projection); positions: [T] int32; q_weight, k_weight: [d] fp32.  q_out and
    k_out may lie apart too, and may be q and k themselves.  Returns (q_out, k_out).
    """
    T, Hq, d = q.shape
    Hkv, dt = k.shape[1], q.dtype
    code = _dtype_code(q)
    dev = _gpu(q, "q", stream)
    qs, ks = _rows(q, "q", (T, Hq, d), dt, dev), _rows(k, "k", (T, Hkv, d), dt, dev)
    _ok(positions, "positions", (T,), _I32T, dev)
    turns, interleaved, factor = rotary
    _ok(turns, "turns", (turns.shape[0],), _I64T, dev)
    if 2 * turns.shape[0] > d:
        raise ValueError(f"the rotation is of {2 * turns.shape[0]} channels, the heads have {d}")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _ok(w, name, (d,), _F32, dev)
    if q_out is None:
        q_out, qo = _empty((T, Hq, d), dt, q.device, stream), Hq * d
    else:
        qo = _rows(q_out, "q_out", (T, Hq, d), dt, dev)
    if k_out is None:
        k_out, ko = _empty((T, Hkv, d), dt, q.device, stream), Hkv * d
    else:
        ko = _rows(k_out, "k_out", (T, Hkv, d), dt, dev)
    dims = make_dims(Hq, Hkv, d, code)
    _check(_lib.kda_norm_rotate(ctypes.byref(dims), T, _ptr(q), qs, _ptr(k), ks, _ptr(positions), _ptr(turns),
                                2 * turns.shape[0], 1 if interleaved else 0, factor, _ptr(q_weight), _ptr(k_weight), eps,
                                _ptr(q_out), qo, _ptr(k_out), ko, _stream_handle(stream, dev)), "kda_norm_rotate")
    return q_out, k_out


def decode_shared_workspace_bytes(q_heads, kv_heads, head_dim, dtype_code, batch, draft_len, max_pages, groups) -> int:
    """Bytes of workspace that :func:`decode_shared` needs."""
    dims = make_dims(q_heads, kv_heads, head_dim, dtype_code)
    return _lib.kda_attn_decode_shared_workspace_bytes(ctypes.byref(dims), batch, draft_len, max_pages, groups)


def _decode_args(q, cache, seq_lens, block_table, table_shape, out, lse, return_lse, stream):
    """What the forms of :func:`decode` check and allocate alike."""
    dev = _gpu(q, "q", stream)
    Hkv, d, c = _check_cache(cache, dev)
    B, D, Hq, _ = q.shape
    dt = q.dtype
    code = _dtype_code(q)
    qs = _rows(q, "q", (B, D, Hq, d), dt, dev)
    _ok(seq_lens, "seq_lens", (B,), _I32T, dev)
    _ok(block_table, "block_table", table_shape(B, Hkv), _I32T, dev)
    if out is None:
        out = _empty((B, D, Hq, d), dt, q.device, stream)
    else:
        _ok(out, "out", (B, D, Hq, d), dt, dev)
    if lse is None:
        if return_lse:
            lse = _empty((B, D, Hq), _F32, q.device, stream)
    else:
        _ok(lse, "lse", (B, D, Hq), _F32, dev)
    return dev, c, (Hq, Hkv, d, code), qs, out, lse


def decode_shared(q, cache: KVCache, seq_lens, block_table, group_start, shared_pages, out=None, *, lse=None,
                  return_lse=False, workspace=None, scale=None, err_flag=None, stream=None):
    """:func:`decode` for sequences that share prefixes, which are read once for all of them.

    group_start: [groups + 1] int32: sequences group_start[g] to
    group_start[g + 1] - 1 are a group; shared_pages: [groups] int32: so many
    entries of their block table rows, from the first, name the same pages.
    How many rows read a prefix together goes by the groups' mean size (see
    ``include/kda_attn.h``): leave out empty groups and groups of one where time
    counts.  The plan and the sum of the parts cost 15 to 35 us, so short prefixes
    are quicker with :func:`decode`: of 64 sequences (32 heads over 8, d = 128,
    bf16) in groups of 16, prefixes of 16, 64 and 256 pages took 53, 81 and 215 us
    there and 54, 58 and 94 here, in groups of 4 55, 85, 317 and 61, 97, 198; of
    windows of 7 tokens (groups of 8) prefixes of 4, 16 and 64 pages 64, 118, 284
    and 78, 78, 117.  Returns out [B, D, Hq, d], then with ``return_lse`` lse [B, D, Hq] fp32.
    """
    width, groups = block_table.shape[1], shared_pages.shape[0]
    dev, c, dims, qs, out, lse = _decode_args(q, cache, seq_lens, block_table, lambda B, Hkv: (B, width), out, lse,
                                              return_lse, stream)
    flag = _flag(err_flag, dev)
    _ok(group_start, "group_start", (groups + 1,), _I32T, dev)
    _ok(shared_pages, "shared_pages", (groups,), _I32T, dev)
    dims = make_dims(*dims, scale)
    pd = ctypes.byref(dims)
    B, D = q.shape[:2]
    workspace, have = _workspace(
        workspace, lambda: _lib.kda_attn_decode_shared_workspace_bytes(pd, B, D, width, groups), q, dev, stream)
    _check(_lib.kda_attn_decode_shared(pd, ctypes.byref(c), B, D, _ptr(q), qs, _ptr(seq_lens), _ptr(block_table), width,
                                       groups, _ptr(group_start), _ptr(shared_pages), _ptr(out), _ptr(lse), _ptr(workspace),
                                       have, flag, _stream_handle(stream, dev)), "kda_attn_decode_shared")
    return (out, lse) if return_lse else out


def alloc_summary(cache: KVCache) -> KeySummary:
    """Summaries for the pages of ``cache``, not yet filled."""
    N, Hkv, _, d = cache.k_pages.shape
    dev = cache.k_pages.device
    return KeySummary(torch.zeros((N, Hkv, 2, d), dtype=_I8, device=dev), torch.ones((N, Hkv), dtype=_F32, device=dev))


def summarise(cache: KVCache, summary: KeySummary, cu_seqlens, total_tokens: int, start_pos, block_table, *, err_flag=None,
              stream=None):
    """Renews the summaries of the pages that an :func:`append` of ``total_tokens`` tokens with the same
    cu_seqlens, start_pos and block_table wrote."""
    dev = _gpu(cu_seqlens, "cu_seqlens", stream)
    flag = _flag(err_flag, dev)
    Hkv, d, c = _check_cache(cache, dev)
    s = _check_summary(summary, cache.k_pages.shape[0], Hkv, d, dev)
    n, width = block_table.shape
    _ok(cu_seqlens, "cu_seqlens", (n + 1,), _I32T, dev)
    _ok(start_pos, "start_pos", (n,), _I32T, dev)
    _ok(block_table, "block_table", (n, width), _I32T, dev)
    dims = make_dims(Hkv, Hkv, d, 0)
    _check(_lib.kda_cache_summarise(ctypes.byref(dims), ctypes.byref(c), ctypes.byref(s), n, _ptr(cu_seqlens), int(total_tokens),
                                    _ptr(start_pos), _ptr(block_table), width, flag, _stream_handle(stream, dev)),
           "kda_cache_summarise")


def select(q, summary: KeySummary, seq_lens, block_table, budget: int, sink: int = 1, recent: int = 2, *, workspace=None,
           err_flag=None, stream=None) -> Selected:
    """The ``budget`` pages of each sequence and kv head that promise the window's rows the most, the first
    ``sink`` and last ``recent`` pages among them (all pages of sequences with no more than ``budget``).

    q: [B, D, Hq, d]; seq_lens: [B] int32; block_table: [B, max_pages] int32.
    """
    dev = _gpu(q, "q", stream)
    flag = _flag(err_flag, dev)
    B, D, Hq, d = q.shape
    N, Hkv = summary.unit.shape
    s = _check_summary(summary, N, Hkv, d, dev)
    code = _dtype_code(q)
    qs = _rows(q, "q", (B, D, Hq, d), q.dtype, dev)
    width, budget = block_table.shape[1], int(budget)
    _ok(seq_lens, "seq_lens", (B,), _I32T, dev)
    _ok(block_table, "block_table", (B, width), _I32T, dev)
    if budget < 1:
        raise ValueError(f"budget must be positive, not {budget}")
    lens = _like(seq_lens, stream)
    table, index = (_empty((B, Hkv, budget), _I32T, q.device, stream) for _ in range(2))
    dims = make_dims(Hq, Hkv, d, code)
    pd = ctypes.byref(dims)
    workspace, have = _workspace(workspace, lambda: _lib.kda_cache_select_workspace_bytes(pd, B, width), q, dev, stream)
    _check(_lib.kda_cache_select(pd, ctypes.byref(s), N, B, D, _ptr(q), qs, _ptr(seq_lens), _ptr(block_table), width, budget,
                                 int(sink), int(recent), _ptr(lens), _ptr(table), _ptr(index), _ptr(workspace), have, flag,
                                 _stream_handle(stream, dev)), "kda_cache_select")
    return Selected(lens, table, index)


def decode_selected(q, cache: KVCache, selected: Selected, out=None, *, lse=None, return_lse=False, workspace=None,
                    scale=None, err_flag=None, stream=None):
    """:func:`decode` over the selected pages of each kv head.

    Returns out [B, D, Hq, d], then with ``return_lse`` lse [B, D, Hq] fp32 (over the selected positions).
    """
    table = selected.block_table
    width = table.shape[2]
    dev, c, dims, qs, out, lse = _decode_args(q, cache, selected.seq_lens, table, lambda B, Hkv: (B, Hkv, width), out, lse,
                                              return_lse, stream)
    flag = _flag(err_flag, dev)
    dims = make_dims(*dims, scale)
    pd = ctypes.byref(dims)
    B, D = q.shape[:2]
    workspace, have = _workspace(
        workspace, lambda: _lib.kda_attn_decode_workspace_bytes(pd, B, D, width, 0), q, dev, stream)
    _check(_lib.kda_attn_decode_selected(pd, ctypes.byref(c), B, D, _ptr(q), qs, _ptr(selected.seq_lens), _ptr(table), width,
                                         _ptr(out), _ptr(lse), _ptr(workspace), have, flag, _stream_handle(stream, dev)),
           "kda_attn_decode_selected")
    return (out, lse) if return_lse else out
