"""CPU checks of the long-context entry points: bad arguments refused before any
launch, sizing, the rotation table, tensors that are elsewhere, and the fp64
definitions against worked examples."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import attention as ref
from test_attn_abi import BAD, BAD_DIMS, P, _dims, attn  # noqa: F401
from test_attn_devices import BF, CACHE, F32, FLAG, I32, Stand, U8
from test_attn_devices import attn as fenced  # noqa: F401


def _lib():
    from gated_delta_rule_decode_gb300 import kda
    return kda.lib()


def _cache(a):
    return ctypes.byref(a.KdaKvCache(256, 256, 256, 256, 4))


def _summary(a, bounds=256, unit=256):
    return ctypes.byref(a.KdaKeySummary(bounds, unit))


@pytest.mark.parametrize("kw,status", BAD_DIMS)
def test_bad_dims(attn, kw, status):  # noqa: F811
    lib, d, c, s = _lib(), _dims(attn, **kw), _cache(attn), _summary(attn)
    assert lib.kda_norm_rotate(d, 4, P, 1 << 16, P, 1 << 16, P, P, 32, 0, 1.0, P, P, 1e-6, P, 1 << 16, P, 1 << 16, None) == status
    assert lib.kda_attn_decode_shared(d, c, 1, 1, P, 1 << 16, P, P, 4, 1, P, P, P, None, P, 1 << 40, None, None) == status
    assert lib.kda_attn_decode_selected(d, c, 1, 1, P, 1 << 16, P, P, 4, P, None, P, 1 << 40, None, None) == status
    assert lib.kda_cache_summarise(d, c, s, 1, P, 64, P, P, 4, None, None) == status
    assert lib.kda_cache_select(d, s, 4, 1, 1, P, 1 << 16, P, P, 4, 3, 1, 2, P, P, P, P, 1 << 40, None, None) == status
    assert lib.kda_attn_decode_shared_workspace_bytes(d, 1, 1, 4, 1) == 0
    assert lib.kda_cache_select_workspace_bytes(d, 1, 4) == 0


def test_norm_rotate_refusals(attn):  # noqa: F811
    d = _dims(attn)

    def call(T=4, q=P, qs=512, k=P, ks=128, pos=P, turns=P, rot=64, factor=1.0, qw=P, kw=None, eps=1e-6, qo=P, qos=512,
             ko=P, kos=128):
        return _lib().kda_norm_rotate(d, T, q, qs, k, ks, pos, turns, rot, 0, factor, qw, kw, eps, qo, qos, ko, kos, None)
    assert call(T=0) == 0
    for kw in (dict(T=-1), dict(T=1 << 31), dict(q=None), dict(k=BAD), dict(pos=None), dict(turns=None),
               dict(turns=ctypes.c_void_p(260)), dict(rot=63), dict(rot=-2), dict(rot=66), dict(factor=math.nan),
               dict(factor=math.inf), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(qw=BAD),
               dict(kw=ctypes.c_void_p(260)), dict(qo=None), dict(ko=BAD), dict(qs=504), dict(ks=127), dict(qos=0),
               dict(kos=129), dict(qos=1024), dict(kos=256)):  # (the last two: in place with another distance)
        assert call(**kw) == -1, kw


def test_shared_refusals_and_sizes(attn):  # noqa: F811
    lib, d = _lib(), _dims(attn)
    need = lib.kda_attn_decode_shared_workspace_bytes(d, 3, 2, 10, 2)
    assert need > 0
    for bad in ((d, -1, 2, 10, 2), (d, 3, 0, 10, 2), (d, 3, 17, 10, 2), (d, 3, 2, -1, 2), (d, 3, 2, 10, -1),
                (d, 3, 2, 10, 1 << 21), (d, (1 << 31) - 1, 2, 10, 1), (d, 0, 2, 10, 1)):
        assert lib.kda_attn_decode_shared_workspace_bytes(*bad) == 0

    def call(B=3, D=2, q=P, qs=512, lens=P, table=P, width=10, groups=2, start=P, shared=P, out=P, lse=None, ws=P, nb=need):
        return lib.kda_attn_decode_shared(d, _cache(attn), B, D, q, qs, lens, table, width, groups, start, shared, out, lse,
                                          ws, nb, None, None)
    assert call(B=0) == 0
    for kw in (dict(B=-1), dict(D=0), dict(D=17), dict(q=BAD), dict(qs=511), dict(lens=None), dict(table=None),
               dict(width=-1), dict(width=1 << 26), dict(out=None), dict(lse=BAD), dict(groups=-1), dict(groups=1 << 21),
               dict(start=None), dict(shared=BAD), dict(B=(1 << 31) - 1)):
        assert call(**kw) == -1, kw
    for kw in (dict(ws=None), dict(nb=need - 1), dict(ws=ctypes.c_void_p(272))):
        assert call(**kw) == -4, kw


def test_selection_refusals_and_sizes(attn):  # noqa: F811
    lib, d = _lib(), _dims(attn)
    assert lib.kda_cache_select_workspace_bytes(d, 3, 10) == 3 * 2 * 10 * 4
    for bad in ((d, -1, 10), (d, 3, -1), (d, 3, 1 << 26)):
        assert lib.kda_cache_select_workspace_bytes(*bad) == 0
    need = 3 * 2 * 10 * 4

    def select(s=None, N=4, B=3, D=1, q=P, qs=512, lens=P, table=P, width=10, budget=4, sink=1, recent=2, lo=P, to=P, io=P,
               ws=P, nb=need):
        return lib.kda_cache_select(d, s or _summary(attn), N, B, D, q, qs, lens, table, width, budget, sink, recent, lo, to,
                                    io, ws, nb, None, None)
    assert select(B=0) == 0
    for kw in (dict(N=-1), dict(N=1 << 31), dict(s=_summary(attn, 0)), dict(s=_summary(attn, 256, 258)),
               dict(s=_summary(attn, 260)), dict(B=-1), dict(D=0), dict(D=17), dict(q=BAD), dict(qs=511), dict(lens=None),
               dict(table=None), dict(width=-1), dict(budget=2), dict(sink=-1), dict(recent=0), dict(D=2, recent=1),
               dict(sink=(1 << 31) - 1), dict(budget=1 << 26), dict(lo=None), dict(to=BAD), dict(io=None)):
        assert select(**kw) == -1, kw
    for kw in (dict(ws=None), dict(nb=need - 1), dict(ws=ctypes.c_void_p(272))):
        assert select(**kw) == -4, kw

    def summarise(c=None, s=None, n=1, cu=P, T=64, start=P, table=P, width=4):
        return lib.kda_cache_summarise(d, c or _cache(attn), s or _summary(attn), n, cu, T, start, table, width, None, None)
    assert summarise(n=0) == 0 and summarise(T=0) == 0
    for kw in (dict(c=ctypes.byref(attn.KdaKvCache(0, 256, 256, 256, 4))), dict(s=_summary(attn, 0)),
               dict(s=_summary(attn, 256, 258)), dict(n=-1), dict(T=-1), dict(T=1 << 31), dict(cu=None), dict(start=None),
               dict(table=None), dict(width=-1), dict(width=1 << 26)):
        assert summarise(**kw) == -1, kw

    size = lib.kda_attn_decode_workspace_bytes(d, 3, 2, 10, 0)

    def attend(B=3, D=2, q=P, qs=512, lens=P, table=P, width=10, out=P, lse=None, ws=P, nb=size):
        return lib.kda_attn_decode_selected(d, _cache(attn), B, D, q, qs, lens, table, width, out, lse, ws, nb, None, None)
    assert attend(B=0) == 0
    for kw in (dict(B=-1), dict(D=17), dict(q=BAD), dict(qs=511), dict(lens=None), dict(table=None), dict(width=-1),
               dict(out=None), dict(lse=BAD)):
        assert attend(**kw) == -1, kw
    for kw in (dict(ws=None), dict(nb=size - 1), dict(ws=ctypes.c_void_p(272))):
        assert attend(**kw) == -4, kw


# ---------------------------------------------------------------- the binding's checks

SUMMARY = dict(bounds=Stand((5, 2, 2, 64), torch.int8), unit=Stand((5, 2), F32))
CALLS = {
    "norm_rotate": dict(q=Stand((9, 4, 64), BF), k=Stand((9, 2, 64), BF), positions=Stand((9,), I32),
                        turns=Stand((16,), torch.int64), q_weight=Stand((64,), F32), k_weight=Stand((64,), F32),
                        q_out=Stand((9, 4, 64), BF), k_out=Stand((9, 2, 64), BF)),
    "decode_shared": dict(**CACHE, q=Stand((3, 2, 4, 64), BF), seq_lens=Stand((3,), I32), block_table=Stand((3, 4), I32),
                          group_start=Stand((2,), I32), shared_pages=Stand((1,), I32), out=Stand((3, 2, 4, 64), BF),
                          lse=Stand((3, 2, 4), F32), workspace=Stand((1 << 24,), U8), **FLAG),
    "summarise": dict(cu_seqlens=Stand((3,), I32), **CACHE, **SUMMARY, start_pos=Stand((2,), I32),
                      block_table=Stand((2, 4), I32), **FLAG),
    "select": dict(q=Stand((2, 3, 4, 64), BF), **SUMMARY, seq_lens=Stand((2,), I32), block_table=Stand((2, 9), I32),
                   workspace=Stand((1 << 20,), U8), **FLAG),
    "decode_selected": dict(**CACHE, q=Stand((2, 3, 4, 64), BF), seq_lens=Stand((2,), I32), block_table=Stand((2, 2, 4), I32),
                            out=Stand((2, 3, 4, 64), BF), lse=Stand((2, 3, 4), F32), workspace=Stand((1 << 24,), U8), **FLAG),
}


def _call(a, name, args, **more):
    args = dict(args)
    if "k_pages" in args:
        args["cache"] = a.KVCache(*(args.pop(x) for x in a.KVCache._fields))
    if "bounds" in args:
        args["summary"] = a.KeySummary(args.pop("bounds"), args.pop("unit"))
    if "turns" in args:
        args["rotary"] = a.Rotary(args.pop("turns"))
    if name == "summarise":
        args["total_tokens"] = 9
    if name == "select":
        args["budget"] = 4
    if name == "decode_selected":
        args["selected"] = a.Selected(args.pop("seq_lens"), args.pop("block_table"), None)
    return getattr(a, name)(**args, **more)


@pytest.mark.parametrize("name,arg", [(n, x) for n, args in CALLS.items() for x in args])
@pytest.mark.parametrize("dev", [1, -1])
def test_a_tensor_elsewhere_is_refused(fenced, name, arg, dev, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch, "empty_like", lambda t: t)
    monkeypatch.setattr(fenced, "_empty", lambda shape, dtype, device, stream: Stand(shape, dtype))
    args = dict(CALLS[name])
    args[arg] = args[arg].on(dev)
    with pytest.raises(ValueError, match=arg.split("_pages")[0]):
        _call(fenced, name, args)


@pytest.mark.parametrize("name", CALLS)
def test_a_call_for_another_gpu_is_refused(fenced, name):  # noqa: F811
    with pytest.raises(ValueError, match="cuda:1"):
        _call(fenced, name, {k: v.on(1) for k, v in CALLS[name].items()})


@pytest.mark.parametrize("name,arg,shape,dtype", [
    ("norm_rotate", "k", (8, 2, 64), BF), ("norm_rotate", "k", (9, 2, 64), F32), ("norm_rotate", "positions", (9,), F32),
    ("norm_rotate", "turns", (33,), torch.int64), ("norm_rotate", "q_weight", (32,), F32), ("norm_rotate", "q_out", (9, 2, 64), BF),
    ("decode_shared", "group_start", (3,), I32), ("decode_shared", "shared_pages", (1,), torch.int64),
    ("decode_shared", "block_table", (2, 4), I32), ("summarise", "bounds", (4, 2, 2, 64), torch.int8),
    ("summarise", "unit", (5, 2), BF), ("summarise", "start_pos", (3,), I32), ("select", "bounds", (5, 2, 64), torch.int8),
    ("select", "seq_lens", (3,), I32), ("decode_selected", "block_table", (2, 1, 4), I32),
    ("decode_selected", "seq_lens", (3,), I32)])
def test_wrong_shapes_and_types_are_refused(fenced, name, arg, shape, dtype):  # noqa: F811
    with pytest.raises((ValueError, TypeError)):
        _call(fenced, name, dict(CALLS[name], **{arg: Stand(shape, dtype)}))


# ---------------------------------------------------------------- the rotation table

def test_turns_are_exact_to_half_a_unit(attn):  # noqa: F811
    # 1 / (2 pi) in 80 digits, of pi by the arctangents of 1/5 and 1/239
    def arctan(n):
        one, total, k, sign = 10 ** 90, 0, 1, 1
        term = one // n
        while term:
            total += sign * (term // k)
            term //= n * n
            k, sign = k + 2, -sign
        return Fraction(total, one)
    pi = 16 * arctan(5) - 4 * arctan(239)
    f = torch.tensor([1.0, 0.1, 3.3e-7, 0.0, -2.5, 1e4], dtype=torch.float64)
    got = attn.rotary(f, device="cpu").turns.tolist()
    for x, t in zip(f.tolist(), got):
        off = (Fraction(x) / (2 * pi) * 2 ** 64 - t) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 1000)
    with pytest.raises(ValueError):
        attn.rotary([math.nan], device="cpu")


def test_frequencies(attn):  # noqa: F811
    f = attn.rotary_frequencies(64)
    assert f.dtype == torch.float64 and f[0] == 1 and math.isclose(f[16], 0.01) and len(f) == 32
    assert torch.allclose(attn.rotary_frequencies(64, stretch=4.0), f / 4)
    g = attn.rotary_frequencies(64, stretch=4.0, trained=8192)
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32]) and torch.allclose(g[turns <= 1], f[turns <= 1] / 4)
    assert ((g <= f) & (g >= f / 4)).all() and len(attn.rotary_frequencies(0)) == 0
    for kw in (dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, base=0), dict(rotary_dim=8, stretch=0),
               dict(rotary_dim=8, stretch=2, trained=64, slow=3, fast=3)):
        with pytest.raises(ValueError):
            attn.rotary_frequencies(**kw)


# ---------------------------------------------------------------- the definitions

def test_rotate_worked_example():
    x = np.array([[[3.0, 4.0, 1.0, 0.0]]])
    quarter = [1 << 62]
    y, _ = ref.rotate(x, [1], quarter, interleaved=True)
    assert np.allclose(y, [[[-4, 3, 1, 0]]])
    y, _ = ref.rotate(x, [2], [1 << 62, 0], factor=2.0)  # half a turn of (x0, x2); (x1, x3) stay, times 2
    assert np.allclose(y, [[[-6, 8, -2, 0]]])
    y, _ = ref.rotate(x, [5], [], weight=[1, 1, 1, 2.0], eps=0.0)
    assert np.allclose(y, x / math.sqrt(26 / 4))


def test_summary_and_selection_worked_example():
    assert ref.unit_of(127) == 1 and ref.unit_of(127.5) == 2 and ref.unit_of(0) == 2.0 ** -126 and ref.unit_of(1) == 2.0 ** -6
    pages, scale = np.zeros((3, 1, 64, 32), np.uint8), np.full((3, 1), 2.0)
    one, two = int(ref.e4m3_round(np.array([1.0]))[0]), int(ref.e4m3_round(np.array([-2.0]))[0])
    pages[1, 0, 0, 3], pages[1, 0, 1, 3], pages[1, 0, 2, 4], pages[1, 0, 0, 5] = one, two, one, 0x7f
    b, u = ref.summarise(pages, scale, np.zeros((3, 1, 2, 32)), np.ones((3, 1)), [0, 2], [0], [[1]])
    # 2 positions: channel 3 has 2 and -4, the third row is not there, a NaN is passed over
    assert u[1, 0] == 2.0 ** -4 and b[1, 0, 0, 3] == 32 and b[1, 0, 1, 3] == -64 and np.abs(b[1, 0]).sum() == 96
    assert u[0, 0] == 1 and u[2, 0] == 1
    q = np.zeros((1, 1, 1, 32))
    q[..., 3] = -1.0  # 64 units of 2^-6: 64 * 64 * 2^-6 * 2^-4 = 4 = -1 * -4
    assert ref.page_scores(q, b, u, [1, 0, 7], 0, 0, 1).tolist() == [4, 0, -math.inf]
    l, t, i = ref.select(q, b, u, np.array([5 * 64 - 3]), np.array([[0, 2, 1, 0, 2]]), 3, 1, 1)
    assert l[0] == 3 * 64 - 3 and i.tolist() == [[[0, 2, 4]]] and t.tolist() == [[[0, 1, 2]]]
    l, t, i = ref.select(q, b, u, np.array([5 * 64 - 3]), np.array([[0, 2, 0, 2, 2]]), 3, 1, 1)
    assert i.tolist() == [[[0, 1, 4]]]  # equal scores: the lower index
