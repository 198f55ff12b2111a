"""CPU checks of the attention entry points: declared and exported, bad
arguments refused before any launch (no call here reaches a kernel), sizing,
and the fp64 definitions against worked examples."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

from oracle import attention as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(256)  # never dereferenced
BAD = ctypes.c_void_p(258)


@pytest.fixture(scope="module")
def attn():
    from gated_delta_rule_decode_gb300 import build
    build.build()
    from gated_delta_rule_decode_gb300 import attn as mod
    return mod


def test_declared_and_exported(attn):
    text = open(os.path.join(ROOT, "include", "kda_attn.h")).read()
    names = re.findall(r"KDA_API\s+[\w\s\*]+?\b(kda_\w+)\s*\(", text)
    assert sorted(names) == sorted(attn.EXPORTED)


def _dims(attn, hq=8, hkv=2, d=64, dt=1, scale=0.0):
    return ctypes.byref(attn.KdaAttnDims(hq, hkv, d, dt, scale))


BAD_DIMS = [(dict(hq=0), -1), (dict(hkv=0), -1), (dict(hq=9), -1), (dict(d=96), -2), (dict(dt=5), -2),
            (dict(hq=129, hkv=1), -2), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1)]


@pytest.mark.parametrize("kw,status", BAD_DIMS)
def test_bad_dims(attn, kw, status):
    from gated_delta_rule_decode_gb300 import kda
    lib, d = kda.lib(), _dims(attn, **kw)
    c = ctypes.byref(attn.KdaKvCache(256, 256, 256, 256, 4))
    assert lib.kda_attn_prefill(d, 1, P, 64, P, 1 << 16, P, 1 << 16, P, 1 << 16, P, None, None, None) == status
    assert lib.kda_cache_append(d, c, 1, P, 64, P, 1 << 16, P, 1 << 16, P, P, 4, None, None) == status
    assert lib.kda_attn_decode(d, c, 1, 1, P, 1 << 16, P, P, 4, P, None, None, None, P, 1 << 30, None, None) == status
    assert lib.kda_attn_decode_workspace_bytes(d, 4, 1, 16, 1) == 0


def test_prefill_refusals(attn):
    from gated_delta_rule_decode_gb300 import kda
    f, d = kda.lib().kda_attn_prefill, _dims(attn)

    def call(n=1, cu=P, T=64, q=P, qs=512, k=P, ks=128, v=P, vs=128, out=P, lse=None):
        return f(d, n, cu, T, q, qs, k, ks, v, vs, out, lse, None, None)
    assert f(None, 1, P, 64, P, 512, P, 128, P, 128, P, None, None, None) == -1
    assert call(n=0) == 0 and call(T=0) == 0
    for kw in (dict(n=-1), dict(T=-1), dict(T=1 << 31), dict(cu=None), dict(q=None), dict(k=BAD), dict(v=BAD),
               dict(out=None), dict(lse=BAD), dict(qs=504), dict(ks=127), dict(ks=129), dict(vs=0), dict(vs=1 << 40)):
        assert call(**kw) == -1, kw


def test_cache_refusals(attn):
    from gated_delta_rule_decode_gb300 import kda
    lib, d = kda.lib(), _dims(attn)
    big = (1 << 31) // 128

    def append(c, n=1, T=64, k=P, start=P, table=P, width=4):
        return lib.kda_cache_append(d, c, n, P, T, k, 128, P, 128, start, table, width, None, None)
    good = ctypes.byref(attn.KdaKvCache(256, 256, 256, 256, 4))
    assert append(good, n=0) == 0 and append(good, T=0) == 0
    for c in (None, ctypes.byref(attn.KdaKvCache(256, 256, 256, 256, -1)), ctypes.byref(attn.KdaKvCache(0, 256, 256, 256, 4)),
              ctypes.byref(attn.KdaKvCache(256, 258, 256, 256, 4)), ctypes.byref(attn.KdaKvCache(256, 256, 0, 256, 4)),
              ctypes.byref(attn.KdaKvCache(256, 256, 256, 256, big))):
        assert append(c) == -1
        assert lib.kda_attn_decode(d, c, 1, 1, P, 512, P, P, 4, P, None, None, None, P, 1 << 30, None, None) == -1
    for kw in (dict(n=-1), dict(k=BAD), dict(start=None), dict(table=None), dict(width=-1), dict(width=1 << 30)):
        assert append(good, **kw) == -1, kw


def test_decode_refusals_and_sizes(attn):
    from gated_delta_rule_decode_gb300 import kda
    lib, d = kda.lib(), _dims(attn)
    c = ctypes.byref(attn.KdaKvCache(256, 256, 256, 256, 4))
    need = lib.kda_attn_decode_workspace_bytes(d, 3, 2, 10, 0)
    more = lib.kda_attn_decode_workspace_bytes(d, 3, 2, 10, 1)
    # the weights' share: lse and a value per page for 3 x 2 x 8 rows, in blocks of 64 floats
    assert need > 0 and more - need == 4 * (64 + 512)
    for bad in ((d, -1, 2, 10, 0), (d, 3, 0, 10, 0), (d, 3, 17, 10, 0), (d, 3, 2, -1, 0), (d, 0, 2, 10, 0)):
        assert lib.kda_attn_decode_workspace_bytes(*bad) == 0

    def call(B=3, D=2, q=P, qs=512, lens=P, table=P, width=10, out=P, lse=None, win=None, wout=None, ws=P, nb=need):
        return lib.kda_attn_decode(d, c, B, D, q, qs, lens, table, width, out, lse, win, wout, ws, nb, None, None)
    assert call(B=0) == 0
    for kw in (dict(B=-1), dict(D=0), dict(D=17), dict(q=BAD), dict(qs=511), dict(lens=None), dict(table=None),
               dict(width=-1), dict(width=1 << 26), dict(out=None), dict(lse=BAD), dict(win=P), dict(win=BAD, wout=P)):
        assert call(**kw) == -1, kw
    for kw in (dict(ws=None), dict(nb=need - 1), dict(ws=ctypes.c_void_p(272)), dict(wout=P, nb=more - 1)):
        assert call(**kw) == -4, kw


def test_evict_refusals(attn):
    from gated_delta_rule_decode_gb300 import kda

    def call(B=2, width=8, budget=4, sink=1, recent=1, **ptr):
        names = ("lens", "table", "weight", "lens_out", "table_out", "weight_out", "freed", "count")
        return kda.lib().kda_cache_evict(B, width, budget, sink, recent, *[ptr.get(x, P) for x in names], None, None)
    assert call(B=0) == 0
    for kw in (dict(B=-1), dict(width=-1), dict(budget=1), dict(sink=-1), dict(recent=0), dict(sink=(1 << 31) - 1),
               dict(lens=None), dict(table=BAD), dict(weight=None), dict(freed=None), dict(count=BAD)):
        assert call(**kw) == -1, kw


# ---------------------------------------------------------------- the definitions

def test_e4m3():
    v = ref.e4m3_values()
    assert v[0x7e] == 448 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1 and math.isnan(v[0x7f])
    fin = ~np.isnan(v)
    assert (ref.e4m3_round(v[fin]) == np.arange(256, dtype=np.uint8)[fin]).all()
    # ties go to the even fraction; beyond the range saturates
    assert ref.e4m3_round(np.array([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 1e9, -1e9])).tolist() == \
        [0x38, 0x3a, 0x00, 0x02, 0x7e, 0xfe]
    import torch
    x = torch.randn(4096, generator=torch.Generator().manual_seed(0)) * 30
    assert (x.to(torch.float8_e4m3fn).view(torch.uint8).numpy() == ref.e4m3_round(x.double().numpy())).all()


def test_pow2_need():
    for a, s in ((448.0, 1.0), (448.1, 2.0), (7.0, 2.0 ** -6), (7.01, 2.0 ** -5), (0.0, 2.0 ** -126), (1.0, 2.0 ** -8)):
        assert ref.pow2_need(a) == s


def test_prompt_worked_example():
    # two tokens, d = 1, scale 1: token 1 weighs the keys by e^0 and e^ln 3
    q = np.array([[[5.0]], [[1.0]]])
    k = np.array([[[0.0]], [[math.log(3)]]])
    v = np.array([[[1.0]], [[9.0]]])
    o, l, a, _ = ref.prompt(q, k, v, [0, 2], scale=1.0)
    assert np.allclose(o.ravel(), [1.0, 7.0]) and np.allclose(l.ravel(), [0.0, math.log(4)])
    o, l, _, _ = ref.prompt(q, k, v, [0, 1, 2], scale=1.0)  # apart: each sees itself only
    assert np.allclose(o.ravel(), [1.0, 9.0])


def test_append_and_decode_definitions_agree_with_prompt():
    rng = np.random.default_rng(0)
    x, y = rng.standard_normal((70, 1, 32)), rng.standard_normal((70, 1, 32))
    kp, ks = ref.append(np.zeros((2, 1, 64, 32), np.uint8), np.ones((2, 1)), x, [0, 70], [0], [[1, 0]], False)
    vp, vs = ref.append(np.zeros((2, 1, 32, 64), np.uint8), np.ones((2, 1)), y, [0, 70], [0], [[1, 0]], True)
    val = ref.e4m3_values()
    k = np.concatenate([val[kp[1, 0]] * ks[1, 0], val[kp[0, 0, :6]] * ks[0, 0]])
    v = np.concatenate([val[vp[1, 0]].T * vs[1, 0], val[vp[0, 0, :, :6]].T * vs[0, 0]])
    assert np.abs(k - x[:, 0]).max() <= 2.0 ** -4 * np.abs(x).max()
    q = rng.standard_normal((70, 2, 32))
    want, lse, _, _ = ref.prompt(q, k[:, None], v[:, None], [0, 70])
    got, l2, _, _, mass = ref.decode(q[None, -3:], kp, vp, ks, vs, np.array([70]), np.array([[1, 0]]))
    assert np.allclose(got[0], want[-3:]) and np.allclose(l2[0], lse[-3:]) and np.isclose(mass.sum(), 6)


def test_evict_worked_example():
    lens, table = np.array([5 * 64 - 1], np.int32), np.array([[10, 11, 12, 13, 14, 15]], np.int32)
    w = np.array([[0, 2, 1, 1, 0, 9]], np.float32)
    l, t, x, f, c = ref.evict(lens, table, w, 4, 1, 1)
    # pages 2 and 3 weigh the same: the lower index stays
    assert l[0] == 4 * 64 - 1 and t.tolist() == [[10, 11, 12, 14, 15, -1]] and f[0, 0] == 13 and c[0] == 1
    assert x.tolist() == [[0, 2, 1, 0, 9, 0]]
