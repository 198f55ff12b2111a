"""Canary pages around every buffer that the attention operators write, and
no change in those that they only read (see test_gpu_canary.py)."""
import pytest
import torch

from attn_testutil import cu_of, gen, make_cache, randn
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu


def _attn():
    from gated_delta_rule_decode_gb300 import attn
    return attn


def _guarded_cache(gd, cache):
    f8 = torch.float8_e4m3fn
    k, v, ks, vs = (gd.like(x.cuda()) for x in cache)
    return _attn().KVCache(k.view(f8), v.view(f8), ks, vs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,hq,hkv", [(32, 3, 1), (64, 4, 4), (128, 10, 2)])
def test_prefill_canaries(d, hq, hkv, dtype):
    g = gen(1)
    lens = [130, 0, 1, 300]
    q, k, v = (gd_t.cuda() for gd_t in (randn(g, 431, hq, d, dtype=dtype), randn(g, 431, hkv, d, dtype=dtype),
                                        randn(g, 431, hkv, d, dtype=dtype)))
    gd = Guarded()
    out, lse = gd.empty((431, hq, d), dtype), gd.empty((431, hq), torch.float32)
    _attn().prefill(q, k, v, cu_of(lens).cuda(), out, lse=lse)
    gd.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,start", [([1, 1, 1], [0, 63, 130]), ([200, 3, 64], [5, 61, 64])])
def test_append_canaries(lens, start, dtype):
    g = gen(2)
    cache = make_cache(g, 24, 2, 64)
    gd = Guarded()
    c = _guarded_cache(gd, cache)
    table = torch.arange(24, dtype=torch.int32).flip(0).view(3, 8)
    T = sum(lens)
    _attn().append(c, randn(g, T, 2, 64, dtype=dtype).cuda(), 100 * randn(g, T, 2, 64, dtype=dtype).cuda(), cu_of(lens).cuda(),
                   torch.tensor(start, dtype=torch.int32).cuda(), table.cuda())
    gd.check()
    # pages that hold none of the new positions are as they were
    used = {int(table[s, x // 64]) for s in range(3) for x in range(start[s], start[s] + lens[s])}
    for page in set(range(24)) - used:
        assert torch.equal(c.k_pages.view(torch.uint8)[page].cpu(), cache[0][page])
        assert torch.equal(c.v_pages.view(torch.uint8)[page].cpu(), cache[1][page])


@pytest.mark.parametrize("dtype,D,hq,hkv", [(torch.bfloat16, 1, 4, 1), (torch.bfloat16, 7, 8, 2), (torch.bfloat16, 3, 4, 1),
                                            (torch.float32, 1, 4, 2), (torch.float32, 5, 8, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_canaries(d, dtype, D, hq, hkv):
    a = _attn()
    g = gen(3)
    lens = [300, 0, 7, 64, 129]
    cache = make_cache(g, 30, hkv, d)
    gd = Guarded()
    c = _guarded_cache(gd, cache)
    table = torch.arange(30, dtype=torch.int32).view(5, 6).cuda()
    q = randn(g, 5, D, hq, d, dtype=dtype).cuda()
    code = 1 if dtype == torch.bfloat16 else 0
    out, lse = gd.empty((5, D, hq, d), dtype), gd.empty((5, D, hq), torch.float32)
    w = gd.empty((5, 6), torch.float32)
    ws = gd.workspace(a.decode_workspace_bytes(hq, hkv, d, code, 5, D, 6, True))
    a.decode(q, c, torch.tensor(lens, dtype=torch.int32).cuda(), table, out, lse=lse, weight_out=w, workspace=ws)
    gd.check()
    for got, want in zip((c.k_pages, c.v_pages), cache[:2]):
        assert torch.equal(got.view(torch.uint8).cpu(), want)


@pytest.mark.parametrize("width", [7, 600])
def test_evict_canaries(width):
    g = gen(4)
    gd = Guarded()
    B = 3
    lens = gd.like(torch.tensor([width * 64, 64, 5 * 64 + 1], dtype=torch.int32).cuda())
    table = gd.like(torch.arange(B * width, dtype=torch.int32).view(B, width).cuda())
    w = gd.like(torch.rand(B, width, generator=g).cuda())
    lib = _attn()._lib
    freed, count = gd.empty((B, width), torch.int32), gd.empty((B,), torch.int32)
    p = [x.data_ptr() for x in (lens, table, w, lens, table, w, freed, count)]
    assert lib.kda_cache_evict(B, width, 4, 1, 1, *p, None, torch.cuda.current_stream().cuda_stream) == 0
    gd.check()
    assert count.tolist() == [width - 4, 0, 2]
