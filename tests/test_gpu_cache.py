"""The 8-bit paged cache: append and eviction against their definitions, byte
for byte."""
import numpy as np
import pytest
import torch

from attn_testutil import DT, cu_of, gen, make_cache, np64, randn, to_device
from oracle import attention as ref

pytestmark = pytest.mark.gpu


def _attn():
    from gated_delta_rule_decode_gb300 import attn
    return attn


def _append(cache, k, v, cu, start, table, **kw):
    c = to_device(cache)
    _attn().append(c, k.cuda(), v.cuda(), cu.cuda(), start.cuda(), table.cuda(), **kw)
    return [x.cpu() for x in (c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.k_scale, c.v_scale)]


def _want(cache, k, v, cu, start, table):
    kp, vp, ks, vs = (x.numpy() for x in cache)
    wk, sk = ref.append(kp, ks, np64(k), cu.tolist(), start.tolist(), table.tolist(), False)
    wv, sv = ref.append(vp, vs, np64(v), cu.tolist(), start.tolist(), table.tolist(), True)
    return wk, wv, sk, sv


def _compare(got, want):
    for g, w, what in zip(got, want, ("k pages", "v pages", "k scales", "v scales")):
        g = g.numpy()
        if g.dtype == np.uint8:
            nan = ((g & 0x7f) == 0x7f) & ((w & 0x7f) == 0x7f)  # a NaN byte's sign is free
            assert ((g == w) | nan).all(), f"{what}: {int(((g != w) & ~nan).sum())} bytes differ"
        else:
            assert (g.astype(np.float64) == w).all(), what


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,heads", [(32, 3), (64, 1), (128, 2)])
@pytest.mark.parametrize("lens,start", [
    ([1], [0]), ([1], [63]), ([1, 1, 1], [64, 5, 130]), ([64], [0]), ([65, 0, 3], [0, 10, 62]),
    ([200, 7], [37, 57]), ([130], [1]),
])
def test_append_matches_definition(lens, start, d, heads, dtype):
    g = gen(sum(lens) + d)
    n, width = len(lens), 7
    cache = make_cache(g, n * width, heads, d)
    cache = (cache[0], cache[1], cache[2] / 4, cache[3] / 4)  # old scales that have to grow
    T = sum(lens)
    k, v = randn(g, T, heads, d).to(DT[dtype]), (100 * randn(g, T, heads, d)).to(DT[dtype])
    table = torch.randperm(n * width, generator=g).reshape(n, width).int()
    cu, st = cu_of(lens), torch.tensor(start, dtype=torch.int32)
    _compare(_append(cache, k, v, cu, st, table), _want(cache, k, v, cu, st, table))


def test_append_extremes():
    """Zeros, the smallest and largest magnitudes, exact ties, infinities and NaN."""
    g = gen(3)
    d, heads = 64, 2
    cache = make_cache(g, 4, heads, d)
    k = randn(g, 70, heads, d)
    v = torch.zeros(70, heads, d)
    k[0] = 0.0
    k[1, 0] = 1e-44
    k[2, 1] = torch.linspace(-448, 448, d)
    k[3] = 8.5                      # half way between two e4m3 values at scale 1
    k[65, 0, 5], k[66, 1, 7], k[67, 1, 7] = float("nan"), float("inf"), -float("inf")
    v[64:] = 3e38
    v[1, 0, 0] = 1e-45
    cu, st = cu_of([70]), torch.tensor([0], dtype=torch.int32)
    table = torch.tensor([[2, 0]], dtype=torch.int32)
    got = _append(cache, k, v, cu, st, table)
    _compare(got, _want(cache, k, v, cu, st, table))
    assert (got[0][0, 0, 1, 5] & 0x7f) == 0x7f
    assert got[0][0, 1, 2, 7] == 0x7e and got[0][0, 1, 3, 7] == 0xfe  # saturated


def test_token_by_token_equals_one_call_up_to_subnormals():
    """Growing a page one token at a time gives the bytes of a single call,
    except where a value passed through e4m3's subnormals on the way."""
    a = _attn()
    g = gen(8)
    d, heads, n = 64, 2, 100
    k, v = randn(g, n, heads, d), randn(g, n, heads, d) * torch.exp(0.02 * torch.arange(n))[:, None, None]
    table = torch.tensor([[1, 0]], dtype=torch.int32).cuda()
    one, many = a.alloc_cache(2, heads, d), a.alloc_cache(2, heads, d)
    a.append(one, k.cuda(), v.cuda(), cu_of([n]).cuda(), torch.zeros(1, dtype=torch.int32).cuda(), table)
    for i in range(n):
        a.append(many, k[i:i + 1].cuda(), v[i:i + 1].cuda(), cu_of([1]).cuda(),
                 torch.tensor([i], dtype=torch.int32).cuda(), table)
    assert torch.equal(one.k_scale, many.k_scale) and torch.equal(one.v_scale, many.v_scale)
    for x, y in ((one.k_pages, many.k_pages), (one.v_pages, many.v_pages)):
        x, y = x.float(), y.float()
        assert (x - y).abs().max() <= 2.0 ** -9  # one subnormal step
        normal = x.abs() >= 2.0 ** -5
        assert torch.equal(x[normal], y[normal])


def test_append_skips_pages_outside_the_cache():
    a = _attn()
    from gated_delta_rule_decode_gb300 import kda
    g = gen(4)
    cache = make_cache(g, 3, 1, 32)
    k, v = randn(g, 140, 1, 32), randn(g, 140, 1, 32)
    cu, st = cu_of([140]), torch.zeros(1, dtype=torch.int32)
    for row in ([1, 3, 0], [1, -1, 0], [1, 0]):  # the last: a row too short
        table = torch.tensor([row], dtype=torch.int32)
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _append(cache, k, v, cu, st, table, err_flag=flag)
        assert flag.item() == a.KDA_DEVERR_PAGE
        _compare(got, _want(cache, k, v, cu, st, table))
    # a negative start skips the sequence
    got = _append(cache, k, v, cu, torch.tensor([-1], dtype=torch.int32), torch.tensor([[0, 1, 2]], dtype=torch.int32))
    _compare(got, [x.numpy() for x in cache])
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    _append(cache, k, v, torch.tensor([0, 141], dtype=torch.int32), st, torch.tensor([[0, 1, 2]], dtype=torch.int32),
            err_flag=flag)
    assert flag.item() & kda.KDA_DEVERR_SEQLENS


def test_append_reads_slices_of_a_fused_projection():
    g = gen(6)
    cache = make_cache(g, 4, 2, 64)
    k, v = randn(g, 90, 2, 64).bfloat16(), randn(g, 90, 2, 64).bfloat16()
    row = torch.cat([randn(g, 90, 4, 64).bfloat16(), k, v], 1)
    cu, st, table = cu_of([90]), torch.tensor([30], dtype=torch.int32), torch.tensor([[3, 1]], dtype=torch.int32)
    _compare(_append(cache, row.cuda()[:, 4:6], row.cuda()[:, 6:], cu, st, table), _want(cache, k, v, cu, st, table))


# ---------------------------------------------------------------- eviction

def _evict_case(B, width, seed, ties=False):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, width * 64 + 1, B).astype(np.int32)
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    w = rng.standard_exponential((B, width)).astype(np.float32)
    if ties:
        w = np.floor(w * 2).astype(np.float32)
    return lens, table, w


def _check_evict(lens, table, w, budget, sink, recent, in_place=False):
    a = _attn()
    want = ref.evict(lens, table, w, budget, sink, recent)
    dev = [torch.from_numpy(x.copy()).cuda() for x in (lens, table, w)]
    r = a.evict(*dev, budget, sink, recent, in_place=in_place)
    for got, ref_, what in zip(r, want, ("lens", "table", "weight", "freed", "count")):
        assert np.array_equal(got.cpu().numpy(), ref_, equal_nan=what == "weight"), what
    if in_place:
        assert r.block_table.data_ptr() == dev[1].data_ptr()
    else:
        assert np.array_equal(dev[1].cpu().numpy(), table)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,width,budget,sink,recent", [
    (1, 1, 1, 0, 1), (3, 8, 3, 1, 2), (5, 33, 10, 0, 1), (4, 64, 64, 2, 4), (3, 511, 100, 1, 1), (3, 512, 2, 1, 1),
    (2, 1100, 700, 3, 8), (2, 2049, 9, 4, 5),
])
def test_evict_matches_definition(B, width, budget, sink, recent, in_place):
    for ties in (False, True):
        _check_evict(*_evict_case(B, width, width + ties, ties), budget, sink, recent, in_place)


def test_evict_orders_special_weights():
    """NaN weighs least, then -inf; -0 equals 0; infinities stay."""
    w = np.array([[1, np.nan, 0.0, -0.0, np.inf, -np.inf, 2, np.nan, 0.0, 5, 5, 5]], np.float32)
    table = np.arange(100, 112, dtype=np.int32)[None]
    for budget in range(2, 12):
        _check_evict(np.array([12 * 64 - 3], np.int32), table, w, budget, 1, 1)


def test_evict_leaves_rows_that_are_too_short():
    a = _attn()
    lens, table, w = _evict_case(2, 6, 1)
    lens[:] = [7 * 64, 6 * 64]
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = a.evict(*(torch.from_numpy(x).cuda() for x in (lens, table, w)), 3, 1, 1, err_flag=flag)
    assert flag.item() == a.KDA_DEVERR_PAGE
    assert r.freed_count.tolist() == [0, 3] and r.seq_lens.tolist() == [7 * 64, 3 * 64]
    assert np.array_equal(r.block_table[0].cpu().numpy(), table[0])


def test_binding_refuses():
    a = _attn()
    lens, table, w = (torch.from_numpy(x).cuda() for x in _evict_case(2, 6, 1))
    for budget, sink, recent in ((2, 2, 1), (3, 1, 0), (3, -1, 1), (0, 0, 1)):
        with pytest.raises(a.KdaError):
            a.evict(lens, table, w, budget, sink, recent)
    with pytest.raises(ValueError):
        a.evict(lens, table, w.double(), 3)
    c = a.alloc_cache(2, 2, 64)
    k = torch.zeros((3, 2, 64), device="cuda")
    cu, st = cu_of([3]).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    t = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        a.append(c, k[:, :1], k[:, :1], cu, st, t)
    with pytest.raises(ValueError):
        a.append(c._replace(k_pages=c.k_pages.view(torch.uint8)), k, k, cu, st, t)
    with pytest.raises(ValueError):
        a.append(c, k, k, cu, st.long(), t)
