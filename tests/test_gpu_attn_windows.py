"""Cache attention of more than 16 rows per kv head (the tcgen05 kernel): stale
and non-finite bytes, pages outside the cache, tables too short, cut rows."""
import pytest
import torch

from test_gpu_attn_decode import _attn, _check, _run, _setup

pytestmark = pytest.mark.gpu

SHAPES = [(7, 16, 2, 64), (7, 16, 2, 128), (16, 24, 2, 128)]  # 56 rows, and 192: two blocks of rows


@pytest.mark.parametrize("D,hq,hkv,d", SHAPES)
def test_bytes_past_the_end_have_no_influence(D, hq, hkv, d):
    """Odd and even page counts: a tile's second page is there or not."""
    for lens in ([70, 5], [130, 64 * 3 - 1], [20, 200, 383]):
        q, cache, n, table = _setup(lens, D, hq, hkv, d, "bf16", seed=51)
        want = _run(q, cache, n, table, return_weight=True)
        kp, vp, ks, vs = (x.clone() for x in cache)
        for s, x in enumerate(lens):
            page = int(table[s, (x - 1) // 64])
            if x % 64:
                kp[page, :, x % 64:] = 0x7f
                vp[page, :, :, x % 64:] = 0xff
        got = _run(q, (kp, vp, ks, vs), n, table, return_weight=True)
        for a, b in zip(got, want):
            assert torch.equal(a, b), lens


@pytest.mark.parametrize("D,hq,hkv,d", SHAPES)
def test_nan_in_a_window_reaches_only_the_rows_that_see_it(D, hq, hkv, d):
    """In one item's window but not in those before and after it."""
    G = hq // hkv
    q, cache, n, table = _setup([130, 131, 67], D, hq, hkv, d, "bf16", seed=52)
    clean = _run(q, cache, n, table)
    kp, vp, ks, vs = (x.clone() for x in cache)
    at = 131 - D + 3                                 # rows 3 and later of sequence 1 see this position
    page, place = int(table[1, at // 64]), at % 64
    vp[page, 1, 9, place] = 0xff
    got = _run(q, (kp, vp, ks, vs), n, table)
    assert torch.isnan(got[0][1, 3:, G:, 9]).all()
    got[0][1, 3:, G:, 9] = clean[0][1, 3:, G:, 9]
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    kp[page, 0, place] = 0x7f                        # a key of the other kv head
    got = _run(q, (kp, cache[1], ks, vs), n, table)
    assert torch.isnan(got[0][1, 3:, :G]).all() and torch.isnan(got[1][1, 3:, :G]).all()
    got[0][1, 3:, :G], got[1][1, 3:, :G] = clean[0][1, 3:, :G], clean[1][1, 3:, :G]
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    vp[page, 1, 9, place] = 0x7f                     # a NaN that every row of sequence 0 sees, and one in a window
    vp[int(table[0, 0]), 0, 5, 3] = 0x7f
    got = _run(q, (cache[0], vp, ks, vs), n, table)
    assert torch.isnan(got[0][0, :, :G, 5]).all() and torch.isnan(got[0][1, 3:, G:, 9]).all()
    got[0][0, :, :G, 5], got[0][1, 3:, G:, 9] = clean[0][0, :, :G, 5], clean[0][1, 3:, G:, 9]
    assert torch.equal(got[0], clean[0])


@pytest.mark.parametrize("D,hq,hkv,d", SHAPES)
def test_pages_outside_the_cache_count_as_unseen(D, hq, hkv, d):
    a = _attn()
    q, cache, n, table = _setup([300, 190, 64], D, hq, hkv, d, "bf16", seed=53)
    for bad, places in ((-1, [(0, 2)]), (1 << 30, [(0, 3), (1, 1)]), (cache[0].shape[0], [(0, 4), (1, 0), (2, 0)])):
        t = table.clone()
        for s, c in places:  # either half of a tile, an item's last page, a whole item
            t[s, c] = bad
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _run(q, cache, n, t, return_weight=True, err_flag=flag)
        assert flag.item() == a.KDA_DEVERR_PAGE
        _check(q, cache, n, t, got)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = table[:, :3].contiguous()  # a row too short
    got = _run(q, cache, n, t, return_weight=True, err_flag=flag)
    assert flag.item() == a.KDA_DEVERR_PAGE
    _check(q, cache, n, t, got)


@pytest.mark.parametrize("D,hq,hkv,d", [(7, 16, 2, 128), (5, 8, 2, 64)])
def test_rows_cut_between_workers(D, hq, hkv, d):
    """More pages than workers, with stale bytes and a page outside the cache."""
    lens = [64 * 30 - 1, 3, 64 * 25 + 1, 0, 64 * 33, 700]
    q, cache, n, table = _setup(lens, D, hq, hkv, d, "bf16", seed=54)
    kp, vp, ks, vs = cache
    for s, x in enumerate(lens):
        if x % 64:
            page = int(table[s, (x - 1) // 64])
            kp[page, :, x % 64:] = 0xff
            vp[page, :, :, x % 64:] = 0x7f
    table[2, 11] = -1
    win = torch.rand(table.shape, generator=torch.Generator().manual_seed(1))
    got = _run(q, cache, n, table, weight_in=win.cuda())
    for s, x in enumerate(lens):  # the oracle reads every byte
        if x % 64:
            page = int(table[s, (x - 1) // 64])
            kp[page, :, x % 64:] = 0
            vp[page, :, :, x % 64:] = 0
    _check(q, cache, n, table, got, weight_in=win)


def test_scales_far_apart_between_pages():
    for lens in ([400, 640], [65, 64 * 9]):
        q, cache, n, table = _setup(lens, 7, 16, 4, 64, "bf16", seed=55, spread=6.0)
        q = q * 1e-3
        _check(q, cache, n, table, _run(q, cache, n, table, return_weight=True))
