"""Attention over the 8-bit paged cache against its fp64 definition: window
lengths, head groups, ragged lengths, page weights, stale and non-finite
bytes, pages outside the cache, refusals."""
import numpy as np
import pytest
import torch

from attn_testutil import DT, bounds, check, gen, make_cache, np64, randn, to_device
from oracle import attention as ref

pytestmark = pytest.mark.gpu


def _attn():
    from gated_delta_rule_decode_gb300 import attn
    return attn


def _setup(lens, D, hq, hkv, d, dtype, seed, spread=1.0):
    g = gen(seed)
    B = len(lens)
    width = max(1, max(-(-x // 64) for x in lens) + 1)
    held = sum(-(-x // 64) for x in lens)
    cache = make_cache(g, max(held, 1), hkv, d, spread)
    perm = torch.randperm(max(held, 1), generator=g).tolist()
    table = torch.full((B, width), -7, dtype=torch.int32)  # entries past the end are never read
    for n, x in enumerate(lens):
        for c in range(-(-x // 64)):
            table[n, c] = perm.pop()
    q = (2 * randn(g, B, D, hq, d)).to(DT[dtype])
    return q, cache, torch.tensor(lens, dtype=torch.int32), table


def _run(q, cache, lens, table, **kw):
    return _attn().decode(q.cuda(), to_device(cache), lens.cuda(), table.cuda(), return_lse=True, **kw)


def _want(q, cache, lens, table, scale=None):
    kp, vp, ks, vs = (x.numpy() for x in cache)
    return ref.decode(np64(q), kp, vp, ks.astype(np.float64), vs.astype(np.float64), lens.numpy(), table.numpy(), scale)


def _check(q, cache, lens, table, got, scale=None, weight_in=None):
    o, l, a, m, mass = _want(q, cache, lens, table, scale)
    to, tl = bounds(o, a, m, q.shape[3], q.dtype)
    check(got[0], o, to, "out")
    check(got[1], l, tl, "lse")
    if len(got) > 2:
        base = 0 if weight_in is None else np64(weight_in)
        score = (q.shape[3] + 8) * 2.0 ** -23 * m.reshape(len(lens), -1).max(1)
        check(got[2], base + mass, (base + mass) * (4 * score[:, None] + 2.0 ** -17) + 1e-30, "weight")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens,D,hq,hkv", [
    ([1], 1, 1, 1),
    ([0, 1, 63, 64, 65], 1, 4, 2),
    ([200, 3, 129], 1, 8, 1),
    ([100, 64], 1, 40, 2),        # 20 rows: two row tiles
    ([7, 130, 3, 0], 4, 8, 2),    # windows longer than the sequence: rows that see nothing
    ([70, 64, 66], 7, 16, 2),     # 56 rows
    ([90], 16, 6, 1),             # 96 rows: two row blocks
    ([65, 10], 2, 3, 3),
])
def test_decode_matches_definition(lens, D, hq, hkv, d, dtype):
    s = _setup(lens, D, hq, hkv, d, dtype, seed=d + D)
    _check(*s, _run(*s, return_weight=True))


@pytest.mark.parametrize("dtype,D,hq,hkv", [("bf16", 1, 8, 2), ("f32", 1, 4, 2), ("bf16", 7, 8, 1)])
def test_long_contexts_are_split_and_joined(dtype, D, hq, hkv):
    """Contexts of many pages: cut over workers, ragged."""
    s = _setup([5000, 64, 2500, 0, 129], D, hq, hkv, 128, dtype, seed=2)
    win = torch.rand((5, s[3].shape[1]), generator=gen(1))
    _check(*s, _run(*s, weight_in=win.cuda()), weight_in=win)


def test_many_short_sequences():
    lens = [(7 * i) % 150 for i in range(300)]
    s = _setup(lens, 1, 4, 2, 64, "bf16", seed=5)
    _check(*s, _run(*s, return_weight=True))


@pytest.mark.parametrize("dtype,d,B,D,hq,hkv,longest", [
    ("bf16", 128, 130, 1, 8, 4, 700),   # rows of up to 12 pages, 520 items: none is cut
    ("f32", 64, 130, 4, 8, 4, 700),
    ("bf16", 32, 130, 8, 12, 4, 500),   # 24 rows: two row tiles
    ("bf16", 128, 17, 7, 32, 4, 900),   # 56 rows, 68 items
    ("bf16", 64, 9, 16, 72, 4, 600),    # 288 rows: three row blocks
    ("bf16", 128, 3, 7, 16, 2, 63),     # tables of one page
    ("f32", 32, 3, 1, 2, 1, 63),
])
def test_short_rows_of_the_table_are_not_cut(dtype, d, B, D, hq, hkv, longest):
    lens = [0, 1, longest] + [(37 * i) % (longest + 1) for i in range(B - 3)]
    q, cache, n, table = _setup(lens, D, hq, hkv, d, dtype, seed=B + D)
    if longest < 64:
        table = table[:, :1].contiguous()
    s = q, cache, n, table
    got = _run(*s, return_weight=True)
    _check(*s, got)
    plain = _run(*s)  # without weights nothing follows the kernel
    assert torch.equal(plain[0], got[0]) and torch.equal(plain[1], got[1])


def test_scales_far_apart_between_pages():
    """Pages whose scales differ by many powers of two, in both orders."""
    for dtype in ("bf16", "f32"):
        s = _setup([400, 640], 1, 4, 1, 64, dtype, seed=7, spread=6.0)
        q = s[0] * 1e-3
        _check(q, *s[1:], _run(q, *s[1:]))


def test_scale_argument_and_tiny_queries():
    for dtype, mul, scale in (("bf16", 1.0, 0.3), ("bf16", 1e-30, None), ("f32", 1e-30, None), ("bf16", 0.0, None)):
        s = _setup([150], 2, 4, 2, 64, dtype, seed=8)
        q = s[0] * mul
        _check(q, *s[1:], _run(q, *s[1:], scale=scale), scale)


@pytest.mark.parametrize("D", [1, 3])
def test_bytes_past_the_end_have_no_influence(D):
    """NaN bytes in the unused places of a sequence's last page."""
    q, cache, lens, table = _setup([70, 5], D, 8, 2, 64, "bf16", seed=3)
    want = _run(q, cache, lens, table, return_weight=True)
    kp, vp, ks, vs = (x.clone() for x in cache)
    for n, x in enumerate(lens.tolist()):
        page = int(table[n, (x - 1) // 64])
        kp[page, :, x % 64:] = 0x7f
        vp[page, :, :, x % 64:] = 0xff
    got = _run(q, (kp, vp, ks, vs), lens, table, return_weight=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_nan_in_a_window_reaches_only_the_rows_that_see_it():
    q, cache, lens, table = _setup([130], 4, 4, 2, 64, "bf16", seed=3)
    clean = _run(q, cache, lens, table)
    kp, vp, ks, vs = (x.clone() for x in cache)
    page = int(table[0, 2])  # positions 128, 129: window rows 2 and 3
    vp[page, 1, 9, 0] = 0x7f  # value channel 9 of position 128, kv head 1
    got = _run(q, (kp, vp, ks, vs), lens, table)
    assert torch.equal(got[0][0, :2], clean[0][0, :2])
    assert torch.isnan(got[0][0, 2:, 2:, 9]).all()
    got[0][0, 2:, 2:, 9] = clean[0][0, 2:, 2:, 9]
    assert torch.equal(got[0], clean[0])
    kp[page, 0, 1] = 0x7f     # key of position 129, kv head 0: row 3 only
    got = _run(q, (kp, cache[1], ks, vs), lens, table)
    assert torch.equal(got[0][0, :3], clean[0][0, :3])
    assert torch.isnan(got[0][0, 3, :2]).all() and torch.equal(got[0][0, 3, 2:], clean[0][0, 3, 2:])


def test_pages_outside_the_cache_count_as_unseen():
    a = _attn()
    q, cache, lens, table = _setup([300, 64], 1, 4, 2, 64, "bf16", seed=6)
    for bad in (-1, 1 << 30, cache[0].shape[0]):
        t = table.clone()
        t[0, 2] = bad
        t[1, 0] = bad  # the second sequence is left with nothing
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _run(q, cache, lens, t, return_weight=True, err_flag=flag)
        assert flag.item() == a.KDA_DEVERR_PAGE
        _check(q, cache, lens, t, got)
    # a sequence longer than its row
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = table[:, :3].contiguous()
    got = _run(q, cache, lens, t, err_flag=flag)
    assert flag.item() == a.KDA_DEVERR_PAGE
    _check(q, cache, lens, t, got)


def test_stream_strides_and_repeats():
    """Rows of a fused projection, another stream, three times: the same bits."""
    a = _attn()
    q, cache, lens, table = _setup([500, 77, 1000], 2, 8, 2, 128, "bf16", seed=4)
    c = to_device(cache)
    dev = (lens.cuda(), table.cuda())
    want = a.decode(q.cuda(), c, *dev, return_lse=True, return_weight=True)
    row = torch.cat([q.reshape(6, 8, 128), torch.zeros(6, 4, 128, dtype=q.dtype)], 1).cuda().view(3, 2, 12, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = a.decode(row[:, :, :8], c, *dev, return_lse=True, return_weight=True, stream=s)
        s.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_weight_accumulates_in_place():
    a = _attn()
    q, cache, lens, table = _setup([130, 20], 1, 4, 2, 64, "bf16", seed=4)
    c = to_device(cache)
    w = torch.ones(table.shape, device="cuda")
    one = a.decode(q.cuda(), c, lens.cuda(), table.cuda(), return_weight=True)[1]
    a.decode(q.cuda(), c, lens.cuda(), table.cuda(), weight_in=w, weight_out=w)
    assert torch.equal(w, 1 + one)
    # every row gives its pages one in all
    assert torch.allclose(one.sum(1), torch.full((2,), 4.0, device="cuda"), rtol=1e-5)


def test_append_then_decode_equals_attention_over_the_stored_values():
    """The two sides of the cache together: what append stores is what decode reads."""
    a = _attn()
    g = gen(12)
    heads, d = 2, 64
    k, v = randn(g, 150, heads, d).bfloat16(), randn(g, 150, heads, d).bfloat16()
    c = a.alloc_cache(3, heads, d)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32).cuda()
    for lo, hi in ((0, 100), (100, 101), (101, 150)):
        a.append(c, k[lo:hi].cuda(), v[lo:hi].cuda(), torch.tensor([0, hi - lo], dtype=torch.int32).cuda(),
                 torch.tensor([lo], dtype=torch.int32).cuda(), table)
    q = randn(g, 1, 1, 4, d).bfloat16()
    lens = torch.tensor([150], dtype=torch.int32)
    got = a.decode(q.cuda(), c, lens.cuda(), table, return_lse=True)
    host = (c.k_pages.view(torch.uint8).cpu(), c.v_pages.view(torch.uint8).cpu(), c.k_scale.cpu(), c.v_scale.cpu())
    _check(q, host, lens, table.cpu(), got)
    # and the stored values are the tokens to e4m3's precision
    o, _, ab, _, = ref.prompt(np.concatenate([np.zeros((149, 4, d)), np64(q)[0]]), np64(k), np64(v), [0, 150])
    err = np.abs(np64(got[0])[0, 0] - o[-1])
    assert err.max() < 0.1 * ab[-1].max()


def test_binding_refuses():
    a = _attn()
    q, cache, lens, table = _setup([70], 1, 4, 2, 64, "bf16", seed=1)
    c, q, lens, table = to_device(cache), q.cuda(), lens.cuda(), table.cuda()
    with pytest.raises(ValueError):
        a.decode(q, c, lens.long(), table)
    with pytest.raises(ValueError):
        a.decode(q, c._replace(v_pages=c.k_pages[:, :, :32]), lens, table)
    with pytest.raises(ValueError):
        a.decode(q, c, lens, table, weight_in=torch.zeros(3, device="cuda"))
    with pytest.raises(a.KdaError):
        a.decode(q[:, :, :3].contiguous(), c, lens, table)
    with pytest.raises(a.KdaError):
        a.decode(q, c, lens, table, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(a.KdaError):
        a.decode(q.expand(1, 17, 4, 64).contiguous(), c, lens, table)
