"""Key summaries, page selection and attention over the selected pages.  Summaries
and selections are whole numbers and equal the definition's."""
import numpy as np
import pytest
import torch

from attn_long_testutil import bounds
from attn_testutil import check, cu_of, gen, make_cache, np64, randn, to_device
from oracle import attention as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _attn():
    from gated_delta_rule_decode_gb300 import attn
    return attn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


# ---------------------------------------------------------------- summaries

def _summary_matches(c, cache, lens, start, table, expect=0):
    """Runs on marked summaries and compares all of them with the definition's."""
    a = _attn()
    N, Hkv, _, d = cache[0].shape
    s = a.alloc_summary(c)
    s.bounds.fill_(77)
    s.unit.fill_(3.0)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    a.summarise(c, s, cu_of(lens).cuda(), sum(lens), _i32(start).cuda(), table.cuda(), err_flag=flag)
    assert flag.item() == expect
    b, u = ref.summarise(cache[0].numpy(), np64(cache[2]), np.full((N, Hkv, 2, d), 77), np.full((N, Hkv), 3.0),
                         cu_of(lens).tolist(), start, table.tolist())
    assert (s.unit.cpu().double().numpy() == u).all()
    assert (s.bounds.cpu().numpy() == b).all()
    return s


@pytest.mark.parametrize("d,hkv", [(32, 1), (64, 3), (128, 2), (128, 11)])
@pytest.mark.parametrize("lens,start", [([1, 1, 1], [0, 63, 130]), ([200, 0, 64, 5], [5, 61, 64, 60]), ([128], [0]), ([1], [191])])
def test_summary_matches_the_definition(d, hkv, lens, start):
    g = gen(d + sum(lens))
    cache = make_cache(g, 32, hkv, d, spread=4.0)
    table = torch.randperm(32, generator=g).int().view(4, 8)[:len(lens)].contiguous()
    _summary_matches(to_device(cache), cache, lens, start, table)


def test_summary_of_odd_bytes():
    """NaN, negative zero, the largest and the smallest values; whole channels and whole pages of them."""
    g = gen(2)
    cache = make_cache(g, 6, 2, 64)
    k = cache[0]
    k[0] = torch.randint(0, 256, k[0].shape, generator=g, dtype=torch.uint8)  # NaN among them
    k[1], k[2], k[3], k[4] = 0x80, 0x7f, 0xfe, 0x01
    k[5] = 0
    k[5, :, 3] = 0xff
    cache[2][0], cache[2][3, 0], cache[2][4, 1] = 2.0 ** -126, 2.0 ** 120, 2.0 ** -126
    _summary_matches(to_device(cache), cache, [384], [0], torch.arange(6, dtype=torch.int32)[None])


def test_summary_errors():
    g, a = gen(3), _attn()
    cache = make_cache(g, 6, 2, 64)
    c = to_device(cache)
    _summary_matches(c, cache, [200], [0], _i32([[0, 9, 2, -1]]), a.KDA_DEVERR_PAGE)
    _summary_matches(c, cache, [200], [0], _i32([[0, 1]]), a.KDA_DEVERR_PAGE)
    _summary_matches(c, cache, [5, 5], [-3, 2], _i32([[0], [1]]))  # a negative start skips the sequence
    s = a.alloc_summary(c)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.k_scale[1, 0], c.k_scale[2, 1] = 3.0, 2.0 ** 126
    s.bounds.fill_(5)
    a.summarise(c, s, cu_of([192]).cuda(), 192, _i32([0]).cuda(), _i32([[0, 1, 2]]).cuda(), err_flag=flag)
    assert flag.item() == a.KDA_DEVERR_SCALE
    assert (s.bounds[1, 0] == 5).all() and (s.bounds[2, 1] == 5).all() and not (s.bounds[1, 1] == 5).all()
    from gated_delta_rule_decode_gb300 import kda
    flag.zero_()
    a.summarise(c, s, _i32([0, 9, 4]).cuda(), 9, _i32([0, 0]).cuda(), _i32([[0], [1]]).cuda(), err_flag=flag)
    assert flag.item() & kda.KDA_DEVERR_SEQLENS


def test_summary_follows_the_appends():
    """Prompts, then steps that raise scales: renewed after each append, the summaries are those of the whole cache."""
    g, a = gen(4), _attn()
    c = a.alloc_cache(12, 2, 64)
    s = a.alloc_summary(c)
    table = torch.randperm(12, generator=g).int().view(3, 4)
    held = torch.zeros(3, dtype=torch.int32)
    for lens, size in (([100, 64, 3], 1.0), ([1, 1, 1], 0.1), ([1, 1, 1], 30.0), ([7, 0, 70], 3.0)):
        k, v = (size * randn(g, sum(lens), 2, 64)).bfloat16().cuda(), randn(g, sum(lens), 2, 64).bfloat16().cuda()
        a.append(c, k, v, cu_of(lens).cuda(), held.cuda(), table.cuda())
        a.summarise(c, s, cu_of(lens).cuda(), sum(lens), held.cuda(), table.cuda())
        held += _i32(lens)
    b, u = ref.summarise(c.k_pages.view(torch.uint8).cpu().numpy(), np64(c.k_scale), np.zeros((12, 2, 2, 64)), np.ones((12, 2)),
                         cu_of(held.tolist()).tolist(), [0, 0, 0], table.tolist())
    assert (s.bounds.cpu().numpy() == b).all() and (s.unit.cpu().double().numpy() == u).all()


# ---------------------------------------------------------------- selection

def _random_summary(g, pages, hkv, d, coarse=False):
    hi, lo = (torch.randint(-127, 128, (pages, hkv, d), generator=g) for _ in range(2))
    if coarse:  # few values, so that scores repeat
        hi, lo = 100 * (hi > 0), -100 * (lo > 90)
    b = torch.stack([torch.maximum(hi, lo), torch.minimum(hi, lo)], 2).to(torch.int8)
    return b, torch.exp2(torch.randint(-3, 3, (pages, hkv), generator=g).float())


def _selects(q, bounds_, unit, lens, table, budget, sink, recent, expect=0):
    a = _attn()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = a.select(q.cuda(), a.KeySummary(bounds_.cuda(), unit.cuda()), lens.cuda(), table.cuda(), budget, sink, recent, err_flag=flag)
    assert flag.item() == expect
    l, t, i = ref.select(np64(q), bounds_.numpy(), np64(unit), lens.numpy(), table.numpy(), budget, sink, recent)
    assert (r.seq_lens.cpu().numpy() == l).all()
    assert (r.index.cpu().numpy() == i).all()
    assert (r.block_table.cpu().numpy() == t).all()
    return r


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,hq,hkv,D", [(32, 2, 1, 1), (64, 12, 2, 1), (128, 8, 2, 1), (128, 10, 2, 7), (64, 34, 2, 2), (32, 5, 5, 16)])
@pytest.mark.parametrize("budget,sink,recent", [(4, 1, 2), (3, 0, 3), (9, 2, 2), (40, 1, 2)])
def test_selection_matches_the_definition(dtype, d, hq, hkv, D, budget, sink, recent):
    g = gen(d + D + budget)
    lens = _i32([0, 1, 64 * 3, 64 * 4 + 1, 64 * 30 - 5, 64 * 30, 64 * 9])
    table = torch.randperm(7 * 30, generator=g).int().view(7, 30)
    b, u = _random_summary(g, 210, hkv, d)
    _selects((2 * randn(g, 7, D, hq, d)).to(dtype), b, u, lens, table, budget, sink, recent)


@pytest.mark.parametrize("P,budget", [(127, 20), (128, 20), (129, 64), (300, 7), (1000, 300), (1000, 999)])
def test_selection_of_long_rows(P, budget):
    g = gen(P)
    b, u = _random_summary(g, P, 2, 64)
    table = torch.randperm(P, generator=g).int().view(1, P)
    _selects(randn(g, 1, 1, 4, 64).bfloat16(), b, u, _i32([P * 64 - 9]), table, budget, 1, 2)


@pytest.mark.parametrize("P,budget", [(40, 6), (700, 100), (700, 690)])
def test_of_equal_scores_the_lower_index(P, budget):
    g = gen(P + 1)
    b, u = _random_summary(g, P, 1, 32, coarse=True)
    q = torch.zeros(2, 1, 1, 32)
    q[0, 0, 0, :3] = 1.0  # the second sequence's query is zero: all scores are
    table = torch.arange(P, dtype=torch.int32).flip(0).repeat(2, 1)
    for sink, recent in ((0, 1), (1, 2), (2, budget - 2)):
        _selects(q, b, u * 0 + 1, _i32([P * 64, P * 64 - 63]), table, budget, sink, recent)


def test_scores_of_both_signs_and_odd_queries():
    g = gen(6)
    b, u = _random_summary(g, 60, 2, 64)
    b[::2] = -b[::2].abs()  # some pages' scores are negative
    b[:, :, 0], b[:, :, 1] = torch.maximum(b[:, :, 0], b[:, :, 1]), torch.minimum(b[:, :, 0], b[:, :, 1])
    u[3], u[4] = 2.0 ** 126, 2.0 ** -126
    for dtype in (BF, F32):
        q = randn(g, 4, 2, 4, 64).to(dtype)
        q[0, 0, 0, 0], q[0, 1, 3, 5], q[1, 0, 1, 7] = float("inf"), float("-inf"), float("nan")
        q[2] *= 2.0 ** 100
        q[3] *= 2.0 ** -120
        q[1, 1, 2] = float("nan")
        _selects(q, b, u, _i32([50 * 64, 60 * 64, 60 * 64, 33 * 64]), torch.arange(60, dtype=torch.int32).repeat(4, 1), 12, 1, 2)


def test_units_at_their_borders():
    """Rows whose largest element is 127 units, or the next number."""
    g = gen(7)
    b, u = _random_summary(g, 50, 1, 32)
    q = 0.1 * randn(g, 4, 1, 1, 32)
    q[:, 0, 0, 3] = torch.tensor([127.0, 127.00001, -127 * 2.0 ** -5, 63.5])
    _selects(q, b, u, _i32([50 * 64] * 4), torch.arange(50, dtype=torch.int32).repeat(4, 1), 8, 0, 2)


def test_pages_that_cannot_be_scored_come_last():
    g, a = gen(8), _attn()
    b, u = _random_summary(g, 20, 1, 32)
    table = torch.arange(20, dtype=torch.int32)[None].clone()
    table[0, 4], table[0, 7] = -1, 20
    q = randn(g, 1, 1, 2, 32)
    r = _selects(q, b, u, _i32([20 * 64]), table, 6, 1, 2, a.KDA_DEVERR_PAGE)
    assert not {4, 7} & set(r.index[0, 0].tolist())
    r = _selects(q, b, u, _i32([20 * 64]), table, 19, 1, 2, a.KDA_DEVERR_PAGE)  # all but one of the two: the lower index
    assert 4 in r.index[0, 0].tolist() and 7 not in r.index[0, 0].tolist()
    u[3] = 1.5
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = a.select(q.cuda(), a.KeySummary(b.cuda(), u.cuda()), _i32([20 * 64]).cuda(), table.cuda().clamp(0, 19), 6, err_flag=flag)
    assert flag.item() == a.KDA_DEVERR_SCALE and 3 not in r.index[0, 0].tolist()
    # a sequence longer than its row ends with the row
    _selects(q, b, u * 0 + 1, _i32([25 * 64]), table.clamp(0, 19), 6, 1, 2, a.KDA_DEVERR_PAGE)


def test_no_pages_and_no_sequences():
    a, g = _attn(), gen(9)
    b, u = _random_summary(g, 4, 2, 64)
    s = a.KeySummary(b.cuda(), u.cuda())
    r = a.select(randn(g, 2, 1, 4, 64).cuda(), s, _i32([0, 0]).cuda(), torch.zeros(2, 0, dtype=torch.int32).cuda(), 5)
    assert r.seq_lens.tolist() == [0, 0] and (r.index == -1).all() and (r.block_table == -1).all()
    r = a.select(randn(g, 0, 1, 4, 64).cuda(), s, _i32([]).cuda(), torch.zeros(0, 7, dtype=torch.int32).cuda(), 5)
    assert r.block_table.shape == (0, 2, 5)


# ---------------------------------------------------------------- attention over the selected pages

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,hq,hkv,d", [(1, 4, 2, 64), (1, 8, 4, 128), (3, 6, 2, 32), (7, 16, 2, 128), (1, 40, 2, 64), (5, 12, 3, 128)])
@pytest.mark.parametrize("K", [5, 23])
def test_attention_matches_the_definition(dtype, D, hq, hkv, d, K):
    g, a = gen(D + hq + K), _attn()
    cache = make_cache(g, 4 * hkv * K, hkv, d, spread=3.0)
    table = torch.randperm(4 * hkv * K, generator=g).int().view(4, hkv, K)
    lens = _i32([K * 64 - 5, 0, 100, 64 * (K - 1) + 1])
    q = (2 * randn(g, 4, D, hq, d)).to(dtype)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = a.decode_selected(q.cuda(), to_device(cache), a.Selected(lens.cuda(), table.cuda(), None), return_lse=True,
                                 err_flag=flag)
    assert flag.item() == 0
    k, v, ks, vs = cache
    want, want_lse, absout, mag = ref.decode_selected(np64(q), k.numpy(), v.numpy(), np64(ks), np64(vs), lens.numpy(), table.numpy())
    tol, tol_lse = bounds(want, absout, mag, d, dtype)
    check(out, want, tol, "out")
    check(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("dtype,D,hq", [(BF, 1, 8), (BF, 7, 8), (F32, 2, 8)])
def test_all_pages_selected_is_the_whole_attention(dtype, D, hq):
    g, a = gen(11), _attn()
    c = to_device(make_cache(g, 60, 2, 128))
    table, lens = torch.randperm(60, generator=g).int().view(3, 20).cuda(), _i32([1280, 77, 900]).cuda()
    q = randn(g, 3, D, hq, 128).to(dtype).cuda()
    s = a.alloc_summary(c)
    a.summarise(c, s, cu_of(lens.tolist()).cuda(), int(lens.sum()), (lens * 0), table)
    r = a.select(q, s, lens, table, 20)
    assert torch.equal(r.seq_lens, lens)
    assert torch.equal(a.decode_selected(q, c, r), a.decode(q, c, lens, table))


def _course(a, g, c, s, table, held, w):
    """Prompts, then a step: norm and rotation, append, summaries, selection, attention; all as a serving loop calls them."""
    r = a.rotary(a.rotary_frequencies(64))
    lens = [1500, 700]
    row = randn(g, sum(lens), 10, 128).bfloat16().cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    cu = cu_of(lens).cuda()
    q, k = a.norm_rotate(row[:, :6], row[:, 6:8], pos, r, row[:, :6], row[:, 6:8], q_weight=w, k_weight=w)
    out = a.prefill(q, k, row[:, 8:], cu)
    a.append(c, k, row[:, 8:], cu, held, table)
    a.summarise(c, s, cu, sum(lens), held, table)
    held += _i32(lens).cuda()
    return r, out


def _step(a, c, s, table, held, w, r, row, cu, one, budget):
    q, k = a.norm_rotate(row[:, :6], row[:, 6:8], held, r, q_weight=w, k_weight=w)
    a.append(c, k, row[:, 8:], cu, held, table)
    a.summarise(c, s, cu, 2, held, table)
    now = held + one
    chosen = a.select(q[:, None], s, now, table, budget)
    return q, now, chosen, a.decode_selected(q[:, None], c, chosen)


def test_a_serving_course_and_its_captured_step():
    a, g = _attn(), gen(12)
    c = a.alloc_cache(60, 2, 128)
    s = a.alloc_summary(c)
    table = torch.randperm(60, generator=g).int().view(2, 30).cuda()
    held, one = torch.zeros(2, dtype=torch.int32).cuda(), torch.ones(2, dtype=torch.int32).cuda()
    w = (1 + 0.1 * randn(g, 128)).cuda()
    r, out = _course(a, g, c, s, table, held, w)
    assert torch.isfinite(out.float()).all()
    cu, budget = _i32([0, 1, 2]).cuda(), 12
    row = randn(g, 2, 10, 128).bfloat16().cuda()
    saved = [x.clone() for x in (*c, *s)]
    q, now, chosen, out = _step(a, c, s, table, held, w, r, row, cu, one, budget)
    kp, vp = (x.view(torch.uint8).cpu().numpy() for x in (c.k_pages, c.v_pages))
    l, t, i = ref.select(np64(q[:, None]), s.bounds.cpu().numpy(), np64(s.unit), now.cpu().numpy(), table.cpu().numpy(), budget, 1, 2)
    assert (chosen.index.cpu().numpy() == i).all() and (chosen.seq_lens.cpu().numpy() == l).all()
    want, _, absout, mag = ref.decode_selected(np64(q[:, None]), kp, vp, np64(c.k_scale), np64(c.v_scale), l, t)
    check(out, want, bounds(want, absout, mag, 128, BF)[0], "out")
    # the same step captured, replayed from the same state
    for x, y in zip((*c, *s), saved):
        x.view(torch.uint8).copy_(y.view(torch.uint8)) if x.element_size() == 1 else x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(a, c, s, table, held, w, r, row, cu, one, budget)
    graph.replay()
    assert torch.equal(got[3], out) and torch.equal(got[2].index, chosen.index)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    again = a.select(q[:, None], s, now, table, budget, stream=stream)
    there = a.decode_selected(q[:, None], c, again, stream=stream)
    stream.synchronize()
    assert torch.equal(there, out) and torch.equal(again.index, chosen.index)
