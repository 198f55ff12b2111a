"""Attention of batches that share prefixes against the fp64 definition over the
whole sequences (the shared pages are named by every row of the group)."""
import pytest
import torch

from attn_long_testutil import bounds, query_terms
from attn_testutil import check, gen, make_cache, np64, randn, to_device
from oracle import attention as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _attn():
    from gated_delta_rule_decode_gb300 import attn
    return attn


def _case(g, groups, hkv, d, width=0, spread=1.0):
    """groups: (shared pages, lengths in all) each -> cache, lens, table, group_start, shared_pages."""
    start, shared, lens, rows = [0], [], [], []
    need = sum(s for s, _ in groups) + sum(max(0, -(-n // 64) - s) for s, ls in groups for n in ls) + 1
    free = torch.randperm(need, generator=g).tolist()
    width = max([width] + [-(-n // 64) for _, ls in groups for n in ls] + [s for s, _ in groups])
    for s, ls in groups:
        mine = [free.pop() for _ in range(s)]
        for n in ls:
            held = -(-n // 64)
            row = mine[:held] + [free.pop() for _ in range(max(0, held - s))]
            if len(lens) == start[-1]:  # the group's first row names the whole prefix
                row = mine + row[s:]
            rows.append(row + [-1] * (width - len(row)))
            lens.append(n)
        shared.append(s)
        start.append(len(lens))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return make_cache(g, need, hkv, d, spread), i32(lens), i32(rows).view(len(lens), width), i32(start), i32(shared)


def _run(case, q, **kw):
    cache, lens, table, start, shared = case
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _attn().decode_shared(q.cuda(), to_device(cache), lens.cuda(), table.cuda(), start.cuda(), shared.cuda(),
                                     return_lse=True, err_flag=flag, **kw)
    return out, lse, flag.item()


def _want(case, q, dtype, lens=None):
    k, v, ks, vs = case[0]
    lens = case[1].numpy() if lens is None else lens
    out, lse, absout, mag, _ = ref.decode(np64(q), k.numpy(), v.numpy(), np64(ks), np64(vs), lens, case[2].numpy())
    return (out, lse) + bounds(out, absout, mag, q.shape[-1], dtype, _terms(case, q, dtype, lens))


def _terms(case, q, dtype, lens, scale=None):
    if dtype != BF or q.shape[-1] < 64:
        return 0.0
    return query_terms(np64(q), case[0][0].numpy(), np64(case[0][2]), lens, case[2].numpy(), scale)


def _compare(case, q, dtype):
    out, lse, flag = _run(case, q)
    want, want_lse, tol, tol_lse = _want(case, q, dtype)
    assert flag == 0
    check(out, want, tol, "out")
    check(lse, want_lse, tol_lse, "lse")


GROUPS = [
    [(3, [300, 200, 193])],                                     # one group
    [(2, [128 + 1, 128 + 70]), (0, [65, 0, 1]), (1, [64 + 9])],  # none shared; a padded sequence; a group of one
    [(4, [300, 17, 0, 256, 257, 64, 400])],                     # sequences that end inside the prefix, or with it
    [(5, [])] + [(1, [100])] * 2 + [(0, [])] + [(2, [200] * 9)],  # empty groups
]


@pytest.mark.parametrize("groups", range(len(GROUPS)))
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,hq,hkv,d", [(1, 4, 2, 64), (1, 8, 1, 128), (3, 6, 2, 32), (7, 16, 2, 128), (4, 12, 1, 64)])
def test_matches_the_definition(groups, dtype, D, hq, hkv, d):
    g = gen(groups * 100 + D)
    case = _case(g, GROUPS[groups], hkv, d)
    _compare(case, (2 * randn(g, case[1].shape[0], D, hq, d)).to(dtype), dtype)


@pytest.mark.parametrize("dtype,D,hq,hkv,d", [(BF, 1, 40, 1, 128), (BF, 2, 128, 1, 64), (F32, 1, 128, 1, 32), (BF, 16, 24, 1, 128),
                                              (F32, 16, 20, 2, 64), (BF, 1, 67, 1, 128), (BF, 5, 5, 5, 128)])
def test_rows_that_do_not_fill_chunks(dtype, D, hq, hkv, d):
    g = gen(hq)
    case = _case(g, [(3, [260, 400, 250, 300, 193 + D]), (1, [90, 100])], hkv, d)
    _compare(case, (2 * randn(g, 7, D, hq, d)).to(dtype), dtype)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_long_rows_of_the_table(dtype, d):
    """More than 16 pages: items are cut between workers, and parts joined."""
    g = gen(7)
    case = _case(g, [(40, [40 * 64 + 5, 40 * 64 + 900]), (25, [25 * 64 + 64, 25 * 64 + 1, 1700, 3])], 2, d, width=60)
    _compare(case, (2 * randn(g, 6, 2, 12, d)).to(dtype), dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_and_pages(d):
    """Chunks of 128 rows and more, several of a group, each cut between many workers."""
    g = gen(8)
    case = _case(g, [(70, [70 * 64 + 10 * i + 4 for i in range(11)])], 1, d)
    _compare(case, (2 * randn(g, 11, 4, 8, d)).bfloat16(), BF)


def test_scales_that_differ_widely():
    g = gen(9)
    for dtype in (BF, F32):
        case = _case(g, [(20, [1400, 1300, 1290] * 3)], 2, 64, spread=8.0)
        _compare(case, (0.01 * randn(g, 9, 2, 10, 64)).to(dtype), dtype)


@pytest.mark.parametrize("D", [1, 6])
def test_masked_places_have_no_influence(D):
    """NaN bytes past a sequence's end, in the pages of others, and NaN values that later rows alone see."""
    g = gen(10)
    case = _case(g, [(18, [18 * 64 + 30, 18 * 64 + 75, 0])], 1, 128)
    q = randn(g, 3, D, 8, 128).bfloat16()
    k, v, _, _ = case[0]
    for n, length in enumerate(case[1].tolist()):
        if length:
            page = int(case[2][n, length // 64])
            k[page, :, length % 64:], v[page, :, :, length % 64:] = 0x7f, 0xff
    _compare(case, q, BF)
    page = int(case[2][1, 19])
    v[page, :, 5, 75 - 64 - 1] = 0x7f  # the last token's value, channel 5
    out, _, flag = _run(case, q)
    want, _, tol, _ = _want(case, q, BF)
    assert flag == 0 and torch.isnan(out[1, D - 1, :, 5]).all() and int(torch.isnan(out).sum()) == 8
    check(out, want, tol, "out")


def test_pages_that_are_not_there():
    g = gen(11)
    for dtype in (BF, F32):
        case = _case(g, [(20, [1300, 1281]), (2, [200])], 2, 64)
        case[2][0, 3], case[2][1, 3], case[2][2, 3] = 1 << 20, 1 << 20, -7
        q = randn(g, 3, 3, 8, 64).to(dtype)
        out, lse, flag = _run(case, q)
        want, want_lse, tol, tol_lse = _want(case, q, dtype)
        assert flag == _attn().KDA_DEVERR_PAGE
        check(out, want, tol, "out")
        check(lse, want_lse, tol_lse, "lse")


def test_sequences_of_no_group_and_rows_that_are_too_short():
    g = gen(12)
    case = list(_case(g, [(0, [150]), (2, [170, 180]), (0, [70, 900])], 2, 64))
    q = randn(g, 5, 1, 4, 64).bfloat16()
    want, want_lse, tol, tol_lse = _want(case, q, BF)
    case[3], case[4] = torch.tensor([1, 3], dtype=torch.int32), torch.tensor([2], dtype=torch.int32)
    out, lse, flag = _run(case, q)
    assert flag == 0
    check(out, want, tol, "out")
    check(lse, want_lse, tol_lse, "lse")
    # no groups at all; a length past the row's end counts as the row's
    case[3], case[4] = torch.tensor([0], dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    case[1] = case[1].clone()
    case[1][4] = 15 * 64 + 40
    out, lse, flag = _run(case, q)
    want, _, tol, _ = _want(case, q, BF)
    assert flag == _attn().KDA_DEVERR_PAGE
    check(out, want, tol, "out")


def test_wrong_groups_are_flagged():
    g, a = gen(13), _attn()
    from gated_delta_rule_decode_gb300 import kda
    base = _case(g, [(1, [150, 100]), (1, [170, 180])], 2, 64)
    q = randn(g, 4, 1, 4, 64).bfloat16()
    for start in ([0, 3, 2], [-1, 2, 4], [0, 2, 5], [1 << 30, 2, 4]):
        case = base[:3] + (torch.tensor(start, dtype=torch.int32), base[4])
        assert _run(case, q)[2] & kda.KDA_DEVERR_SEQLENS
    for shared in ([-1, 1], [1, 100]):
        case = base[:4] + (torch.tensor(shared, dtype=torch.int32),)
        assert _run(case, q)[2] & a.KDA_DEVERR_PAGE
    out, _, flag = _run(base, q)
    assert flag == 0


def test_repeats_and_is_captured():
    g, a = gen(14), _attn()
    case = _case(g, [(30, [2000 + 40 * i for i in range(6)])], 2, 128)
    q = randn(g, 6, 1, 16, 128).bfloat16().cuda()
    c, lens, table, start, shared = to_device(case[0]), *[x.cuda() for x in case[1:]]
    want = a.decode_shared(q, c, lens, table, start, shared, return_lse=True)
    again = a.decode_shared(q, c, lens, table, start, shared, return_lse=True)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = a.decode_shared(q, c, lens, table, start, shared, return_lse=True, stream=s)
    s.synchronize()
    assert torch.equal(want[0], other[0]) and torch.equal(want[1], other[1])
    # two graphs with workspaces of their own, replayed in turn with other lengths
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = a.decode_shared(q, c, lens, table, start, shared)
        graphs.append((graph, got))
    lens.sub_(33)
    want = a.decode_shared(q, c, lens, table, start, shared)
    for graph, got in graphs + graphs[::-1]:
        graph.replay()
    for graph, got in graphs:
        assert torch.equal(got, want)


def test_given_results_scale_and_workspace():
    g, a = gen(15), _attn()
    case = _case(g, [(3, [300, 200])], 2, 64)
    q = randn(g, 2, 2, 8, 64)
    c, lens, table, start, shared = to_device(case[0]), *[x.cuda() for x in case[1:]]
    ws = torch.empty(a.decode_shared_workspace_bytes(8, 2, 64, 1, 2, 2, table.shape[1], 1), dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)
    out, lse = torch.empty(2, 2, 8, 64, dtype=BF, device="cuda"), torch.empty(2, 2, 8, device="cuda")
    fused = torch.cat([q, q], 2).bfloat16().cuda()
    got = a.decode_shared(fused[:, :, :8], c, lens, table, start, shared, out, lse=lse, workspace=ws, scale=0.3)
    assert got is out
    k, v, ks, vs = case[0]
    want, want_lse, absout, mag, _ = ref.decode(np64(q.bfloat16()), k.numpy(), v.numpy(), np64(ks), np64(vs), case[1].numpy(),
                                                case[2].numpy(), scale=0.3)
    tol, tol_lse = bounds(want, absout, mag, 64, BF, _terms(case, q.bfloat16(), BF, case[1].numpy(), 0.3))
    check(out, want, tol, "out")
    check(lse, want_lse, tol_lse, "lse")
    assert a.decode_shared(fused[:0, :, :8], c, lens[:0], table[:0], start[:1] * 0, shared[:0]).shape == (0, 2, 8, 64)
    with pytest.raises(a.KdaError):
        a.decode_shared(fused[:, :, :8], c, lens, table, start, shared, workspace=ws[:-256].clone())


def test_queries_of_all_sizes():
    """Elements far below the row's largest, subnormal and huge rows, and infinities and NaN, which are the row's alone."""
    g = gen(16)
    case = _case(g, [(20, [1400, 1290, 1300])], 1, 128)
    q = randn(g, 3, 2, 10, 128) * torch.exp2(torch.randint(-20, 1, (3, 2, 10, 128), generator=g).float())
    q[0, 0, 1] *= 2.0 ** -110
    q[1, 0, 2] = 0
    q[1, 1, 3] *= 2.0 ** 60
    q = q.bfloat16()
    case[0][2].mul_(0).add_(2.0 ** -8)  # (one scale, so that the large row's weights are not all on one key by its page's scale)
    _compare(case, q, BF)
    bad = q.clone()
    bad[0, 1, 4, 7], bad[2, 0, 5, 9] = float("nan"), float("-inf")
    out, _, flag = _run(case, bad)
    good, _, _ = _run(case, q)
    rows = torch.zeros(3, 2, 10, dtype=torch.bool)
    rows[0, 1, 4] = rows[2, 0, 5] = True
    assert flag == 0 and torch.isnan(out[rows]).all() and torch.equal(out[~rows], good[~rows])


@pytest.mark.parametrize("dtype,D,d", [(BF, 1, 128), (BF, 7, 128), (BF, 7, 64), (F32, 1, 64)])
def test_queries_that_are_no_numbers_stay_in_their_rows(dtype, D, d):
    g = gen(33)
    case = _case(g, [(3, [500, 700, 260]), (0, [130])], 2, d)
    q = randn(g, 4, D, 8, d).to(dtype)
    want, want_lse, _ = _run(case, q)
    odd = q.clone()
    odd[0, 0, 1, 3] = float("nan")
    odd[2, D - 1, 6, 0] = float("inf")
    odd[3, 0, 0, d - 1] = float("-inf")
    out, lse, flag = _run(case, odd)
    assert flag == 0
    rows = torch.zeros(4, D, 8, dtype=torch.bool, device="cuda")
    rows[0, 0, 1] = rows[2, D - 1, 6] = rows[3, 0, 0] = True
    assert out[rows].isnan().all()
    assert torch.equal(out[~rows], want[~rows]) and torch.equal(lse[~rows], want_lse[~rows])


def _serve_step(a, c, table, held, rot, w, row, cu, one, start, shared):
    """A token of each sequence: norm and rotation, into the cache, attention; (q, lengths, out, lse)."""
    q, k, v = row[:, :8], row[:, 8:10], row[:, 10:]
    q, k = a.norm_rotate(q, k, held, rot, q_weight=w, k_weight=w)
    a.append(c, k, v, cu, held, table)
    now = held + one
    return (q, now) + a.decode_shared(q[:, None], c, now, table, start, shared, return_lse=True)


def test_a_course_with_a_system_prompt():
    """A prefix goes into the cache once; three sequences of a group and one by itself go on from there."""
    a, g = _attn(), gen(51)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    c = a.alloc_cache(40, 2, 128)
    pages = torch.randperm(40, generator=g).int()
    table = torch.stack([torch.cat([pages[:4], pages[4 + 3 * n:7 + 3 * n]]) for n in range(3)] + [pages[20:27]]).cuda()
    rot, w = a.rotary(a.rotary_frequencies(128)), (1 + 0.1 * randn(g, 128)).cuda()
    start, shared = i32([0, 3, 4]), i32([4, 0])
    # the prefix, through the first sequence's row, and the other sequence's prompt
    row = randn(g, 256 + 70, 12, 128).bfloat16().cuda()
    pos = torch.cat([torch.arange(256), torch.arange(70)]).int().cuda()
    _, k = a.norm_rotate(row[:, :8], row[:, 8:10], pos, rot, q_weight=w, k_weight=w)
    a.append(c, k, row[:, 10:], i32([0, 256, 326]), i32([0, 0]), table[[0, 3]].contiguous())
    # what the sequences of the group ask, behind the prefix
    row = randn(g, 100 + 1 + 64, 12, 128).bfloat16().cuda()
    pos = torch.cat([256 + torch.arange(n) for n in (100, 1, 64)]).int().cuda()
    _, k = a.norm_rotate(row[:, :8], row[:, 8:10], pos, rot, q_weight=w, k_weight=w)
    a.append(c, k, row[:, 10:], i32([0, 100, 101, 165]), i32([256] * 3), table[:3].contiguous())
    held, one, cu = i32([356, 257, 320, 70]), i32([1] * 4), i32([0, 1, 2, 3, 4])
    row = randn(g, 4, 12, 128).bfloat16().cuda()
    saved = [x.clone() for x in c]
    q, now, out, lse = _serve_step(a, c, table, held, rot, w, row, cu, one, start, shared)
    kp, vp = (x.view(torch.uint8).cpu() for x in (c.k_pages, c.v_pages))
    case = ((kp, vp, c.k_scale.cpu(), c.v_scale.cpu()), now.cpu(), table.cpu(), None, None)
    want, want_lse, tol, tol_lse = _want(case, q[:, None], BF)
    check(out, want, tol, "out")
    check(lse, want_lse, tol_lse, "lse")
    # the same step captured, replayed from the same state
    for x, y in zip(c, saved):
        x.view(torch.uint8).copy_(y.view(torch.uint8)) if x.element_size() == 1 else x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _serve_step(a, c, table, held, rot, w, row, cu, one, start, shared)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[2], out) and torch.equal(got[3], lse)
