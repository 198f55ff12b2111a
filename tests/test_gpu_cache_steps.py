"""Append of a few tokens per sequence (draft windows, mixed batches), byte for
byte, and packed batches of many sequences."""
import pytest
import torch

from attn_testutil import DT, cu_of, gen, make_cache, randn
from test_gpu_attn_prefill import _attn, _check as _check_prompt, _inputs
from test_gpu_cache import _append, _compare, _want

pytestmark = pytest.mark.gpu


def _case(lens, start, d, heads, dtype, seed, width=8):
    g = gen(seed)
    n, T = len(lens), sum(lens)
    cache = make_cache(g, n * width, heads, d)
    cache = (cache[0], cache[1], cache[2] / 4, cache[3] / 4)  # old scales that have to grow
    k, v = randn(g, T, heads, d).to(DT[dtype]), (100 * randn(g, T, heads, d)).to(DT[dtype])
    table = torch.randperm(n * width, generator=g).reshape(n, width).int()
    args = cache, k, v, cu_of(lens), torch.tensor(start, dtype=torch.int32), table
    _compare(_append(*args), _want(*args))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,heads", [(32, 3), (64, 2), (128, 5)])
@pytest.mark.parametrize("each", [2, 3, 4, 7, 8])
def test_windows(each, d, heads, dtype):
    """Windows that begin a page, end it and cross into the next."""
    start = [0, 1, 30, 57, 58, 59, 60, 61, 62, 63, 64, 121, 127]
    _case([each] * len(start), start, d, heads, dtype, seed=each + d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_chunk_among_single_tokens(dtype):
    for n in (40, 80):  # a mean above and below 4: both kernels
        lens = [1] * n
        lens[7] = 200
        lens[20] = 0
        _case(lens, [(13 * i) % 200 for i in range(n)], 64, 2, dtype, seed=61)


@pytest.mark.parametrize("n", [33, 65, 1100])
@pytest.mark.parametrize("few", [True, False])
def test_many_sequences(n, few):
    lens = [(5 * i) % 4 if few else (29 * i) % 40 for i in range(n)]  # empty ones among them
    assert (sum(lens) <= 4 * n) == few
    _case(lens, [(17 * i) % 90 for i in range(n)], 32, 1, "bf16", seed=n, width=3)


@pytest.mark.parametrize("n", [33, 65, 1100])
@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 2, 1), ("bf16", 8, 1), ("f32", 2, 2)])
def test_prompts_of_many_sequences(n, dtype, hq, hkv):
    lens = [(7 * i) % 5 if n > 100 else (29 * i) % 60 for i in range(n)]
    q, k, v, cu = _inputs(lens, hq, hkv, 32, dtype, seed=n)
    out, lse = _attn().prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), return_lse=True)
    _check_prompt(q, k, v, cu, out, lse)


@pytest.mark.parametrize("lens", [[1, 3, 2], [70, 64, 1]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.75, 0.0, -1.0, float("inf"), float("nan"), 2.0 ** -127, 2.0 ** 127])
def test_scales_of_earlier_positions_that_cannot_be_used(scale, dtype, lens):
    """Flagged, and that page and head stay as they are; the scale of a page without earlier positions is free."""
    a = _attn()
    g = gen(91)
    heads, d, width = 2, 64, 4
    T = sum(lens)
    cache = make_cache(g, 3 * width, heads, d)
    k, v = randn(g, T, heads, d).to(DT[dtype]), randn(g, T, heads, d).to(DT[dtype])
    table = torch.randperm(3 * width, generator=g).reshape(3, width).int()
    cu, start = cu_of(lens), torch.tensor([5, 64, 100], dtype=torch.int32)
    want = _want(cache, k, v, cu, start, table)
    bad = [x.clone() for x in cache]
    first, fresh, last = int(table[0, 0]), int(table[1, 1]), int(table[2, 1])
    bad[2][first, 1] = scale  # keys of sequence 0's first page
    bad[3][last, 0] = scale   # values of sequence 2's
    bad[2][fresh], bad[3][fresh] = scale, scale
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _append(bad, k, v, cu, start, table, err_flag=flag)
    assert flag.item() == a.KDA_DEVERR_SCALE
    for i, page, h in ((0, first, 1), (1, last, 0)):
        assert torch.equal(got[i][page, h], cache[i][page, h])
        assert torch.equal(got[i + 2][page, h].view(torch.int32), bad[i + 2][page, h].view(torch.int32))
        got[i][page, h], got[i + 2][page, h] = torch.from_numpy(want[i])[page, h], float(want[i + 2][page, h])
    _compare(got, want)
