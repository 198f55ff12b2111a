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
