"""Shared prefixes at the ends of their ranges: the largest queries, long prefixes, many groups and sequences."""
import numpy as np
import pytest
import torch

from attn_long_testutil import bounds
from attn_testutil import check, gen, make_cache, np64, randn
from oracle import attention as ref
from test_gpu_attn_shared import BF, F32, _case, _compare, _run
from test_gpu_shared_precision import OFF

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_fp32s_last_binade(d):
    """Elements of 2^127 and more keep their bits like others (the keys' scales and the score scale bring them back)."""
    g = gen(d)
    case = _case(g, [(20, [1400, 1290, 1300])], 1, d)
    case[0][2].mul_(0).add_(2.0 ** -126)
    q = randn(g, 3, 1, 16, d).clamp(-2.9, 2.9) / 3
    q[..., ::5] = torch.sign(q[..., ::5]) * (0.5 + 0.49 * torch.rand(q[..., ::5].shape, generator=g))
    q = (q.double() * 2.0 ** 128).bfloat16()
    assert torch.isfinite(q).all()
    out, lse, flag = _run(case, q, scale=2.0 ** -8)
    k, v, ks, vs = case[0]
    want, want_lse, absout, mag, _ = ref.decode(np64(q), k.numpy(), v.numpy(), np64(ks), np64(vs), case[1].numpy(), case[2].numpy(),
                                                scale=2.0 ** -8)
    tol, tol_lse = bounds(want, absout, mag, d, BF, OFF)
    assert flag == 0
    check(out, want, tol, "out")
    check(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("d,hkv,rows", [(128, 4, 4), (64, 4, 6)])
def test_a_prefix_of_1600_pages(d, hkv, rows):
    """A worker's share is dozens of blocks, whose products are added up in tensor memory, 16 positions at a time, by
    tensor cores that may truncate each sum: off by 2^-22 of it each time, at most."""
    g = gen(d + 1)
    shared, lens = 1600, [1600 * 64 + 40, 1600 * 64 + 3, 1600 * 64 + 64]
    cache = make_cache(g, 48, hkv, d)  # (the pages repeat)
    table = torch.randint(0, 48, (3, shared + 1), generator=g, dtype=torch.int32)
    table[:, :shared] = table[0, :shared]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    case = (cache, i32(lens), table, i32([0, 3]), i32([shared]))
    q = (2 * randn(g, 3, 1, rows * hkv, d)).bfloat16()
    out, lse, flag = _run(case, q)
    k, v, ks, vs = cache
    want, want_lse, absout, mag, _ = ref.decode(np64(q), k.numpy(), v.numpy(), np64(ks), np64(vs), case[1].numpy(), table.numpy())
    tol, tol_lse = bounds(want, absout, mag, d, BF, OFF)
    # a kv head's share of the 152 workers is `per` of them; a tile has every other block of a worker's pages
    per = 152 // hkv
    steps = 4 * (shared // per + 2)
    assert flag == 0
    check(out, want, tol + absout * steps * 2.0 ** -22, "out")
    check(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("dtype,hq,hkv,d", [(BF, 1, 1, 64), (BF, 20, 1, 64), (F32, 2, 1, 32)])
def test_more_groups_and_sequences_than_the_plan_has_threads(dtype, hq, hkv, d):
    """1300 groups, 2300 sequences: chunks beyond those that the plan keeps in shared memory."""
    g = gen(hq)
    sizes = np.random.default_rng(0).integers(0, 4, 1300)
    sizes[7] = 2300 - (sizes.sum() - sizes[7]) if sizes.sum() - sizes[7] < 2300 else 1
    groups = [(int(i % 3), [int(1 + (i * 37 + 11 * j) % 200) for j in range(n)]) for i, n in enumerate(sizes)]
    case = _case(g, groups, hkv, d)
    assert case[1].shape[0] > 1024 and case[3].shape[0] > 1024
    _compare(case, (2 * randn(g, case[1].shape[0], 1, hq, d)).to(dtype), dtype)
