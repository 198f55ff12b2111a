"""Shared prefixes: groups of all kinds in one batch."""
import pytest
import torch

from attn_testutil import check, gen, randn
from test_gpu_attn_shared import BF, F32, _attn, _case, _compare, _run, _want

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("dtype,D,hq,d", [(BF, 1, 4, 64), (BF, 1, 12, 128), (BF, 7, 8, 128), (F32, 2, 4, 64)])
def test_table_entries_past_a_sequences_last_page_are_not_read(dtype, D, hq, d):
    """Groups that end inside their prefix, the first row among them, and groups of padding alone: their rows name no
    page behind their own last one."""
    g = gen(D + hq)
    case = list(_case(g, [(6, [70, 300, 129, 0]), (5, [0, 0, 0]), (9, [64, 640, 1]), (4, [0, 200])], 2, d))
    table = case[2]
    for n, length in enumerate(case[1].tolist()):
        held = -(-length // 64)
        for j in range(held):  # (the first row may be the only one that names a page yet)
            assert table[n, j] >= 0
        table[n, held:] = -1
    _compare(tuple(case), (2 * randn(g, len(case[1]), D, hq, d)).to(dtype), dtype)


def test_wrong_offsets_whose_groups_sum_past_31_bits():
    """Groups that overlap again and again have more chunks of rows than 31 bits count; no result is looked for there."""
    from gated_delta_rule_decode_gb300 import kda
    a, B = _attn(), 60000
    c = a.alloc_cache(4, 1, 32)
    q = torch.ones(B, 1, 8, 32, dtype=BF, device="cuda")
    lens, table = torch.full((B,), 64, dtype=torch.int32, device="cuda"), torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    start = torch.tensor([0, B], dtype=torch.int32).repeat(65537).cuda()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    a.decode_shared(q, c, lens, table, start, torch.ones(start.shape[0] - 1, dtype=torch.int32, device="cuda"), err_flag=flag)
    assert flag.item() & kda.KDA_DEVERR_SEQLENS
    flag.zero_()
    out = a.decode_shared(q, c, lens, table, _i32([0, B]).cuda(), _i32([1]).cuda(), err_flag=flag)
    assert flag.item() == 0 and (out == 0).all()  # (the cache's values)
