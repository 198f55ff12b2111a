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
