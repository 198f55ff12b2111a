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


WIDE = 2000  # columns of a table in which reading a large group's prefix for few rows at a time would cost


def _mixed(g, big, small, hkv, d, width=WIDE):
    """One large group among small ones, of one, two and five sequences, of none, and sequences of no group."""
    groups = [(0, [70])] + [(2, [130 + i]) for i in range(small)] + [(3, [200 + 3 * i for i in range(big)])]
    groups += [(1, [100, 65]), (4, [300] * 5), (2, []), (3, [])] + [(1, [64 + i]) for i in range(small)]
    return _case(g, groups, hkv, d, width=width)


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("dtype,D,hq,hkv,d", [(BF, 1, 8, 2, 128), (BF, 2, 3, 1, 64), (F32, 1, 8, 2, 64), (BF, 1, 8, 2, 32), (F32, 3, 4, 2, 128),
                                              (BF, 1, 32, 2, 128), (BF, 1, 1, 1, 64)])
def test_a_large_group_among_small_ones(dtype, D, hq, hkv, d, width):
    g = gen(d + D + hq)
    case = _mixed(g, 37, 20, hkv, d, width)
    _compare(case, (2 * randn(g, case[1].shape[0], D, hq, d)).to(dtype), dtype)


@pytest.mark.parametrize("dtype,d,together", [(BF, 128, 64), (BF, 64, 64), (F32, 64, 16)])
def test_a_large_groups_prefix_is_read_for_many_rows_together(dtype, d, together):
    """The pages are named by one row of the table for as many sequences as are computed together: 256 rows of queries,
    64 where the tensor cores do not compute them."""
    g = gen(d)
    groups = [(1, [80 + i]) for i in range(70)] + [(3, [193 + i % 50 + (60 if i % together == 7 else 0) for i in range(64)])]
    case = list(_case(g, groups, 2, d, width=WIDE))
    q = randn(g, 134, 1, 8, d).to(dtype)
    want, want_lse, tol, tol_lse = _want(case, q, dtype)
    case[2] = case[2].clone()
    for i in range(64):
        if i % together != 7:  # (not the longest of them)
            case[2][70 + i, :3] = -1
    out, lse, flag = _run(tuple(case), q)
    assert flag == 0
    check(out, want, tol, "out")
    check(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("B", [1, 3])
def test_windows_of_no_group(B):
    """No prefixes at all: the sequences' own rows choose how they are attended."""
    g = gen(B)
    case = list(_case(g, [(0, [900, 130, 16][:B])], 2, 128))
    case[3], case[4] = _i32([0]), torch.zeros(0, dtype=torch.int32)
    _compare(tuple(case), (2 * randn(g, B, 16, 16, 128)).to(BF), BF)
