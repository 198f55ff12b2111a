"""Bounded waits of the attention over shared prefixes and selected pages: a
library whose waits give up after one poll (see test_gpu_timeout.py) returns,
reports KDA_DEVERR_TIMEOUT and leaves the context usable."""
import pytest
import torch

from attn_testutil import gen, make_cache, randn, to_device
from test_gpu_attn_timeout import _with_lib, variant  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_waits_give_up_and_the_context_stays_usable(variant, d):  # noqa: F811
    from gated_delta_rule_decode_gb300 import attn, kda
    g = gen(91)
    cache = to_device(make_cache(g, 60, 2, d))
    table = torch.arange(60, dtype=torch.int32).view(4, 15)
    table[1, :9], table[3, :4] = table[0, :9], table[2, :4]
    table = table.cuda()
    lens = torch.tensor([900, 700, 500, 256 + 7], dtype=torch.int32).cuda()
    start = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    shared = torch.tensor([9, 4], dtype=torch.int32).cuda()
    index = torch.arange(15, dtype=torch.int32).expand(4, 2, 15).contiguous().cuda()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    one, all4 = torch.tensor([0, 4], dtype=torch.int32).cuda(), torch.tensor([4], dtype=torch.int32).cuda()
    gave_up, either = (kda.KDA_DEVERR_TIMEOUT,), (0, kda.KDA_DEVERR_TIMEOUT)
    # 28 rows of a sequence and kv head: all on tcgen05, whose roles wait for one another; 4 rows, prefixes of groups
    # of 8, fp32: by warps that wait for copies which may have landed; a group of 16 rows: its prefix on tcgen05
    for D, dtype, groups, flags in ((7, torch.bfloat16, (start, shared), gave_up), (1, torch.bfloat16, (start, shared), either),
                                    (2, torch.float32, (start, shared), either), (1, torch.bfloat16, (one, all4), gave_up)):
        q = randn(g, 4, D, 8, d).to(dtype).cuda()
        call = lambda: attn.decode_shared(q, cache, lens, table, *groups, return_lse=True, err_flag=flag)  # noqa: E731,B023
        flag.zero_()
        want = call()
        assert flag.item() == 0
        _with_lib(variant, call)
        torch.cuda.synchronize()
        assert flag.item() in flags
        flag.zero_()
        for x, y in zip(call(), want):
            assert torch.equal(x, y)
        assert flag.item() == 0
    q = randn(g, 4, 1, 8, d).bfloat16().cuda()
    selected = attn.Selected(lens, table.view(4, 1, 15).expand(4, 2, 15).contiguous(), index)
    call = lambda: attn.decode_selected(q, cache, selected, err_flag=flag)  # noqa: E731
    want = call()
    assert flag.item() == 0
    _with_lib(variant, call)
    torch.cuda.synchronize()
    assert flag.item() in (0, kda.KDA_DEVERR_TIMEOUT)
    assert torch.equal(call(), want)
