"""Offsets that are not in order set the error flag, wherever they are; offsets
in order do not."""
import pytest
import torch

from attn_testutil import DT, cu_of, gen, randn

pytestmark = pytest.mark.gpu

# falling and rising again past the units of the sequences in between, beyond the
# end, below zero
BAD = [[0, 1000, 0, 1000], [0, 600, 300, 1000], [0, 600, 500, 1000], [0, 2000, 500, 3000], [0, 40, 30, 64], [0, 40, 30],
       [0, 10, 9, 10], [0, 70, 64], [0, -1, 64], [-5, 64], [0, 64, 0], [5, 4, 64, 64]]
GOOD = [[0, 1000], [0, 0, 1, 1, 700, 1000], [3, 3, 60, 64]]


def _attn():
    from gated_delta_rule_decode_gb300 import attn
    return attn


def _flagged(call):
    from gated_delta_rule_decode_gb300 import kda
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(flag)
    assert flag.item() in (0, kda.KDA_DEVERR_SEQLENS)
    return flag.item() != 0


def _prompt(cu, total, hq, hkv, dtype):
    g = gen(71)
    q, k, v = (randn(g, total, h, 32).to(DT[dtype]).cuda() for h in (hq, hkv, hkv))
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    return _flagged(lambda flag: _attn().prefill(q, k, v, c, err_flag=flag))


def _append(cu, total, dtype):
    g = gen(72)
    n, width = len(cu) - 1, -(-max(total, 1) // 64) + 1
    cache = _attn().alloc_cache(n * width, 1, 32)
    k, v = (randn(g, total, 1, 32).to(DT[dtype]).cuda() for _ in range(2))
    table = torch.arange(n * width, dtype=torch.int32).view(n, width).cuda()
    c, start = torch.tensor(cu, dtype=torch.int32).cuda(), torch.zeros(n, dtype=torch.int32).cuda()
    return _flagged(lambda flag: _attn().append(cache, k, v, c, start, table, err_flag=flag))


@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 2, 2), ("bf16", 8, 1), ("bf16", 100, 1), ("f32", 2, 1)])
def test_prompts(dtype, hq, hkv):
    for cu in BAD:
        assert _prompt(cu, 64 if cu == [0, 70, 64] else max(cu), hq, hkv, dtype), cu
    for cu in GOOD:
        assert not _prompt(cu, 1000, hq, hkv, dtype), cu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append(dtype):
    for cu in BAD:
        assert _append(cu, 64 if cu == [0, 70, 64] else max(cu), dtype), cu
    for cu in GOOD:
        assert not _append(cu, 1000, dtype), cu


@pytest.mark.parametrize("at", [0, 1, 150, 298])
def test_among_many_sequences(at):
    """300 sequences, one of them in disorder: append's kernel for few tokens, and prompts."""
    lens = [3] * 300
    cu = cu_of(lens).tolist()
    assert not _append(cu, 900, "bf16") and not _prompt(cu, 900, 2, 1, "bf16")
    cu[at + 1] = cu[at] - 1 if at else 900
    assert _append(cu, 900, "bf16") and _prompt(cu, 900, 2, 1, "bf16") and _prompt(cu, 900, 2, 1, "f32")
