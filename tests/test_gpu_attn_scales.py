"""Rows whose attention lies on pages of small values beside pages of huge ones:
the output keeps its precision whatever the ratio of the pages' value scales."""
import math

import pytest
import torch

from test_gpu_attn_decode import _check, _run, _setup

pytestmark = pytest.mark.gpu


def _case(lens, D, hq, hkv, d, dtype, hot, factors, gap):
    """Keys of page `hot` score `gap` (natural log) above the others; page c's
    values are multiplied by 2^factors[c] (of every sequence, modulo the list)."""
    q, cache, n, table = _setup(lens, D, hq, hkv, d, dtype, seed=41, spread=0.0)
    kp, vp, ks, vs = cache
    ks[:] = 2.0 ** -7  # bytes of +-448 stand for +-3.5
    q[..., 0] = gap * math.sqrt(d) / 7
    for s, x in enumerate(lens):
        for c in range(-(-x // 64)):
            page = int(table[s, c])
            kp[page, :, :, 0] = 0x7e if c == hot else 0xfe
            vs[page] *= 2.0 ** factors[c % len(factors)]
    return q, (kp, vp, ks, vs), n, table


# (D, hq, hkv, d, dtype): the warps' products with one and two row tiles, fp32, and tcgen05
KERNELS = [(1, 32, 8, 128, "bf16"), (3, 32, 8, 64, "bf16"), (1, 16, 8, 64, "f32"), (5, 16, 2, 32, "bf16"),
           (7, 16, 4, 128, "bf16"), (9, 8, 2, 64, "bf16")]


@pytest.mark.parametrize("D,hq,hkv,d,dtype", KERNELS)
@pytest.mark.parametrize("hot,factors,gap", [
    (0, [0, 0, 0, 28, 0], 60.0),        # the huge page after the one that carries the weight
    (3, [40, 0, 0, 0, 0], 80.0),        # and before it
    (2, [0, 0, 0, 100, 0], 120.0),      # side by side, the ratio beyond any 16-bit type
    (3, [0, 0, 100, 0, 0], 120.0),
    (1, [0, -60, 30, -100, 50], 60.0),
    (2, [40, 40, 0, 40, 40], 27.7),     # weight 2^-40 on values 2^40 larger: both count
    (4, [0, 0, 0, 0, 90], 30.0),        # the page of the weight is the huge one
])
def test_attention_on_small_values_beside_huge_ones(D, hq, hkv, d, dtype, hot, factors, gap):
    B = 64 * 8 // hkv if D * hq // hkv <= 16 else max(16, 64 // hkv)  # enough items that none is cut
    if dtype == "bf16" and D * hq // hkv > 16 and d == 32:
        B = 256
    lens = [300 if i % 5 else 257 + i % 60 for i in range(min(B, 64) if D == 1 else min(B, 24))]
    if len(lens) < B:  # the other sequences are padding
        lens += [0] * (B - len(lens))
    s = _case(lens, D, hq, hkv, d, dtype, hot, factors, gap)
    _check(*s, _run(*s, return_weight=True))


@pytest.mark.parametrize("D,hq,hkv,d,dtype", [(1, 8, 8, 64, "bf16"), (1, 8, 8, 64, "f32"), (8, 12, 4, 64, "bf16")])
def test_the_same_where_sequences_are_cut(D, hq, hkv, d, dtype):
    lens = [64 * 40 - 7 * i for i in range(12)] if D == 1 else [64 * 24 - 5 * i for i in range(6)]
    lens += [2560] * (28 if D == 1 else 0)
    for hot, factors, gap in ((7, [0, 30, 0, 0, 60, 0, 0], 70.0), (20, [50, -50], 60.0)):
        q, cache, n, table = _case(lens[:12], D, hq, hkv, d, dtype, hot, factors, gap)
        if len(lens) > 12:  # more copies of the first sequences, so that a worker holds several pages
            rep = [i % 12 for i in range(len(lens))]
            q, n, table = q[rep], n[rep], table[rep]
            got = [x[:12] for x in _run(q, cache, n, table, return_weight=True)]
            q, n, table = q[:12], n[:12], table[:12]
        else:
            got = _run(q, cache, n, table, return_weight=True)
        _check(q, cache, n, table, got)


@pytest.mark.parametrize("D,hq,hkv,d,dtype", [(1, 8, 2, 64, "bf16"), (2, 4, 2, 32, "f32"), (7, 16, 2, 128, "bf16")])
@pytest.mark.parametrize("of,scale", [(3, 0.75), (3, 1.5), (3, 0.0), (3, -0.5), (3, math.inf), (3, math.nan),
                                      (3, 2.0 ** -127), (3, 2.0 ** 127), (3, 3.4e38), (2, 0.0), (2, -1.0), (2, math.inf), (2, math.nan)])
def test_scales_that_cannot_be_used_are_flagged(D, hq, hkv, d, dtype, of, scale):
    """Value scales (3) are used by their exponent, key scales (2) as a factor: a
    page and head with another counts as unseen."""
    from gated_delta_rule_decode_gb300 import attn
    q, cache, n, table = _setup([300, 130], D, hq, hkv, d, dtype, seed=44)
    page, h = int(table[0, 2]), 1
    good = cache[of][page, h].item()
    cache[of][page, h] = scale
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(q, cache, n, table, return_weight=True, err_flag=flag)
    assert flag.item() == attn.KDA_DEVERR_SCALE
    G = hq // hkv
    cache[of][page, h] = good
    seen, gone = _run(q, cache, n, table, return_weight=True), table.clone()
    gone[0, 2] = -1
    unseen = _run(q, cache, n, gone, return_weight=True)
    for x, a, b in zip(got[:2], seen, unseen):  # the other head sees it
        assert torch.equal(x[1], a[1])
        assert torch.equal(x[0, :, :G], a[0, :, :G]) and torch.equal(x[0, :, G:], b[0, :, G:])
    for extreme in (2.0 ** -126, 2.0 ** 100):
        cache[3][page, h] = extreme
        flag.zero_()
        _check(q, cache, n, table, _run(q, cache, n, table, err_flag=flag))
        assert flag.item() == 0
