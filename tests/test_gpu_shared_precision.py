"""Shared prefixes on tcgen05: queries whose channels differ by any factor give the results of kda_attn_decode.

There a query row is scaled so that its largest element is in 2^7..2^8 and multiplied as an e4m3 term and an e5m2
term of what the first leaves.  With x an element of 2^e.., 8 bits, steps of 2^(e-7): the first term leaves at most
half its step, max(2^(e-4), 2^-10), in steps of 2^(e-7).  Down to e = -6 that is a sum of 3 bits, which e5m2 holds
exactly (its smallest step is 2^-16).  Where what the terms leave (the sum of its magnitudes times the largest key that
the page's scale can hold) may be more than 2^-11 of a score in units of log 2, the scores get it in fp32: a score is off
by at most 2^-11 ln 2, as much as a weight's rounding moves it, besides what `bounds` counts for every kernel."""
import numpy as np
import pytest
import torch

from attn_long_testutil import bounds
from attn_testutil import check, gen, np64, randn
from oracle import attention as ref
from test_gpu_attn_shared import _case, _run

BF = torch.bfloat16
OFF = 2.0 ** -11 * np.log(2)


def _compare(case, q):
    out, lse, flag = _run(case, q)
    k, v, ks, vs = case[0]
    want, want_lse, absout, mag, _ = ref.decode(np64(q), k.numpy(), v.numpy(), np64(ks), np64(vs), case[1].numpy(), case[2].numpy())
    tol, tol_lse = bounds(want, absout, mag, q.shape[-1], BF, OFF)
    assert flag == 0
    check(out, want, tol, "out")
    check(lse, want_lse, tol_lse, "lse")


def _e5m2_round(x):
    """To nearest, ties to even, of finite |x| <= 57344: 3 bits, steps of 2^-16 at least."""
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -16))) - 2, -16))
    return np.rint(x / step) * step


def test_two_terms_hold_an_element():
    """All 128 significands of bf16 at every size: exact from 2^-6 on, and off by at most 2^-14 below."""
    for e in range(-30, 8):
        x = np.ldexp(1 + np.arange(128) / 128, e)
        first = ref._VALUES[ref.e4m3_round(x)]
        left = np.abs(x - first - _e5m2_round(x - first))
        assert left.max() <= (0 if e >= -6 else 2.0 ** -14)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [9, 13, 16, 20, 27])
@pytest.mark.parametrize("D,hq", [(1, 10), (2, 10), (16, 20)])
def test_an_outlier_that_meets_no_key_changes_nothing(power, d, D, hq):
    """A channel 2^power times the others, whose keys are zero: the scores are the other channels'."""
    g = gen(power + D)
    case = _case(g, [(20, [1400, 1290, 1300])], 1, d)
    case[0][0][..., 5] = 0
    q = 2 * randn(g, 3, D, hq, d)
    q[:, :, ::2, 5] = 2.0 ** power * (1 + torch.rand(3, D, (hq + 1) // 2, generator=g))
    _compare(case, q.bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [1, 5])
def test_elements_of_all_sizes(D):
    """Elements over 2^20, every third channel's keys zero, two kv heads, pages that are not there among them."""
    g = gen(71 + D)
    case = _case(g, [(18, [1300, 1290, 1170, 1200]), (3, [400, 200])], 2, 128, spread=3.0)
    case[0][0][..., ::3] = 0
    q = 8 * randn(g, 6, D, 20, 128) * torch.exp2(torch.randint(-20, 1, (6, D, 20, 128), generator=g).float())
    _compare(case, q.bfloat16())


@pytest.mark.gpu
def test_a_row_does_not_change_others():
    """A row that needs more than two terms gets it by itself: the other rows' bits stay."""
    g = gen(73)
    case = _case(g, [(20, [1400, 1290, 1300])], 1, 128)
    q = randn(g, 3, 2, 10, 128).bfloat16()
    want, want_lse, _ = _run(case, q)
    q[1, 1, 4, 7] = 2.0 ** 25
    out, lse, flag = _run(case, q)
    rest = torch.ones(3, 2, 10, dtype=torch.bool)
    rest[1, 1, 4] = False
    assert flag == 0 and torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [[5], [5, 6, 7], [0, 63], [3, 20, 40], [1, 9, 17, 25, 33, 41, 49, 57]])
@pytest.mark.parametrize("D,hq", [(1, 12), (8, 24)])
def test_large_channels_that_meet_small_keys(d, at, D, hq):
    """Channels of 2^4 to 2^14 times the others, in one piece of a row and in all, whose keys are as much smaller."""
    g = gen(len(at) + D)
    case = _case(g, [(20, [1400, 1290, 1300])], 1, d)
    q = 2 * randn(g, 3, D, hq, d)
    q[..., at] *= torch.exp2(torch.randint(4, 15, (3, D, hq, 1), generator=g).float())
    case[0][0][..., at] = 0x01 + 0x80 * torch.randint(0, 2, case[0][0][..., at].shape, generator=g, dtype=torch.uint8)
    _compare(case, q.bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("power", [95, 120])
def test_elements_further_apart_than_a_score_holds(power):
    """A channel 2^95 and 2^120 times the others, whose keys are zero.  (Windows of 24 rows, all of them on tcgen05: the
    warps' kernel rounds what is below 2^-28 of a row's largest.)"""
    g = gen(power)
    case = _case(g, [(20, [1400, 1290, 1300])], 1, 128)
    case[0][0][..., 9] = 0
    q = randn(g, 3, 2, 12, 128)
    q[:, :, 1::2, 9] = 2.0 ** power
    _compare(case, q.bfloat16())
