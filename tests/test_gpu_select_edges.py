"""Page selection: windows of many rows, rows of many pages, scores of any size, errors whatever the budget."""
import pytest
import torch

from attn_testutil import gen, randn
from test_gpu_select import BF, F32, _attn, _i32, _random_summary, _selects

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,hq,hkv,d", [(BF, 16, 16, 2, 128), (BF, 13, 5, 1, 64), (F32, 16, 20, 2, 32), (BF, 3, 128, 1, 128)])
def test_windows_of_more_than_64_rows(dtype, D, hq, hkv, d):
    g = gen(D + hq)
    b, u = _random_summary(g, 150, hkv, d)
    lens = _i32([150 * 64, 149 * 64 + 1, 64 * 40, 700])
    table = torch.stack([torch.randperm(150, generator=g) for _ in range(4)]).int()
    _selects((2 * randn(g, 4, D, hq, d)).to(dtype), b, u, lens, table, 11, 1, 2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_power,unit_power", [(110, 60), (120, -100), (-110, -60), (-130, 100), (-126, -126), (126, 126)])
def test_scores_beyond_fp32s_range(dtype, q_power, unit_power):
    """Whole numbers times powers of two whose product leaves fp32's range keep their order, zero and both signs too."""
    g = gen(q_power + 200)
    b, u = _random_summary(g, 90, 2, 64)
    b[::3] = -b[::3].abs()
    b[:, :, 0], b[:, :, 1] = torch.maximum(b[:, :, 0], b[:, :, 1]), torch.minimum(b[:, :, 0], b[:, :, 1])
    b[10:14] = 0
    u = u * 0 + 2.0 ** unit_power
    u[1::2] *= 0.5 if unit_power > 0 else 2.0
    q = randn(g, 3, 2, 8, 64).double()
    q[1, 0], q[2, 1] = q[1, 0] * 2.0 ** -9, q[2, 1] * 2.0 ** -14
    q = (q.clamp(-1.9, 1.9) * 2.0 ** q_power).to(dtype)
    lens = _i32([90 * 64, 80 * 64 - 5, 90 * 64 - 63])
    _selects(q, b, u, lens, torch.arange(90, dtype=torch.int32).repeat(3, 1), 20, 1, 2)


def test_rows_of_units_far_apart():
    """A row of much larger unit that scores nothing or below leaves the choice to the small one."""
    g = gen(5)
    b, u = _random_summary(g, 70, 1, 32)
    b[:, :, :, :4] = 0  # the first channels' keys
    b[:20, :, 0, 4:], b[:20, :, 1, 4:] = -1, -3
    q = torch.zeros(1, 1, 3, 32)
    q[0, 0, 0, :4] = 2.0 ** 90           # scores 0 everywhere
    q[0, 0, 1, 4:] = 2.0 ** -120         # below 0 for the first pages
    q[0, 0, 2, 4:] = 2.0 ** -120 * torch.rand(28, generator=g)
    for dtype in (BF, F32):
        _selects(q.to(dtype), b, u, _i32([70 * 64]), torch.arange(70, dtype=torch.int32)[None], 9, 0, 1)


@pytest.mark.parametrize("width", [6, 30])
def test_errors_of_sequences_that_keep_all_their_pages(width):
    """Entries outside the cache and units that are no powers of two are flagged for them as for others."""
    g, a = gen(8), _attn()
    b, u = _random_summary(g, 20, 2, 32)
    q = randn(g, 2, 1, 4, 32)
    base = torch.full((2, width), -1, dtype=torch.int32)
    base[:, :4] = torch.arange(8, dtype=torch.int32).view(2, 4)
    lens = _i32([4 * 64 - 3, 4 * 64])
    _selects(q, b, u, lens, base, 8, 1, 2)  # (entries past the last page are not looked at)
    for bad in (-1, 20, 1 << 30):
        table = base.clone()
        table[1, 2] = bad
        _selects(q, b, u, lens, table, 8, 1, 2, a.KDA_DEVERR_PAGE)
    for bad in (3.0, 0.0, float("nan"), -1.0, 2.0 ** 127):
        odd = u.clone()
        odd[5, 1] = bad
        _selects(q, b, odd, lens, base, 8, 1, 2, a.KDA_DEVERR_SCALE)
        odd[5, 1], odd[9, 0] = u[5, 1], bad  # of a page that no row names
        _selects(q, b, odd, lens, base, 8, 1, 2)


@pytest.mark.parametrize("P,budget", [(50001, 300), (52000, 51990)])
def test_rows_whose_scores_do_not_fit_shared_memory(P, budget):
    g = gen(P)
    b, u = _random_summary(g, 900, 1, 32)  # (pages repeat, and so do scores)
    table = torch.randint(0, 900, (1, P), generator=g, dtype=torch.int32)
    _selects(randn(g, 1, 1, 1, 32).to(BF), b, u, _i32([P * 64 - 9]), table, budget, 1, 2)
