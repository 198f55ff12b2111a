"""Infinite and NaN values that a prompt's rows see: the fp64 definition's
infinity or NaN in exactly those rows and channels."""
import numpy as np
import pytest

from test_gpu_attn_prefill import _attn, _check, _inputs

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dtype,d", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 1), (10, 2)])
@pytest.mark.parametrize("values", [
    [(0, 1, INF)],                                  # the sequence's first token
    [(100, 1, -INF)],                               # among the first block of keys
    [(0, 2, INF), (290, 2, INF), (300, 5, -INF)],   # one channel twice; one that few rows see
    [(3, 0, INF), (280, 0, -INF)],                  # both signs: NaN from the second on
    [(129, 7, float("nan")), (140, 8, -INF), (140, 31, INF)],
])
def test_visible_values_that_are_not_finite(dtype, d, hq, hkv, values):
    a = _attn()
    q, k, v, cu = _inputs([50, 330], hq, hkv, d, dtype, seed=21, qstd=1.0)
    for at, c, x in values:
        v[50 + at, 0, c] = x  # the first kv head of the second sequence
    out, lse = a.prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), return_lse=True)
    with np.errstate(invalid="ignore"):
        _check(q, k, v, cu, out, lse)


def test_an_infinite_value_early_in_a_long_prompt():
    """Tiles whose first token lies far behind the value."""
    a = _attn()
    q, k, v, cu = _inputs([900], 2, 1, 64, "bf16", seed=22, qstd=1.0)
    clean = a.prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda()).cpu()
    v[40, 0, 9], v[200, 0, 10], v[700, 0, 11] = INF, -INF, INF
    out = a.prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda()).cpu()
    assert (out[40:, :, 9] == INF).all() and (out[200:, :, 10] == -INF).all() and (out[700:, :, 11] == INF).all()
    out[40:, :, 9], out[200:, :, 10], out[700:, :, 11] = clean[40:, :, 9], clean[200:, :, 10], clean[700:, :, 11]
    assert (out == clean).all()
