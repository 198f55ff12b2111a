"""Query elements near the largest fp32 value."""
import pytest
import torch

from test_gpu_attn_decode import _check, _run, _setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [3e-39, 1e-38])
def test_the_largest_fp32_queries(scale):
    """Query elements above 2^127 (a score scale brings the scores back)."""
    q, cache, n, table = _setup([150, 70], 1, 4, 2, 64, "f32", seed=43, spread=0.0)
    q = q / q.abs().amax() * torch.finfo(torch.float32).max
    _check(q, cache, n, table, _run(q, cache, n, table, scale=scale), scale)
