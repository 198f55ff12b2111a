"""The hybrid serving example: KDA and attention blocks together, each
attention step against the values that the cache stores."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_serving.py")


def _example():
    spec = importlib.util.spec_from_file_location("hybrid_serving", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_course_matches_the_stored_values_and_repeats():
    ex = _example()
    one = ex.run(check=True)
    two = ex.run()
    assert [w for w, _ in one] == [w for w, _ in two]
    for (what, a), (_, b) in zip(one, two):
        assert torch.equal(a, b), what
        if what == "evicted":
            assert a.tolist() == [1, 0, 0]  # 306 positions hold 5 pages, the budget is 4
        else:
            assert torch.isfinite(a.float()).all(), what


def test_other_sizes():
    _example().run(prompts=(65, 200), steps=2, draft=3, accepted=3, budget=3, check=True, q_heads=12, kv_heads=1,
                   d=64, kda_heads=2, hidden=256)
