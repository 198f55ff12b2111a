"""Later tokens have no influence on a prompt's rows, to the last bit."""
import pytest
import torch

from attn_testutil import cu_of
from test_gpu_attn_prefill import _attn, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 2, 2), ("bf16", 64, 8, 1), ("bf16", 128, 5, 1),
                                            ("bf16", 32, 4, 2), ("f32", 64, 2, 1)])
def test_a_prefix_gives_the_same_bits(dtype, d, hq, hkv):
    a = _attn()
    q, k, v, cu = (x.cuda() for x in _inputs([1000], hq, hkv, d, dtype, seed=31))
    out, lse = a.prefill(q, k, v, cu, return_lse=True)
    for n in (1, 17, 100, 129, 160, 257, 300, 500, 777, 999):
        o, l = a.prefill(q[:n], k[:n], v[:n], cu_of([n]).cuda(), return_lse=True)
        assert torch.equal(o, out[:n]) and torch.equal(l, lse[:n]), n


@pytest.mark.parametrize("d,hq,hkv", [(128, 2, 2), (64, 8, 1)])
def test_other_later_tokens_give_the_same_bits(d, hq, hkv):
    a = _attn()
    q, k, v, cu = (x.cuda() for x in _inputs([800], hq, hkv, d, "bf16", seed=32))
    out, lse = a.prefill(q, k, v, cu, return_lse=True)
    for n in (150, 270, 390, 530, 650):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        q2[n:] *= 30
        k2[n:] = -k2[n:]
        v2[n:] *= 1000
        o, l = a.prefill(q2, k2, v2, cu, return_lse=True)
        assert torch.equal(o[:n], out[:n]) and torch.equal(l[:n], lse[:n]), n
