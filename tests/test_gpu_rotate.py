"""Norm and rotation of query and key heads against the fp64 definition.

Tolerance: the sum of squares is off by at most 13 roundings of 2^-24 (half of
that after the root), the reciprocal root by 2^-22, three products follow:
below 2^-20 of the normed value.  cos and sin are off by 2^-23 and the angle's
2^-24, two products and sums follow: below 2^-21 of the pair's magnitude.  So
1.5 * 2^-20 of |y_a| + |y_b|, and the output's own half step."""
import numpy as np
import pytest
import torch

from attn_testutil import check, gen, np64, randn
from oracle import attention as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _attn():
    from gated_delta_rule_decode_gb300 import attn
    return attn


def _tol(out, size, dtype):
    return 1.5 * 2.0 ** -20 * size + np.abs(out) * (torch.finfo(dtype).eps / 2) + 1e-38


def _compare(got, x, pos, rot, weight, dtype, eps=1e-6):
    turns, inter, factor = rot
    want, size = ref.rotate(np64(x), pos.tolist(), turns.tolist(), inter, factor, None if weight is None else np64(weight), eps)
    check(got, want, _tol(want, size, dtype), "rotated")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,hq,hkv", [(32, 3, 1), (64, 4, 4), (128, 10, 2), (128, 33, 11), (32, 1, 1)])
@pytest.mark.parametrize("rot,inter", [(1.0, False), (1.0, True), (0.5, False), (0.25, True), ("odd", False), ("odd", True),
                                       (0, False)])
@pytest.mark.parametrize("fused", [False, True])
def test_matches_the_definition(dtype, d, hq, hkv, rot, inter, fused):
    a, g = _attn(), gen(d + hq)
    rd = d // 2 - 2 if rot == "odd" else int(rot * d)
    T = 7
    q, k = randn(g, T, hq, d, dtype=dtype).cuda(), (5 * randn(g, T, hkv, d)).to(dtype).cuda()
    if fused:
        row = torch.cat([q, k, k], 1)
        q, k = row[:, :hq], row[:, hq:hq + hkv]
    pos = torch.tensor([0, 1, -3, 102399, 1000003, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    r = a.rotary(a.rotary_frequencies(rd, stretch=8.0, trained=4096), interleaved=inter, factor=1.2)
    qw, kw = 1 + 0.3 * randn(g, d), 1 + 0.3 * randn(g, d)
    for w1, w2 in ((qw, kw), (None, None), (None, kw)):
        qo, ko = a.norm_rotate(q, k, pos.cuda(), r, q_weight=None if w1 is None else w1.cuda(),
                               k_weight=None if w2 is None else w2.cuda(), eps=1e-3)
        _compare(qo, q, pos, r, w1, dtype, 1e-3)
        _compare(ko, k, pos, r, w2, dtype, 1e-3)


@pytest.mark.parametrize("T", [0, 1, 2, 1000])
def test_lengths(T):
    a, g = _attn(), gen(T)
    q, k = randn(g, T, 4, 64).bfloat16().cuda(), randn(g, T, 2, 64).bfloat16().cuda()
    pos = torch.arange(T, dtype=torch.int32) * 131
    r = a.rotary(a.rotary_frequencies(64))
    w = torch.ones(64, device="cuda")
    qo, ko = a.norm_rotate(q, k, pos.cuda(), r, q_weight=w, k_weight=w)
    assert qo.shape == q.shape and ko.shape == k.shape
    at = [i for i in (0, 1, 500, 999) if i < T]
    if at:
        _compare(qo[at], q[at], pos[at], r, torch.ones(64), BF)
        _compare(ko[at], k[at], pos[at], r, torch.ones(64), BF)


@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (24, False), (50, False)])
def test_in_place_of_a_fused_projection(rot, inter):
    a, g = _attn(), gen(3)
    row = randn(g, 40, 14, 128).bfloat16().cuda()
    pos = torch.randint(0, 5000, (40,), generator=g, dtype=torch.int32).cuda()
    r, w = a.rotary(a.rotary_frequencies(rot), interleaved=inter), (1 + 0.1 * randn(g, 128)).cuda()
    want = a.norm_rotate(row[:, :10], row[:, 10:12], pos, r, q_weight=w, k_weight=w)
    v = row[:, 12:].clone()
    got = a.norm_rotate(row[:, :10], row[:, 10:12], pos, r, row[:, :10], row[:, 10:12], q_weight=w, k_weight=w)
    assert got[0].data_ptr() == row.data_ptr()
    assert torch.equal(row[:, :10], want[0]) and torch.equal(row[:, 10:12], want[1]) and torch.equal(row[:, 12:], v)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rot,inter", [(32, False), (30, False), (30, True)])
def test_values_that_are_no_numbers_stay_where_they_are(dtype, rot, inter):
    a, g = _attn(), gen(4)
    q, k = randn(g, 3, 2, 64).to(dtype), randn(g, 3, 1, 64).to(dtype)
    bad = q.clone()
    bad[1, 0, 40], bad[1, 0, 63], bad[2, 1, 0] = float("nan"), float("inf"), float("inf")
    pos = torch.tensor([1, 2, 3], dtype=torch.int32).cuda()
    r = a.rotary(a.rotary_frequencies(rot), interleaved=inter)
    want, _ = a.norm_rotate(q.cuda(), k.cuda(), pos, r)
    got, _ = a.norm_rotate(bad.cuda(), k.cuda(), pos, r)
    differ = ~((got == want) | (got.isnan() & want.isnan()))
    assert set(map(tuple, differ.nonzero().tolist())) == {(1, 0, 40), (1, 0, 63), (2, 1, 0), (2, 1, 1 if inter else rot // 2)}


def test_captured_and_on_another_stream():
    a, g = _attn(), gen(5)
    q, k = randn(g, 300, 4, 128).bfloat16().cuda(), randn(g, 300, 2, 128).bfloat16().cuda()
    pos = torch.arange(300, dtype=torch.int32).cuda()
    r = a.rotary(a.rotary_frequencies(128))
    want = a.norm_rotate(q, k, pos, r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = a.norm_rotate(q, k, pos, r, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = a.norm_rotate(q, k, pos, r)
    q.mul_(2)
    pos.add_(7)
    graph.replay()
    want = a.norm_rotate(q, k, pos, r)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
