"""Attention over packed prompts against its fp64 definition: types, head
groups, lengths around the tiles' edges, fused-projection strides, values that
must not be read, refusals."""
import ctypes

import numpy as np
import pytest
import torch

from attn_testutil import DT, bounds, check, cu_of, gen, np64, randn
from oracle import attention as ref

pytestmark = pytest.mark.gpu


def _attn():
    from gated_delta_rule_decode_gb300 import attn
    return attn


def _inputs(lens, hq, hkv, d, dtype, seed, qstd=2.0):
    g = gen(seed)
    T = sum(lens)
    dt = DT[dtype]
    return ((qstd * randn(g, T, hq, d)).to(dt), randn(g, T, hkv, d).to(dt), randn(g, T, hkv, d).to(dt), cu_of(lens))


def _check(q, k, v, cu, out, lse, scale=None):
    o, l, a, m = ref.prompt(np64(q), np64(k), np64(v), cu.tolist(), scale)
    to, tl = bounds(o, a, m, q.shape[2], q.dtype)
    check(out, o, to, "out")
    check(lse, l, tl, "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens,hq,hkv", [
    ([1], 1, 1),
    ([5, 0, 1, 2], 2, 2),
    ([63, 64, 65], 3, 1),
    ([127, 1, 129, 0, 128], 4, 2),
    ([300], 8, 1),
    ([17, 260], 10, 2),
    ([40, 3], 32, 2),
    ([9, 30], 24, 1),
])
def test_prompt_matches_definition(lens, hq, hkv, d, dtype):
    q, k, v, cu = _inputs(lens, hq, hkv, d, dtype, seed=hq * d + len(lens))
    out, lse = _attn().prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), return_lse=True)
    _check(q, k, v, cu, out, lse)


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 4, 1), ("bf16", 64, 2, 2), ("f32", 64, 2, 1)])
def test_long_prompt_rows(dtype, d, hq, hkv):
    """A prompt of many key blocks, checked in full against a 64-bit torch form."""
    T = 1543
    q, k, v, cu = _inputs([T], hq, hkv, d, dtype, seed=11)
    out, lse = _attn().prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), return_lse=True)
    seen = np.tril(np.ones((T, T), bool))
    for h in range(hq):
        kk, vv = np64(k[:, h * hkv // hq]), np64(v[:, h * hkv // hq])
        s = np.where(seen, np64(q[:, h]) @ kk.T * d ** -0.5, -np.inf)
        mx = s.max(1, keepdims=True)
        w = np.exp(s - mx)
        l = w.sum(1, keepdims=True)
        o, a = w @ vv / l, w @ np.abs(vv) / l
        mag = (np.abs(np64(q[:, h])) @ np.abs(kk).T * d ** -0.5 * seen).max(1)
        to, tl = bounds(o, a, mag, d, q.dtype)
        check(out[:, h], o, to, "out")
        check(lse[:, h], (mx + np.log(l))[:, 0], tl, "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_a_fused_projection(dtype):
    """Rows that lie apart give the bits of contiguous ones."""
    a = _attn()
    q, k, v, cu = _inputs([70, 33], 6, 2, 64, dtype, seed=3)
    want = a.prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda())
    row = torch.cat([q, k, v], 1).cuda()
    got = a.prefill(row[:, :6], row[:, 6:8], row[:, 8:], cu.cuda())
    assert torch.equal(got, want)


def test_scale_and_peaked_scores():
    """A scale of its own, and scores so far apart that one key takes all."""
    a = _attn()
    for dtype, qstd, scale in (("bf16", 2.0, 0.5), ("bf16", 60.0, None), ("f32", 60.0, None)):
        q, k, v, cu = _inputs([90], 2, 1, 64, dtype, seed=5, qstd=qstd)
        out, lse = a.prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), return_lse=True, scale=scale)
        _check(q, k, v, cu, out, lse, scale)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_masked_values_have_no_influence(dtype, d, bad):
    """Non-finite keys and values of later tokens and of other sequences."""
    a = _attn()
    q, k, v, cu = _inputs([50, 140, 30], 4, 2, d, dtype, seed=9)
    clean = a.prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda())
    at = 50 + 100  # a token inside the second sequence
    k2, v2 = k.clone(), v.clone()
    k2[at, 1] = bad
    v2[at, 1, 3] = bad
    out = a.prefill(q.cuda(), k2.cuda(), v2.cuda(), cu.cuda())
    assert torch.equal(out[:at], clean[:at])
    assert torch.equal(out[190:], clean[190:])
    assert torch.equal(out[at:190, :2], clean[at:190, :2])  # the heads of kv head 0
    # values alone: the rows that see them get them, other channels keep theirs
    out = a.prefill(q.cuda(), k.cuda(), v2.cuda(), cu.cuda())
    assert torch.equal(out[:at], clean[:at])
    hit = out[at:190, 2:, 3].float()
    assert not torch.isfinite(hit).any()
    other = [c for c in range(d) if c != 3]
    assert torch.equal(out[at:190, 2:][..., other], clean[at:190, 2:][..., other])


def test_tokens_of_no_sequence_are_not_written():
    a = _attn()
    q, k, v, _ = _inputs([100], 2, 1, 64, "bf16", seed=2)
    cu = torch.tensor([10, 40, 90], dtype=torch.int32)
    out = torch.full((100, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    a.prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), out)
    assert (out[:10] == 7).all() and (out[90:] == 7).all()
    want = a.prefill(q[10:90].cuda(), k[10:90].cuda(), v[10:90].cuda(), torch.tensor([0, 30, 80], dtype=torch.int32).cuda())
    assert torch.equal(out[10:90], want)


def test_bad_offsets_set_the_flag():
    a = _attn()
    from gated_delta_rule_decode_gb300 import kda
    q, k, v, _ = _inputs([64], 2, 1, 64, "bf16", seed=2)
    for cu in ([0, 70], [0, 40, 30], [-1, 64]):
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        a.prefill(q.cuda(), k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), err_flag=flag)
        assert flag.item() & kda.KDA_DEVERR_SEQLENS, cu


def test_runs_on_the_given_stream_and_repeats_bit_for_bit():
    a = _attn()
    q, k, v, cu = (x.cuda() for x in _inputs([700, 5, 333], 8, 2, 128, "bf16", seed=4))
    want, wl = a.prefill(q, k, v, cu, return_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [a.prefill(q, k, v, cu, return_lse=True, stream=s) for _ in range(3)]
    s.synchronize()
    for o, l in outs:
        assert torch.equal(o, want) and torch.equal(l, wl)


def test_empty_calls():
    a = _attn()
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    out = a.prefill(e, e[:, :2], e[:, :2], torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64)


def test_binding_refuses():
    a = _attn()
    q, k, v, cu = (x.cuda() for x in _inputs([8], 4, 2, 64, "bf16", seed=1))
    with pytest.raises(ValueError):
        a.prefill(q, k.float(), v, cu)
    with pytest.raises(ValueError):
        a.prefill(q, k, v[:4], cu)
    with pytest.raises(ValueError):
        a.prefill(q, k.transpose(1, 2).contiguous().transpose(1, 2), v, cu)
    with pytest.raises(ValueError):
        a.prefill(q, k, v, cu.long())
    with pytest.raises(TypeError):
        a.prefill(q.half(), k.half(), v.half(), cu)
    with pytest.raises(a.KdaError):
        a.prefill(q[:, :3], k, v, cu)  # 3 query heads over 2 kv heads
    odd = torch.empty((8, 4 * 64 + 1), dtype=torch.bfloat16, device="cuda")[:, :256].view(8, 4, 64)
    with pytest.raises(ValueError):
        a.prefill(odd, k, v, cu)
    assert ctypes.sizeof(a.KdaAttnDims) == 20
