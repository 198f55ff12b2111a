"""Canary pages around every buffer that the long-context operators write, and no
change in those that they only read (see test_gpu_canary.py)."""
import pytest
import torch

from attn_testutil import cu_of, gen, make_cache, randn
from test_gpu_attn_canary import _guarded_cache
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _attn():
    from gated_delta_rule_decode_gb300 import attn
    return attn


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,hq,hkv,rot", [(32, 3, 1, 32), (64, 4, 4, 30), (128, 10, 2, 64)])
def test_norm_rotate_canaries(d, hq, hkv, rot, dtype):
    a, g, gd = _attn(), gen(1), Guarded()
    q, k = randn(g, 37, hq, d, dtype=dtype).cuda(), randn(g, 37, hkv, d, dtype=dtype).cuda()
    qo, ko = gd.empty((37, hq, d), dtype), gd.empty((37, hkv, d), dtype)
    w = torch.ones(d, device="cuda")
    for inter in (False, True):
        a.norm_rotate(q, k, torch.arange(37, dtype=torch.int32).cuda(), a.rotary(a.rotary_frequencies(rot), interleaved=inter), qo, ko,
                      q_weight=w, k_weight=w)
        gd.check()


@pytest.mark.parametrize("dtype,D,hq,hkv", [(BF, 1, 4, 1), (BF, 7, 8, 2), (BF, 1, 40, 2), (F32, 1, 4, 2), (F32, 5, 8, 1)])
@pytest.mark.parametrize("d,width", [(64, 6), (128, 40)])
def test_shared_and_selected_canaries(d, width, dtype, D, hq, hkv):
    a, g, gd = _attn(), gen(3), Guarded()
    lens = torch.tensor([width * 64 - 3, 0, 200, 64, 129], dtype=torch.int32).cuda()
    cache = make_cache(g, 3 * width, hkv, d)
    c = _guarded_cache(gd, cache)
    table = torch.randint(0, 3 * width, (5, width), generator=g, dtype=torch.int32).cuda()
    table[:3, :2] = table[:1, :2].clone()
    q = randn(g, 5, D, hq, d, dtype=dtype).cuda()
    code = 1 if dtype == BF else 0
    out, lse = gd.empty((5, D, hq, d), dtype), gd.empty((5, D, hq), F32)
    start, shared = torch.tensor([0, 3, 5], dtype=torch.int32).cuda(), torch.tensor([2, 0], dtype=torch.int32).cuda()
    ws = gd.workspace(a.decode_shared_workspace_bytes(hq, hkv, d, code, 5, D, width, 2))
    a.decode_shared(q, c, lens, table, start, shared, out, lse=lse, workspace=ws)
    gd.check()
    heads = torch.randint(0, 3 * width, (5, hkv, width), generator=g, dtype=torch.int32).cuda()
    ws = gd.workspace(a.decode_workspace_bytes(hq, hkv, d, code, 5, D, width, False))
    a.decode_selected(q, c, a.Selected(lens, heads, None), out, lse=lse, workspace=ws)
    gd.check()
    for got, want in zip((c.k_pages, c.v_pages), cache[:2]):
        assert torch.equal(got.view(torch.uint8).cpu(), want)


@pytest.mark.parametrize("d,hkv", [(32, 3), (128, 2)])
def test_summary_and_selection_canaries(d, hkv):
    a, g, gd = _attn(), gen(4), Guarded()
    cache = make_cache(g, 40, hkv, d)
    c = _guarded_cache(gd, cache)
    s = a.KeySummary(gd.empty((40, hkv, 2, d), torch.int8), gd.empty((40, hkv), F32))
    table = torch.arange(40, dtype=torch.int32).flip(0).view(2, 20).cuda()
    lens = [1279, 600]
    a.summarise(c, s, cu_of(lens).cuda(), sum(lens), torch.zeros(2, dtype=torch.int32).cuda(), table)
    gd.check()
    held = torch.tensor(lens, dtype=torch.int32).cuda()
    q = randn(g, 2, 2, 3 * hkv, d).bfloat16().cuda()
    import ctypes
    for budget in (6, 25):
        lo, to, io = gd.empty((2,), torch.int32), gd.empty((2, hkv, budget), torch.int32), gd.empty((2, hkv, budget), torch.int32)
        need = a._lib.kda_cache_select_workspace_bytes(ctypes.byref(a.make_dims(3 * hkv, hkv, d, 1)), 2, 20)
        ws = gd.workspace(need)
        ks = a.KdaKeySummary(s.bounds.data_ptr(), s.unit.data_ptr())
        assert a._lib.kda_cache_select(ctypes.byref(a.make_dims(3 * hkv, hkv, d, 1)), ctypes.byref(ks), 40, 2, 2, q.data_ptr(),
                                       3 * hkv * d, held.data_ptr(), table.data_ptr(), 20, budget, 1, 2, lo.data_ptr(), to.data_ptr(),
                                       io.data_ptr(), ws.data_ptr(), need, None, torch.cuda.current_stream().cuda_stream) == 0
        gd.check()
        assert (to[..., :min(budget, 10)] >= 0).all()
