"""The attention kernels' bounded waits: a library whose waits give up after
one poll (see test_gpu_timeout.py) returns, reports KDA_DEVERR_TIMEOUT and
leaves the context usable."""
import pytest
import torch

from attn_testutil import cu_of, gen, make_cache, randn, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def variant(tmp_path_factory):
    import ctypes

    from gated_delta_rule_decode_gb300 import attn, build
    path = build.build(force=True, extra_flags=["-DKDA_WAIT_LIMIT=1", "-DKDA_WAIT_NONBLOCKING"],
                       out_path=str(tmp_path_factory.mktemp("waitlimit") / "libkda_wait1.so"))
    return attn._declare(ctypes.CDLL(path))


def _with_lib(lib, fn):
    from gated_delta_rule_decode_gb300 import attn
    saved = attn._lib
    attn._lib = lib
    try:
        return fn()
    finally:
        attn._lib = saved


@pytest.mark.parametrize("d", [64, 128])
def test_waits_give_up_and_the_context_stays_usable(variant, d):
    from gated_delta_rule_decode_gb300 import attn, kda
    g = gen(1)
    q, k, v = (randn(g, 900, h, d).bfloat16().cuda() for h in (8, 2, 2))
    cu = cu_of([700, 200]).cuda()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = attn.prefill(q, k, v, cu, err_flag=flag)
    assert flag.item() == 0
    _with_lib(variant, lambda: attn.prefill(q, k, v, cu, err_flag=flag))
    torch.cuda.synchronize()
    assert flag.item() == kda.KDA_DEVERR_TIMEOUT
    assert torch.equal(attn.prefill(q, k, v, cu), want)

    c = to_device(make_cache(g, 40, 2, d))
    table = torch.arange(40, dtype=torch.int32).view(2, 20).cuda()
    lens = torch.tensor([1280, 700], dtype=torch.int32).cuda()
    # 28 rows of a kv head: the converter-fed kernel, whose roles wait for one
    # another; 4 and 8: a warp waits only for copies that it issued a page ago,
    # which have usually landed, and the call returns either way
    for D, flags in ((7, (kda.KDA_DEVERR_TIMEOUT,)), (1, (0, kda.KDA_DEVERR_TIMEOUT)), (2, (0, kda.KDA_DEVERR_TIMEOUT))):
        qd = randn(g, 2, D, 8, d).bfloat16().cuda()
        flag.zero_()
        want = attn.decode(qd, c, lens, table, err_flag=flag)
        assert flag.item() == 0
        _with_lib(variant, lambda: attn.decode(qd, c, lens, table, err_flag=flag))
        torch.cuda.synchronize()
        assert flag.item() in flags
        assert torch.equal(attn.decode(qd, c, lens, table), want)
