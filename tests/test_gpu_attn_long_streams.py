"""The entry points of long contexts on another stream: what they allocate is
that stream's memory (see test_gpu_attn_streams.py), two of them at once do not
meet, and a captured one replays."""
import pytest
import torch

from attn_testutil import gen, make_cache, randn, to_device

pytestmark = pytest.mark.gpu


def _calls():
    from gated_delta_rule_decode_gb300 import attn as a
    g = gen(82)
    cache = to_device(make_cache(g, 12, 2, 64))
    table = torch.arange(12, dtype=torch.int32).view(3, 4)
    table[1, :2] = table[0, :2]
    table = table.cuda()
    lens = torch.tensor([200, 170, 256], dtype=torch.int32).cuda()
    start, shared = torch.tensor([0, 2, 3], dtype=torch.int32).cuda(), torch.tensor([2, 0], dtype=torch.int32).cuda()
    summary = a.alloc_summary(cache)
    a.summarise(cache, summary, torch.tensor([0, 256, 512, 768], dtype=torch.int32).cuda(), 768,
                torch.zeros(3, dtype=torch.int32).cuda(), table)
    qd = randn(g, 3, 1, 4, 64).bfloat16().cuda()
    q, k = randn(g, 300, 4, 64).bfloat16().cuda(), randn(g, 300, 2, 64).bfloat16().cuda()
    pos = torch.arange(300, dtype=torch.int32).cuda()
    rot = a.rotary(a.rotary_frequencies(64))
    sel = a.select(qd, summary, lens, table, 3)
    return {
        "norm_rotate": lambda s: a.norm_rotate(q, k, pos, rot, stream=s),
        "decode_shared": lambda s: a.decode_shared(qd, cache, lens, table, start, shared, return_lse=True, stream=s),
        "select": lambda s: tuple(a.select(qd, summary, lens, table, 3, stream=s)),
        "decode_selected": lambda s: a.decode_selected(qd, cache, sel, return_lse=True, stream=s),
    }


NAMES = ["norm_rotate", "decode_shared", "select", "decode_selected"]


@pytest.mark.parametrize("name", NAMES)
def test_dropped_results_stay_with_their_stream(name):
    call = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(s)
    held = [(t.data_ptr(), t.shape, t.dtype) for t in got]
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    del got, x, y
    for ptr, shape, dtype in held:
        again = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(8)]
        assert ptr not in [t.data_ptr() for t in again]
    with torch.cuda.stream(s):
        again = call(s)
    assert {t.data_ptr() for t in again} & {ptr for ptr, _, _ in held}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_current_stream_is_not_taken(name):
    call = _calls()[name]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    freed = [t.data_ptr() for t in call(None)]
    got = call(s)
    assert not set(freed) & {t.data_ptr() for t in got}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_two_calls_at_once_and_captured(name):
    call = _calls()[name]
    want = call(None)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [call(streams[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    for outs in got:
        for x, y in zip(outs, want):
            assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(None)
    for t in held:
        t.fill_(7)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(held, want):
        assert torch.equal(x, y)
