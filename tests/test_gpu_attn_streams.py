"""What a call on another stream allocates is that stream's memory: a dropped
result or scratch is not handed to the current stream while the call may still
write it, and memory that the current stream still uses is not handed to it."""
import pytest
import torch

from attn_testutil import cu_of, gen, make_cache, randn, to_device

pytestmark = pytest.mark.gpu


def _calls():
    from gated_delta_rule_decode_gb300 import attn as a
    g = gen(81)
    q, k, v = (randn(g, 300, h, 64).bfloat16().cuda() for h in (4, 2, 2))
    cu = cu_of([200, 100]).cuda()
    c = to_device(make_cache(g, 12, 2, 64))
    table = torch.arange(12, dtype=torch.int32).view(3, 4).cuda()
    lens = torch.tensor([200, 70, 256], dtype=torch.int32).cuda()
    w = torch.rand(3, 4, generator=g).cuda()
    qd = randn(g, 3, 2, 4, 64).bfloat16().cuda()
    return {
        "prefill": lambda s: a.prefill(q, k, v, cu, return_lse=True, stream=s),
        "decode": lambda s: a.decode(qd, c, lens, table, return_lse=True, weight_in=w, stream=s),
        "evict": lambda s: tuple(a.evict(lens, table, w, 2, 0, 1, stream=s)),
    }


@pytest.mark.parametrize("name", ["prefill", "decode", "evict"])
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
    # and the stream itself gets them again: they are its own
    with torch.cuda.stream(s):
        again = call(s)
    assert {t.data_ptr() for t in again} & {ptr for ptr, _, _ in held}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["prefill", "decode", "evict"])
def test_memory_of_the_current_stream_is_not_taken(name):
    """Blocks of every size that the call asks for, freed on the current stream, where work on them may be queued."""
    call = _calls()[name]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    freed = [t.data_ptr() for t in call(None)]
    got = call(s)
    assert not set(freed) & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
