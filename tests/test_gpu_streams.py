"""What a KDA call on another stream allocates is that stream's memory (see
test_gpu_attn_streams.py)."""
import pytest
import torch

from gated_delta_rule_decode_gb300 import inputs

pytestmark = pytest.mark.gpu


def _calls():
    from gated_delta_rule_decode_gb300 import kda
    x = inputs.decode_inputs(4, 2, 128, 128, num_slots=6, seed=1, device="cuda")
    y = inputs.verify_inputs(4, 3, 2, 128, 128, num_slots=6, seed=2, device="cuda")
    z = inputs.prefill_inputs([100, 30], 2, 128, 128, num_slots=4, seed=3, device="cuda")

    def flat(out, rec):
        return (out,) + tuple(rec.values())
    return {
        "decode": lambda s: (kda.decode(x.q, x.k, x.v, x.g, x.b, x.slot_ids, x.pool.clone(), stream=s),),
        "verify": lambda s: flat(*kda.verify_record(y.q, y.k, y.v, y.g, y.b, y.slot_ids, y.pool, stream=s)),
        "verify_u": lambda s: flat(*kda.verify_record_u(y.q, y.k, y.v, y.g, y.b, y.slot_ids, y.pool, stream=s)),
        "prefill": lambda s: (kda.prefill_chunked(z.q, z.k, z.v, z.g, z.b, z.cu_seqlens, z.slot_ids, z.pool, stream=s),),
    }


@pytest.mark.parametrize("name", ["decode", "verify", "verify_u", "prefill"])
def test_dropped_results_stay_with_their_stream(name):
    call = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(s)  # (the pool's copy too is of this stream)
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    got = None
    if name != "decode":
        got = call(s)  # from another current stream
        s.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        taken = {t.data_ptr() for t in got}
        shapes = [(t.shape, t.dtype) for t in got]
        del got, x, y
        fresh = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(8)]
        assert not taken & {t.data_ptr() for t in fresh}


def test_a_prepared_call_holds_its_results_on_its_stream():
    from gated_delta_rule_decode_gb300 import kda
    x = inputs.decode_inputs(4, 2, 128, 128, num_slots=6, seed=1, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty_like(x.v) for _ in range(4)]
    ptrs = {t.data_ptr() for t in freed}
    del freed
    run = kda.decode(x.q, x.k, x.v, x.g, x.b, x.slot_ids, x.pool.clone(), stream=s, _prepare=True)
    assert run.result.data_ptr() not in ptrs
