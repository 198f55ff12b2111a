"""CPU checks of the attention binding's look at devices: a tensor on another GPU
or on the host is refused before anything is launched.  The tensors are stand-ins
that say where they are; no call here reaches the library."""
import pytest
import torch


class Stand:
    """What the binding asks of a tensor."""

    def __init__(self, shape, dtype, dev=0):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, dev
        self.is_cuda, self.device = dev >= 0, f"cuda:{dev}"

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.dtype.itemsize

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 4096

    def on(self, dev):
        return Stand(self.shape, self.dtype, dev)


class Library:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was reached")
        return call


@pytest.fixture
def attn(monkeypatch):
    from gated_delta_rule_decode_gb300 import build
    build.build()
    from gated_delta_rule_decode_gb300 import attn as mod
    monkeypatch.setattr(mod, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return mod


BF, F32, I32, F8, U8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn, torch.uint8
CACHE = dict(k_pages=Stand((5, 2, 64, 64), F8), v_pages=Stand((5, 2, 64, 64), F8), k_scale=Stand((5, 2), F32),
             v_scale=Stand((5, 2), F32))
FLAG = dict(err_flag=Stand((1,), I32))
CALLS = {
    "prefill": dict(q=Stand((9, 4, 64), BF), k=Stand((9, 2, 64), BF), v=Stand((9, 2, 64), BF), cu_seqlens=Stand((3,), I32),
                    out=Stand((9, 4, 64), BF), lse=Stand((9, 4), F32), **FLAG),
    "append": dict(**CACHE, k=Stand((9, 2, 64), BF), v=Stand((9, 2, 64), BF), cu_seqlens=Stand((3,), I32),
                   start_pos=Stand((2,), I32), block_table=Stand((2, 4), I32), **FLAG),
    "decode": dict(**CACHE, q=Stand((2, 3, 4, 64), BF), seq_lens=Stand((2,), I32), block_table=Stand((2, 4), I32),
                   out=Stand((2, 3, 4, 64), BF), lse=Stand((2, 3, 4), F32), weight_in=Stand((2, 4), F32),
                   weight_out=Stand((2, 4), F32), workspace=Stand((1 << 20,), U8), **FLAG),
    "evict": dict(seq_lens=Stand((2,), I32), block_table=Stand((2, 4), I32), weight=Stand((2, 4), F32), **FLAG),
}


def _call(attn, name, args, **more):
    args = dict(args)
    if "k_pages" in args:
        args["cache"] = attn.KVCache(*(args.pop(x) for x in attn.KVCache._fields))
    if name == "evict":
        args.update(budget=2, in_place=True)
    return getattr(attn, name)(**args, **more)


@pytest.mark.parametrize("name,arg", [(n, a) for n, args in CALLS.items() for a in args])
@pytest.mark.parametrize("dev", [1, -1])
def test_a_tensor_elsewhere_is_refused(attn, name, arg, dev):
    args = dict(CALLS[name])
    args[arg] = args[arg].on(dev)
    with pytest.raises(ValueError, match=arg.split("_pages")[0]):
        _call(attn, name, args)


@pytest.mark.parametrize("name", CALLS)
def test_a_call_for_another_gpu_is_refused(attn, name):
    """All on cuda:1 while cuda:0 is current, or the stream is of another GPU."""
    with pytest.raises(ValueError, match="cuda:1"):
        _call(attn, name, {k: v.on(1) for k, v in CALLS[name].items()})

    class Stream:
        device_index = 1
        cuda_stream = 0
    with pytest.raises(ValueError, match="cuda:1"):
        _call(attn, name, CALLS[name], stream=Stream())


@pytest.mark.parametrize("flag", [Stand((1,), torch.int64), Stand((0,), I32)])
def test_the_error_flag_is_looked_at(attn, flag):
    for name, args in CALLS.items():
        with pytest.raises(ValueError, match="err_flag"):
            _call(attn, name, dict(args, err_flag=flag))
