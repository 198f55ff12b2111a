"""CPU checks of the largest sizes that the long-context entry points take."""
from test_attn_abi import P, _dims, attn  # noqa: F401
from test_attn_long_abi import _cache, _lib


def test_rotation_refuses_tokens_that_its_rounds_would_count_past_31_bits(attn):  # noqa: F811
    d = _dims(attn)
    for T in ((1 << 31) - 1, (1 << 31) - (1 << 14)):
        assert _lib().kda_norm_rotate(d, T, P, 512, P, 128, P, P, 64, 0, 1.0, P, None, 1e-6, P, 512, P, 128, None) == -1
