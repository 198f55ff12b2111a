"""CPU checks of the largest sizes that the long-context entry points take."""
from test_attn_abi import P, _dims, attn  # noqa: F401
from test_attn_long_abi import _cache, _lib


def test_rotation_refuses_tokens_that_its_rounds_would_count_past_31_bits(attn):  # noqa: F811
    d = _dims(attn)
    for T in ((1 << 31) - 1, (1 << 31) - (1 << 14)):
        assert _lib().kda_norm_rotate(d, T, P, 512, P, 128, P, P, 64, 0, 1.0, P, None, 1e-6, P, 512, P, 128, None) == -1


def test_shared_refuses_more_rows_or_groups_than_it_counts(attn):  # noqa: F811
    lib = _lib()
    for heads, batch, D, groups in ((65535, 1, 1, 1 << 20), (4096, 2, 1, 1 << 20), (65535, 1 << 13, 16, 1)):
        d = _dims(attn, hq=heads, hkv=heads)
        assert lib.kda_attn_decode_shared_workspace_bytes(d, batch, D, 4, groups) == 0
        assert lib.kda_attn_decode_shared(d, _cache(attn), batch, D, P, heads * 64, P, P, 4, groups, P, P, P, None, P, 1 << 50,
                                          None, None) == -1
    assert lib.kda_attn_decode_shared_workspace_bytes(_dims(attn, hq=2048, hkv=2048), 2, 1, 4, 1 << 20) > 0
