"""Further refusals of the attention operators (test_attention_host.py has the others). No GPU needed."""

import ctypes

import pytest

from test_attention_host import L, decode_args, prefill_args  # noqa: F401  (L is a fixture)

APART = [dict(out_token=0), dict(out_head=0), dict(out_token=56), dict(out_head=56), dict(out_token=0, out_head=0)]


@pytest.mark.parametrize("change", APART)
def test_rows_of_out_must_lie_apart(L, change):  # noqa: F811
    for f, args in ((L.moe_attn_prefill, prefill_args), (L.moe_attn_decode, decode_args)):
        assert f(ctypes.byref(args(**change)), None) == -1
        assert b"apart" in L.moe_prefill_last_error()


def test_the_stride_of_one_row_says_nothing(L):  # noqa: F811
    """One token, or one head: whatever its stride, the call is not refused for it (without a GPU it ends later)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real")
    for change in (dict(out_token=0), dict(out_head=0, n_heads=1, n_kv_heads=1)):
        one = {**change, "total_q": 1} if "out_token" in change else change
        assert L.moe_attn_prefill(ctypes.byref(prefill_args(**one)), None) in (-4, -6)
        one = {**change, "n_requests": 1} if "out_token" in change else change
        assert L.moe_attn_decode(ctypes.byref(decode_args(**one)), None) in (-4, -6)
