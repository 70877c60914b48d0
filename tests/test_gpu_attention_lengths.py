"""Lengths at the ends of their types and tensors without rows."""

import math

import pytest
import torch

import attention_reference as ref
import test_gpu_kv_cache as kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,columns", [(64, 1 << 24), (128, (1 << 24) + 5), (256, 1 << 24)])
def test_decode_lengths_up_to_the_last_int32(d, columns):
    """A length of 2^31 - 1 with a table that covers it: its first and last blocks hold tokens, the others lie outside the
    cache. A length past the table's end is clipped to it; the other request is an ordinary one."""
    from expert_major_chunked_gb300 import attention
    bs, hq, hk, top = 128, 4, 2, (1 << 31) - 1
    q, dev, small, _, host = kv.decode_case([2 * bs - 1, 100], hq, hk, d, bs)
    kc, vc, ks, vs, _ = host
    table = torch.full((2, columns), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, (1 << 24) - 1], table[1, 0] = small[0, 0], small[0, 1], small[1, 0]
    out, lse = attention.decode(q, dev, table, kv.ints([top, 100]))
    want = ref.decode(q, kc, vc, ks, vs, small.cpu(), [2 * bs - 1, 100], 1 / math.sqrt(d))
    ref.check(out, lse.T, want, ref.U[torch.float16])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_without_any_keys(d, dtype):
    """Queries and not one key in the call: zeros and lse = -inf."""
    from expert_major_chunked_gb300 import attention
    q, none = torch.ones(70, 4, d, dtype=dtype, device="cuda"), torch.empty(0, 2, d, dtype=dtype, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((4, 70), 7.0, device="cuda")
    attention.prefill(q, none, none, kv.ints([0, 30, 30, 70]), kv.ints([0, 0, 0, 0]), out=out, lse=lse)
    attention.raise_on_device_error()
    assert not out.any() and (lse == -math.inf).all()
