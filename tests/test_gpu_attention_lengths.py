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


def test_prefill_tiles_that_take_seconds():
    """2^29 keys, rows 16 bytes apart in one buffer: the only tile takes several seconds, in which most of the kernel's
    roles wait. One key near the end takes all the weight (the others score 200 nats less)."""
    from expert_major_chunked_gb300 import attention
    n, d, key = 1 << 29, 64, (1 << 29) - 6
    x = torch.zeros(8 * n + 3 * d, dtype=torch.bfloat16, device="cuda")
    k, v = x.as_strided((n, 1, d), (8, d, 1)), x.as_strided((n, 1, d), (8, d, 1), 2 * d)
    x[8 * key] = 200.0                       # dimension 0 of this key only
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    v[key] = torch.arange(d, device="cuda")  # (it lies past the end of the keys' 64 values)
    assert k[key + 1:, 0, 0].abs().max() <= d and k[key, 0, 0] == 200
    out, lse = attention.prefill(q, k, v, kv.ints([0, 1]), kv.ints([0, n]), scale=1.0)
    attention.raise_on_device_error()
    assert torch.equal(out[0, 0], v[key, 0]) and abs(lse.item() - 200.0) < 1e-3


@pytest.mark.parametrize("bs", [1 << 30, (1 << 29) + 5])
def test_assign_slots_of_positions_past_int32(bs):
    """A request that passes 2^31 tokens: positions stop at 2^31 - 1, slots go on in the next block."""
    from expert_major_chunked_gb300 import attention
    top = (1 << 31) - 1
    ctx, new, mb = top - 4, 10, 6
    held = -(-ctx // bs)
    table = kv.ints([[3 + i if i < held else -1 for i in range(mb)]])
    s = attention.assign_slots(kv.ints([ctx]), kv.ints([new]), kv.ints([20, 21, 22]), table, bs, 12)
    row = [3 + i for i in range(held)] + [20] * (-(-(ctx + new) // bs) - held)
    at = range(ctx, ctx + new)
    assert table[0].tolist() == row + [-1] * (mb - len(row))
    assert s.positions.tolist() == [min(p, top) for p in at] + [-1, -1]
    assert s.slot_map.tolist() == [row[p // bs] * bs + p % bs for p in at] + [-1, -1]
    assert s.kv_lens.tolist() == [top] and s.cu_new.tolist() == [0, new]


@pytest.mark.parametrize("bs", [16, 128])
def test_append_up_to_the_last_int32(bs):
    """2^31 - 1 tokens (one row, expanded), all without a slot but the first and the last ones."""
    from expert_major_chunked_gb300 import attention
    n, d = (1 << 31) - 1, 64
    dev, small = (attention.KvCache.empty(4, 1, bs, d) for _ in range(2))
    row = torch.randn(1, 1, d, generator=torch.Generator().manual_seed(bs)).to(torch.bfloat16).cuda()
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    ends = [bs + 1, bs + 2, 2 * bs, 2 * bs + 1, 2 * bs + 2]
    slots[:2], slots[-3:] = kv.ints(ends[:2], torch.int64), kv.ints(ends[2:], torch.int64)
    attention.append(row.expand(n, 1, d), row.expand(n, 1, d), slots, dev)
    attention.append(row.expand(5, 1, d), row.expand(5, 1, d), kv.ints(ends, torch.int64), small)
    for a, b in zip(dev, small):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert dev.k.float()[1, 0, 1:3].abs().sum() > 0 and dev.k.float()[2, 0, :3].abs().sum() > 0
