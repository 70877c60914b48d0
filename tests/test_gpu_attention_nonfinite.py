"""NaN and infinities in keys and values, hidden and seen, against the 64-bit reference (attention_reference.py)."""

import math

import pytest
import torch

import attention_reference as ref
from test_gpu_attention_prefill import cu, inputs

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


def check_rows(got, want, rows, dtype):
    """The given rows (a list of token numbers) of a call's results against the reference's."""
    out, lse = got
    o, z, a, d = want
    ref.check(out[rows], lse[:, rows], (o[rows], z[:, rows], a[rows], d[:, rows]), ref.U[dtype])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hq,hk", [(64, 1, 1), (64, 6, 2), (128, 1, 1), (128, 7, 1), (128, 130, 1), (256, 2, 2),
                                     (256, 16, 1)])
def test_one_bad_value_reaches_no_row_that_does_not_see_it(d, hq, hk, dtype, bad):
    """One element of one value (or a whole key and value), at every kind of place in its tile: rows before it are as the
    reference has them for finite inputs, to the bounds of one result. The next sequence's first row and the rows behind the
    last one are such values as well."""
    from expert_major_chunked_gb300 import attention
    lens = [420, 60] if hq < 100 else [150, 20]
    n = lens[0]
    q, k, v = inputs(lens, lens, hq, hk, d, dtype)
    k, v = (torch.cat([x, torch.full((40, hk, d), bad, dtype=dtype, device="cuda")]) for x in (k, v))
    want = ref.prefill(q, k[:sum(lens)], v[:sum(lens)], lens, lens, 1 / math.sqrt(d))
    for at in (1, 15, 16, 100, 127, 128, n - 130, n - 1, n):
        k2, v2 = k.clone(), v.clone()
        if at == n:  # the next sequence's first key
            k2[at], v2[at] = bad, bad
        else:
            v2[at, hk - 1, at % d] = bad
        got = attention.prefill(q, k2, v2, cu(lens), scale=1 / math.sqrt(d))
        attention.raise_on_device_error()
        check_rows(got, want, list(range(min(at, n))) + (list(range(n, sum(lens))) if at < n else []), dtype)
        if at < n:  # rows that see it: that channel of the last kv head's query heads is not finite, the others are right
            seen, heads = slice(at, n), slice(hq - hq // hk, hq)
            assert not torch.isfinite(got[0][seen, heads, at % d]).any()
            keep = [i for i in range(d) if i != at % d]
            o, z, a, dd = want
            ref.check(got[0][seen][..., keep], got[1][:, seen], (o[seen][..., keep], z[:, seen], a[seen][..., keep],
                                                                dd[:, seen]), ref.U[dtype])


def test_seen_nan_scores_make_the_row_nan():
    from expert_major_chunked_gb300 import attention
    for d in (64, 128, 256):
        q, k, v = inputs([200], [200], 4, 2, d, torch.bfloat16)
        k[50, 0, 3] = math.nan
        out, lse = attention.prefill(q, k, v, cu([200]))
        assert out[50:, :2].isnan().all() and lse[:2, 50:].isnan().all()
        assert torch.isfinite(out[:50]).all() and torch.isfinite(out[:, 2:]).all() and torch.isfinite(lse[2:]).all()


def test_sums_that_pass_float32_while_the_reference_maximum_lags():
    """Values of 2^115 in bf16: 300 of them with weights of nearly 2^8 pass float32's range, with weights up to 1 they do
    not. Keys score 5.5 nats (2^7.9) above the first one, too little for the running reference to follow."""
    from expert_major_chunked_gb300 import attention
    for d in (64, 128, 256):
        q = torch.zeros(20, 1, d, dtype=torch.bfloat16, device="cuda")
        k = torch.zeros(320, 1, d, dtype=torch.bfloat16, device="cuda")
        v = (2.0 ** 115 * (1 + torch.rand(320, 1, d, generator=torch.Generator().manual_seed(d)))).to(torch.bfloat16).cuda()
        q[..., 0], k[128:, 0, 0] = 1.0, 5.5
        out, lse = attention.prefill(q, k, v, cu([20]), cu([320]), scale=1.0)
        ref.check(out, lse, ref.prefill(q, k, v, [20], [320], 1.0), ref.U[torch.bfloat16])


def ms(call):
    call()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    call()
    b.record()
    b.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("where", ["an early value", "behind the last key", "the last value"])
def test_bad_values_cost_some_tiles_not_a_pass_over_all_keys_for_each_row(where):
    """The rows that are computed again take what several tiles take: ten times the clean call is asked for. Rows that
    see the value keep what they have, and looking for it costs less than the call."""
    from expert_major_chunked_gb300 import attention
    n, extra = 16022, 100
    q, k, v = inputs([n], [n + extra], 16, 2, 128, torch.bfloat16)
    ends = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    v[{"an early value": 3, "behind the last key": n + 5, "the last value": n - 1}[where], :, 7] = math.nan
    clean = ms(lambda: attention.prefill(q, k[:n], torch.nan_to_num(v[:n]), ends))
    taken = ms(lambda: attention.prefill(q, k, v, ends))
    attention.raise_on_device_error()
    print(f"{where}: {taken:.2f} ms, clean {clean:.2f} ms")
    assert taken < 10 * clean


@pytest.mark.parametrize("d", [64, 128, 256])
def test_more_tiles_with_such_rows_than_a_block_of_the_kernel_takes(d):
    """1300 sequences of six tokens, the last value of each NaN, on 8 heads: tens of tiles an SM have rows to be computed
    again."""
    from expert_major_chunked_gb300 import attention
    lens, h = [6] * 1300, 8
    q, k, v = inputs(lens, lens, h, h, d, torch.bfloat16)
    want = ref.prefill(q, k, v, lens, lens, 1 / math.sqrt(d))
    v[5::6] = math.nan
    got = attention.prefill(q, k, v, cu(lens), scale=1 / math.sqrt(d))
    attention.raise_on_device_error()
    assert got[0][5::6].isnan().all()
    check_rows(got, want, [i for i in range(sum(lens)) if i % 6 != 5], torch.bfloat16)
