"""Weights far below a row's largest, whose values count because the largest meets a value of zero (as a first token that
takes nearly all attention does)."""

import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu


def cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def sink_case(d, dtype, gap, at, keys, before=0.0):
    """40 queries over `keys` keys; key `at` scores `gap` nats above the others and has a value of zero. Where `before` is
    not 0, key 0 scores that much and has a value of zero too."""
    g = torch.Generator().manual_seed(d + at + int(gap))
    q = 0.4 / d ** 0.5 * torch.randn(40, 1, d, generator=g)
    k = torch.randn(keys, 1, d, generator=g)
    v = torch.randn(keys, 1, d, generator=g)
    q[..., 0], k[..., 0] = 1.0, 0.0
    k[0, 0, 0] = before
    k[at, 0, 0] = gap
    v[at] = 0.0
    if before:
        v[0] = 0.0
    return (x.to(dtype).cuda() for x in (q, k, v))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("gap", [10.0, 12.0, 14.0, 16.0])
@pytest.mark.parametrize("at,before", [(0, 0.0), (70, 0.0), (200, 0.0), (200, 10.0)])
def test_prefill_small_weights_keep_their_bits(at, before, gap, d, dtype):
    """f16 has steps of 2^-24 below 2^-14, and the row's largest weight is 2^7 at least, so a weight is off by up to 2^-32
    of the largest besides its relative error of 2^-11: that adds 2^-32 / 2^-11 = 2^-21 of p_max sum_j |v_j| to A."""
    from expert_major_chunked_gb300 import attention
    keys = 260
    q, k, v = sink_case(d, dtype, gap, at, keys, before)
    out, lse = attention.prefill(q, k, v, cu([40]), cu([keys]), scale=1.0)
    attention.raise_on_device_error()
    want, wlse, a, dd = ref.prefill(q, k, v, [40], [keys], 1.0)
    if dtype == torch.float16:
        for i in range(40):
            n = keys - 40 + i + 1
            a[i, 0] += 2.0 ** -21 * v[:n, 0].double().abs().sum(0).cpu()  # (p_max is at most 1)
    ref.check(out, lse, (want, wlse, a, dd), ref.U[dtype])
