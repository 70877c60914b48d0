"""Prompts of ordinary size, call after call: every call's results against float64 on the GPU, and the same bytes each time.
(What goes wrong only at some meeting of the kernel's roles does not show in small prompts.)"""

import math

import pytest
import torch

import attention_reference as ref
from test_gpu_attention_prefill import cu

pytestmark = pytest.mark.gpu


def whole_reference(q, k, v, q_lens, k_lens):
    """What attention_reference.prefill gives, a head of a sequence at a time on the GPU."""
    scale, g = 1 / math.sqrt(q.shape[2]), q.shape[1] // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, a = torch.zeros_like(q), torch.zeros_like(q)
    lse, d = (torch.full((q.shape[1], q.shape[0]), x, dtype=torch.float64, device="cuda") for x in (-math.inf, 0.0))
    q0 = k0 = 0
    for ql, kl in zip(q_lens, k_lens):
        hidden = torch.arange(kl, device="cuda")[None] > torch.arange(ql, device="cuda")[:, None] + kl - ql
        for h in range(q.shape[1]):
            qq, kk, vv = q[q0:q0 + ql, h], k[k0:k0 + kl, h // g], v[k0:k0 + kl, h // g]
            s = (qq @ kk.T * scale).masked_fill_(hidden, -math.inf)
            lse[h, q0:q0 + ql] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[h, q0:q0 + ql, None])
            out[q0:q0 + ql, h], a[q0:q0 + ql, h] = p @ vv, p @ vv.abs()
            big = (qq.abs() @ kk.abs().T * scale).masked_fill_(hidden, 0.0).amax(1)
            d[h, q0:q0 + ql] = big * (q.shape[2] + 16) * 2.0 ** -23
        q0, k0 = q0 + ql, k0 + kl
    return out.cpu(), lse.cpu(), a.cpu(), d.cpu()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,hq,hk", [(64, 16, 4), (128, 16, 2), (256, 16, 2), (256, 4, 4)])
@pytest.mark.parametrize("q_lens,k_lens", [([3001], [3001]), ([700, 1, 1500, 64], [700, 300, 1500, 2100])])
def test_call_after_call(q_lens, k_lens, d, hq, hk, dtype):
    from expert_major_chunked_gb300 import attention
    g = torch.Generator(device="cuda").manual_seed(d)
    sets = []
    for _ in range(2):
        q, k, v = (torch.randn(t, h, d, generator=g, device="cuda").to(dtype)
                   for t, h in ((sum(q_lens), hq), (sum(k_lens), hk), (sum(k_lens), hk)))
        sets.append((q, k, v, cu(q_lens), cu(k_lens)))
    results = []
    for _ in range(40):  # nothing waits between the calls
        for args in sets:
            results.append(attention.prefill(*args))
    attention.raise_on_device_error()
    for i, args in enumerate(sets):
        ref.check(*results[i], whole_reference(*args[:3], q_lens, k_lens), ref.U[dtype])
        for out, lse in results[i::2]:
            assert torch.equal(out, results[i][0]) and torch.equal(lse, results[i][1])
