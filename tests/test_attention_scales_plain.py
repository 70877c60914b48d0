"""That the bound asked of decode attention tells weights scaled to 2^15 before they become f16 from weights of up to 1:
the kernel's arithmetic restated in 64 bits on the CPU, with the rounding of the weights to f16."""

import math

import pytest
import torch

import attention_reference as ref


def scales_apart(hq=4, hk=2, d=64, bs=16, n=200, seed=0):
    """A request whose tokens all weigh the same. Its blocks have, in turn, a V scale of 2^10 with codes of the smallest
    sizes and one of 1.3 * 2^-9 with the largest: values of the same size (2 and 4 against 1.14), weights times scale
    2^18.6 apart. With weights of up to 1 the small ones are 41.6 steps of f16 and round to 42, all of them by 1%."""
    g = torch.Generator().manual_seed(seed)
    blocks = -(-n // bs)
    q = torch.randn(1, hq, d, generator=g).to(torch.float16)
    kc, ks = torch.zeros(blocks, hk, bs, d, dtype=torch.float64), torch.ones(blocks, hk, dtype=torch.float64)
    small = 2.0 ** -9 * torch.randint(1, 3, kc.shape, generator=g).double()
    first = torch.arange(blocks) % 2 == 0
    vc = torch.where(first[:, None, None, None], small, 448.0).double()
    vs = torch.where(first[:, None], 2.0 ** 10, 1.3 * 2.0 ** -9).float().double().expand(blocks, hk).clone()
    return q, kc, vc, ks, vs, torch.arange(blocks)[None], [n]


def with_f16_weights(case, top):
    """One request's output with weights 2^(u + log2 sv - m + top) rounded to f16, m the largest exponent."""
    q, kc, vc, ks, vs, table, (n,) = case
    k, codes = ref.gather(kc, ks, table[0], n), ref.gather(vc, torch.ones_like(vs), table[0], n)
    sv = ref.gather(torch.ones_like(vc), vs, table[0], n)[..., 0]
    out, lse = torch.zeros(q.shape[1:], dtype=torch.float64), torch.zeros(q.shape[1], dtype=torch.float64)
    for h in range(q.shape[1]):
        kv = h // (q.shape[1] // k.shape[1])
        u = (k[:, kv] @ q[0, h].double()) / math.sqrt(q.shape[2]) * math.log2(math.e)
        e = u + torch.log2(sv[:, kv])
        p = torch.exp2(e - e.max() + top)
        l = (p / sv[:, kv]).sum()
        out[h] = p.to(torch.float16).double() @ codes[:, kv] / l
        lse[h] = (e.max() - top + torch.log2(l)) * math.log(2.0)
    return out[None].to(torch.float16), lse[:, None]


@pytest.mark.parametrize("top,passes", [(15, True), (0, False)])
def test_scales_apart_show_weights_that_lose_bits(top, passes):
    case = scales_apart()
    out, lse = with_f16_weights(case, top)
    want = ref.decode(*case, 1 / math.sqrt(64))
    if passes:
        ref.check(out, lse, want, ref.U[torch.float16])
    else:
        with pytest.raises(AssertionError, match="times the bound"):
            ref.check(out, lse, want, ref.U[torch.float16])
