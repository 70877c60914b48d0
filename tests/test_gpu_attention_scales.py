"""The cache's scales at their ends: zeros, and blocks of very different size."""

import math

import pytest
import torch

import attention_reference as ref
import test_gpu_kv_cache as kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("hq", [2, 24])
def test_a_v_scale_of_zero_leaves_its_block_out_whatever_its_codes_are(hq, bs, d):
    """Blocks whose V scale is 0 (or negative, or NaN) and whose codes are NaN, against a table without these blocks."""
    from expert_major_chunked_gb300 import attention
    lens = [9 * bs + 5, bs, 3 * bs - 1]
    q, dev, table, kv_lens, _ = kv.decode_case(lens, hq, 2, d, bs)
    without = table.clone()
    out_of = [(0, 0, 0.0), (0, 4, -1.0), (0, 5, math.nan), (0, 9, 0.0), (1, 0, 0.0), (2, 1, -0.0)]
    for b, i, scale in out_of:
        block = int(table[b, i])
        dev.v_scale[block] = scale
        for codes in dev[:2]:
            codes.view(torch.uint8)[block] = 0x7F
        without[b, i] = -1
    got, want = attention.decode(q, dev, table, kv_lens), attention.decode(q, dev, without, kv_lens)
    assert torch.isfinite(want[0]).all() and not want[0][1].any() and (want[1][1] == -math.inf).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,large", [(torch.float16, 60000.0), (torch.bfloat16, 2.0 ** 20)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_queries_with_one_large_channel(d, dtype, large):
    """One channel of the query is large where the keys have zeros, so that the scores come from the others: these keep
    their bits (the bound has no term for the conversion to f16: it is exact down to 2^-28 of the row's largest)."""
    from expert_major_chunked_gb300 import attention
    lens, hq, hk, bs = [150, 40], 4, 2, 16
    q, dev, table, kv_lens, (kc, vc, ks, vs, tt) = kv.decode_case(lens, hq, hk, d, bs, dtype, stale=False)
    g = torch.Generator().manual_seed(d)
    q = (0.25 * torch.randn(q.shape, generator=g)).to(dtype).cuda()
    q[..., 5] = large
    kc[..., 5] = 0.0
    dev.k.view(torch.uint8)[..., 5] = 0
    ks = torch.exp2(torch.randint(-2, 2, ks.shape, generator=g).double())
    dev = dev._replace(k_scale=ks.float().cuda())
    out, lse = attention.decode(q, dev, table, kv_lens)
    ref.check(out, lse.T, ref.decode(q, kc, vc, ks, vs, tt, lens, 1 / math.sqrt(d)), ref.U[torch.float16])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs,d", [(16, 64), (32, 128), (64, 256), (128, 128)])
@pytest.mark.parametrize("tokens", [1, 9, 300])
def test_append_behind_tokens_of_scale_zero(tokens, bs, d, dtype):
    """Blocks whose tokens have a scale of 0: their values are 0 whatever the codes, and stay 0 under the new scale."""
    from expert_major_chunked_gb300 import attention
    blocks = tokens + 3
    dev, *host = kv.cache(blocks, 2, bs, d)
    slots = ([b * bs + 7 for b in range(tokens)] if tokens < 10 else  # single tokens, or runs over blocks' borders
             [b * bs + 5 + i for b in range(0, 60) for i in range(5)])
    for scale, h in ((dev.k_scale, host[2]), (dev.v_scale, host[3])):
        scale[::2], h[::2] = 0.0, 0.0
    k, v = kv.rows(len(slots), 2, d, dtype, bs)
    attention.append(k, v, kv.ints(slots, torch.int64), dev)
    ref.append(k.cpu(), slots, host[0], host[2])
    ref.append(v.cpu(), slots, host[1], host[3])
    kv.same_cache(dev, *host)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("hq,hk", [(4, 2), (24, 2)])
def test_scales_apart(hq, hk, bs, d):
    """Blocks of a large V scale and small codes beside ones of a small scale and large codes, to the reference's own bound
    (test_attention_scales_plain.py shows that weights of up to 1 would not meet it)."""
    from expert_major_chunked_gb300 import attention
    from test_attention_scales_plain import scales_apart
    q, kc, vc, ks, vs, table, lens = scales_apart(hq, hk, d, bs, 900, d)
    dev = attention.KvCache(*(x.float().to(torch.float8_e4m3fn).cuda() for x in (kc, vc)),
                            *(x.float().cuda() for x in (ks, vs)))
    out, lse = attention.decode(q.cuda(), dev, table.int().cuda(), kv.ints(lens))
    ref.check(out, lse.T, ref.decode(q, kc, vc, ks, vs, table, lens, 1 / math.sqrt(d)), ref.U[torch.float16])


def test_scales_of_all_sizes_to_the_references_bound():
    """V scales from 2^-30 to 2^30, K scales that are no powers of two."""
    from expert_major_chunked_gb300 import attention
    for d, lens in ((64, [300, 77]), (128, [300, 77]), (256, [500])):
        q, dev, table, kv_lens, (kc, vc, ks, vs, tt) = kv.decode_case(lens, 4, 2, d, 16)
        g = torch.Generator().manual_seed(5)
        vs = torch.exp2(torch.randint(-30, 31, vs.shape, generator=g).double())
        ks = (ks * (1 + torch.rand(ks.shape, generator=g).double())).float().double()
        dev = dev._replace(v_scale=vs.float().cuda(), k_scale=ks.float().cuda())
        out, lse = attention.decode(q, dev, table, kv_lens)
        ref.check(out, lse.T, ref.decode(q, kc, vc, ks, vs, tt, lens, 1 / math.sqrt(d)), ref.U[torch.float16])
