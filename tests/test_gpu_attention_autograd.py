"""What autograd is told: there is no backward pass, and tensors are changed in place."""

import pytest
import torch

import test_gpu_kv_cache as kv

pytestmark = pytest.mark.gpu


def test_gradients_through_the_results_raise():
    from expert_major_chunked_gb300 import attention
    q, dev, table, lens, _ = kv.decode_case([5, 7], 4, 2, 64, 16)
    x, cu = q[:, :2].contiguous(), kv.ints([0, 2])
    want_p, want_d = attention.prefill(q, x, x, cu), attention.decode(q, dev, table, lens)
    assert not any(t.requires_grad for t in (*want_p, *want_d))
    w, y = q.clone().requires_grad_(), x.clone().requires_grad_()
    for stream in (None, torch.cuda.Stream()):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        calls = (lambda: attention.prefill(w * 1, x, x, cu, stream=stream), lambda: attention.prefill(q, y, x, cu, stream=stream),
                 lambda: attention.prefill(q, x, y, cu, stream=stream), lambda: attention.decode(w, dev, table, lens, stream=stream))
        for call, want in zip(calls, (want_p, want_p, want_p, want_d)):
            got = call()
            torch.cuda.synchronize()
            for r, expected in zip(got, want):
                assert r.requires_grad and torch.equal(r, expected)
                with pytest.raises(RuntimeError, match="no backward pass"):
                    r.float().sum().backward()
            with torch.no_grad():
                assert not any(r.requires_grad for r in call())
            with torch.inference_mode():
                assert not any(r.requires_grad for r in call())
            torch.cuda.synchronize()
    assert w.grad is None and y.grad is None


def test_given_buffers_have_no_gradient():
    from expert_major_chunked_gb300 import attention
    q, dev, table, lens, _ = kv.decode_case([5, 7], 4, 2, 64, 16)
    want = attention.decode(q, dev, table, lens)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    got = attention.decode(q.clone().requires_grad_(), dev, table, lens, out=out)
    assert got[0] is out and not out.requires_grad and got[1].requires_grad and torch.equal(out, want[0])
    got = attention.decode(q.clone().requires_grad_(), dev, table, lens, out=out, lse=lse)
    assert got[0] is out and got[1] is lse and torch.equal(lse, want[1])


def test_changes_in_place_are_counted():
    """Backward passes of other operators find out that a tensor which they saved has changed."""
    from expert_major_chunked_gb300 import attention
    q, dev, table, lens, _ = kv.decode_case([5, 7], 4, 2, 64, 16)
    x, slots = q[:, :2].contiguous(), kv.ints([3, 19], torch.int64)
    out, lse = attention.decode(q, dev, table, lens)
    before = [t._version for t in (out, lse, table, *dev, q, lens)]
    attention.decode(q, dev, table, lens, out=out, lse=lse)
    attention.assign_slots(lens, lens, lens, table, 16, 4)
    attention.append(x, x, slots, dev)
    after = [t._version for t in (out, lse, table, *dev, q, lens)]
    assert [b > a for a, b in zip(before, after)] == [True] * 7 + [False] * 2
    p, z = attention.prefill(q, x, x, kv.ints([0, 2]))
    versions = p._version, z._version
    attention.prefill(q, x, x, kv.ints([0, 2]), out=p, lse=z)
    assert p._version > versions[0] and z._version > versions[1]
    with torch.inference_mode():
        a, b = attention.decode(q, dev, table, lens)
    attention.decode(q, dev, table, lens, out=a, lse=b)  # tensors made in inference mode count nothing
    a = torch.ones(3, 64, device="cuda", requires_grad=True)
    scale = dev.k_scale
    y = (a[:2, :2] * scale[:2]).sum()
    attention.append(x, x, slots, dev)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
