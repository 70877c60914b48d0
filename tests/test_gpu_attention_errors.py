"""Errors that another call of the program has left behind are not a call's own, and none is left behind."""

import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

# A check that waits for its stream fails while the stream is being captured (on the host; nothing reaches the GPU). The
# layer's check leaves that error with the runtime, the attention operators' check takes it along.
PROGRAM = """
import ctypes, sys
sys.path.insert(0, {root!r})
import torch
from expert_major_chunked_gb300 import attention, binding, workloads

rt = ctypes.CDLL("libcudart.so." + torch.version.cuda.split(".")[0])
dev = torch.device("cuda")
wl = workloads.WORKLOADS["tiny"]
inp = {{k: v.to(dev) for k, v in workloads.generate(wl).items()}}
layer = binding.MoePrefill({{k: inp[k] for k in ("w_router", "w_gu", "w_down", "ws_gu", "ws_down")}}, top_k=wl.top_k,
                           max_chunk=16)
want_y = layer.run(inp["x"], 16)
q = torch.randn(3, 4, 64, device=dev).to(torch.bfloat16)
k = q[:, :2].contiguous()
cu = torch.tensor([0, 3], dtype=torch.int32, device=dev)
cache = attention.KvCache.empty(4, 2, 16, 64)
one, none = torch.ones(1, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
free, table = torch.arange(4, dtype=torch.int32, device=dev), torch.full((1, 4), -1, dtype=torch.int32, device=dev)


def calls():
    s = attention.assign_slots(none, 3 * one, free, table, 16, 3)
    attention.append(k, k, s.slot_map, cache)
    return (*attention.prefill(q, k, k, cu), *attention.decode(q[:1], cache, table, s.kv_lens))


def fail(check):
    stream = torch.cuda.Stream()
    graph = ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(ctypes.c_void_p(stream.cuda_stream), 1) == 0
    try:
        check(stream)
        raise SystemExit("the check did not fail")
    except binding.MoeError as e:
        assert e.status == -4, e  # MOE_ERR_CUDA
    assert rt.cudaStreamEndCapture(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph)) != 0
    rt.cudaGetLastError()  # (of the runtime that torch uses; the library has its own)


want = calls()
torch.cuda.synchronize()
for check in ({checks}):
    fail(check)
    {after}
torch.cuda.synchronize()
print("done")
"""


def run(checks, after):
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(root=ROOT, checks=checks, after=after)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr


def test_an_error_that_is_there_is_not_the_calls_own():
    run("layer.raise_on_device_error,", "assert all(torch.equal(a, b) for a, b in zip(calls(), want))")


def test_a_call_that_fails_leaves_no_error():
    run("attention.raise_on_device_error,", "assert torch.equal(layer.run(inp['x'], 16), want_y)")


def test_refusals_name_the_argument():
    """What the calls on tensors do not take, with the argument that is to blame in the message."""
    import torch

    import test_gpu_kv_cache as kv
    from expert_major_chunked_gb300 import attention
    q, dev, table, lens, _ = kv.decode_case([5, 7], 4, 2, 64, 16)
    x, cu, slots = q[:, :2].contiguous(), kv.ints([0, 2]), kv.ints([0, 1], torch.int64)
    for name, call in (
            ("cache", lambda: attention.decode(q, list(dev), table, lens)),
            ("cache", lambda: attention.append(x, x, slots, list(dev))),
            ("cache", lambda: attention.append(x, x, slots, dev[:3])),
            ("v_scale", lambda: attention.append(x, x, slots, dev._replace(v_scale=1.0))),
            ("scale", lambda: attention.prefill(q, x, x, cu, scale="x")),
            ("scale", lambda: attention.decode(q, dev, table, lens, scale=[1.0])),
            ("block_size", lambda: attention.assign_slots(lens, lens, lens, table, 16.0, 4)),
            ("block_size", lambda: attention.assign_slots(lens, lens, lens, table, -16, 4)),
            ("max_tokens", lambda: attention.assign_slots(lens, lens, lens, table, 16, 1 << 31)),
            ("max_tokens", lambda: attention.assign_slots(lens, lens, lens, table, 16, None)),
            ("k", lambda: attention.prefill(q, None, x, cu)), ("out", lambda: attention.prefill(q, x, x, cu, out=3)),
            ("lse", lambda: attention.decode(q, dev, table, lens, lse=3)),
            ("workspace", lambda: attention.decode(q, dev, table, lens, workspace=3)),
            ("slot_map", lambda: attention.append(x, x, [0, 1], dev)),
            ("kv_lens", lambda: attention.decode(q, dev, table, [5, 7]))):
        with pytest.raises(ValueError, match=rf"\b{name}\b"):
            call()
    with pytest.raises(ValueError, match="below 2"):
        attention.assign_slots(lens[:1].expand(1 << 31), lens, lens, table, 16, 4)
