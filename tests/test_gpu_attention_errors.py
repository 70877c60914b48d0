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
