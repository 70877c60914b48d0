"""What is set up once for each device: the helper on the CPU with a stand-in for the runtime, the calls on a second
device where there is one."""

import os
import subprocess

import pytest
import torch

from conftest import ROOT

PROGRAM = r"""
#include "attn.h"
#include <cstdio>

static int current;
extern "C" cudaError_t cudaGetDevice(int* dev) { *dev = current; return current < 0 ? cudaErrorNoDevice : cudaSuccess; }

#define EXPECT(x) if (!(x)) { std::printf("line %d: " #x "\n", __LINE__); return 1; }

int main() {
  static moe::OncePerDevice once;
  int calls = 0;
  cudaError_t answer = cudaErrorMemoryAllocation;
  auto prepare = [&] { ++calls; return answer; };
  EXPECT(once(prepare) == cudaErrorMemoryAllocation && calls == 1);
  EXPECT(once(prepare) == cudaErrorMemoryAllocation && calls == 2);  // a failure is not kept
  answer = cudaSuccess;
  EXPECT(once(prepare) == cudaSuccess && calls == 3);
  EXPECT(once(prepare) == cudaSuccess && calls == 3);
  for (int dev = 1; dev < 64; ++dev) {  // every device is prepared, once
    current = dev;
    EXPECT(once(prepare) == cudaSuccess && calls == 3 + dev);
    EXPECT(once(prepare) == cudaSuccess && calls == 3 + dev);
  }
  current = 64;
  EXPECT(once(prepare) == cudaErrorInvalidDevice && calls == 66);
  current = -1;
  EXPECT(once(prepare) == cudaErrorNoDevice && calls == 66);
  return 0;
}
"""


def test_every_device_is_prepared_and_failures_are_tried_again(tmp_path):
    from expert_major_chunked_gb300 import build
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", f"-I{build.CSRC}", f"-I{os.path.join(cuda, 'include')}", str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
def test_calls_on_a_second_device():
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    from expert_major_chunked_gb300 import attention
    results = []
    for dev in ("cuda:0", "cuda:1"):
        g = torch.Generator().manual_seed(1)
        q, k, v = (torch.randn(70, h, 128, generator=g).to(torch.bfloat16).to(dev) for h in (4, 2, 2))
        cu = torch.tensor([0, 70], dtype=torch.int32, device=dev)
        cache = attention.KvCache.empty(8, 2, 16, 128, device=dev)
        attention.append(k, v, torch.arange(70, device=dev), cache)
        table = torch.arange(5, dtype=torch.int32, device=dev)[None]
        results.append([x.cpu() for x in (*attention.prefill(q, k, v, cu),
                                          *attention.decode(q[-1:], cache, table, cu[1:]))])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_the_error_check_runs_on_the_streams_device(monkeypatch):
    """Its word is the current device's, which need not be the stream's. (Stand-ins for torch's device switch, the
    stream and the library.)"""
    from types import SimpleNamespace

    from expert_major_chunked_gb300 import attention
    current, asked = ["cuda:0"], []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, current[0] = current[0], self.device

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(attention._b, "lib", lambda: SimpleNamespace(
        moe_attn_check=lambda stream: asked.append((current[0], stream)) or 0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(device="cuda:0", cuda_stream=7))
    attention.raise_on_device_error(SimpleNamespace(device="cuda:1", cuda_stream=5))
    attention.raise_on_device_error()
    assert asked == [("cuda:1", 5), ("cuda:0", 7)] and current == ["cuda:0"]
