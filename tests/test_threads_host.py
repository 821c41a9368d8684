"""First calls made by two threads at once: what the library looks up on first use is complete
for the second thread too. No GPU: the look-ups are slowed down by stand-ins."""

import os
import shutil
import subprocess
import threading

import pytest

import tenant_serving_b200 as bd
from tenant_serving_b200 import _lib, build

ENCODER = r"""
#include <cuda.h>
#include <cuda_runtime.h>

#include <chrono>
#include <cstdio>
#include <thread>

static int entry_point;
// stands in for the driver's look-up: it takes a while
static cudaError_t slow_entry_point(const char*, void** p, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  std::this_thread::sleep_for(std::chrono::milliseconds(300));
  *p = &entry_point;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
#define cudaGetDriverEntryPoint slow_entry_point
#include "bd_tc.cuh"

int main() {
  bool found[8];
  std::thread t[8];
  for (int i = 0; i < 8; ++i)
    t[i] = std::thread([&found, i] {
      std::this_thread::sleep_for(std::chrono::milliseconds(20 * i));
      found[i] = bd::tensor_map_encoder() != nullptr;
    });
  int n = 0;
  for (int i = 0; i < 8; ++i) {
    t[i].join();
    n += found[i];
  }
  std::printf("%d\n", n);
  return n == 8 ? 0 : 1;
}
"""


def test_tensor_map_encoder(tmp_path):
    nvcc = build.nvcc_path()
    if shutil.which(nvcc) is None and not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "encoder.cu"
    src.write_text(ENCODER)
    exe = tmp_path / "encoder"
    subprocess.run([nvcc, *build.ARCH, "-std=c++17", "-I", build.CSRC, "-o", str(exe), str(src)], check=True,
                   capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert (r.returncode, r.stdout.strip()) == (0, "8")


class _SlowTorch:
    """torch whose attributes take a while: a second thread gets in between any two of them."""

    def __init__(self, torch, step):
        self._torch, self._step = torch, step

    def __getattr__(self, name):
        self._step()
        return getattr(self._torch, name)


def test_what_the_4_bit_calls_keep(monkeypatch):
    import torch
    monkeypatch.setattr(_lib, "_FP4", {})
    seen, failed = [], []

    def other():
        try:
            seen.append(_lib._fp4_code(torch.zeros(1, dtype=torch.bfloat16)))
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    def step():
        if _lib._FP4:  # the first thread is not done, the others already take it for complete
            t = threading.Thread(target=other)
            t.start()
            t.join()

    monkeypatch.setattr(_lib, "_torch", lambda: _SlowTorch(torch, step))
    assert _lib._fp4_code(torch.zeros(1, dtype=torch.float32)) == bd.BD_F32
    other()
    assert not failed and seen and set(seen) == {bd.BD_BF16}
