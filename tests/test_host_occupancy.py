"""The cached count of CTAs that an SM holds (csrc/fs_host.h) goes by the shared memory asked for,
in any order of calls; checked on the CPU with a runtime that answers by arithmetic."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "streaming_sinkhorn_b200/csrc/fs_host.h"
static int device = 0, asked = 0;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaGetLastError() { return cudaSuccess; }
extern "C" cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int,
                                                                     size_t smem) {
  ++asked;
  *n = static_cast<int>(227 * 1024 / (smem ? smem : 1));
  return cudaSuccess;
}
int main() {
  fs::PerDeviceOccupancy o;
  const size_t sizes[] = {68 * 1024, 35 * 1024, 68 * 1024, 35 * 1024, 35 * 1024, 113 * 1024};
  for (int d = 0; d < 2; ++d) {
    device = d;
    for (size_t s : sizes)
      if (o.get(nullptr, 256, s) != static_cast<int>(227 * 1024 / s)) {
        std::printf("device %d, %zu bytes: %d\n", d, s, o.get(nullptr, 256, s));
        return 1;
      }
  }
  const int before = asked;
  for (int i = 0; i < 100; ++i) o.get(nullptr, 256, 113 * 1024);
  return asked == before ? 0 : 2;  // the same question is asked once
}
"""


def test_occupancy_goes_by_shared_memory(tmp_path):
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    if not shutil.which("g++") or not os.path.exists(os.path.join(cuda, "include", "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    src, exe = tmp_path / "occupancy.cpp", tmp_path / "occupancy"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", ROOT, "-I", os.path.join(cuda, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
