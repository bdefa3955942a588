"""The once-per-device setting of a kernel's shared-memory limit, compiled against a stand-in of the runtime."""
import os
import shutil
import subprocess

import pytest

from bit_nf4_quantized_linear_gb300 import build

PROGRAM = r"""
#include "smem_limit.h"
#include <cstdio>
#include <thread>
#include <vector>

static thread_local int device = 0;
static int sets[128], failing = -1;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) {
  if (device == failing) return cudaErrorInvalidValue;
  __atomic_fetch_add(&sets[device], 1, __ATOMIC_RELAXED);
  return cudaSuccess;
}
static void kernel() {}
static int check(bool ok, const char* what) {
  if (!ok) std::printf("%s\n", what);
  return ok ? 0 : 1;
}
int main() {
  nf4::SmemLimit limit;
  int bad = 0;
  for (int round = 0; round < 3; ++round)
    for (device = 0; device < 100; ++device) bad += check(limit.allow(kernel, 1000) == cudaSuccess, "allow");
  for (int d = 0; d < 64; ++d) bad += check(sets[d] == 1, "once a device");
  for (int d = 64; d < 100; ++d) bad += check(sets[d] == 3, "beyond the flags: each time");
  nf4::SmemLimit other;
  failing = device = 3;
  bad += check(other.allow(kernel, 1000) == cudaErrorInvalidValue, "a failure is reported");
  failing = -1;
  bad += check(other.allow(kernel, 1000) == cudaSuccess && sets[3] == 2, "and tried again");
  nf4::SmemLimit shared;
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&, t] {
      device = t;
      for (int i = 0; i < 1000; ++i) shared.allow(kernel, 1000);
    });
  for (auto& t : threads) t.join();
  for (int d = 0; d < 8; ++d) bad += check(sets[d] == (d == 3 ? 3 : 2), "threads on devices of their own");
  return bad;
}
"""


def test_limit_is_set_once_a_device(tmp_path):
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    if shutil.which("g++") is None or not os.path.exists(os.path.join(cuda, "cuda_runtime_api.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", build.CSRC, "-I", cuda, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_no_launch_keeps_a_limit_for_the_whole_process():
    """The limit belongs to a device's context: every launcher that sets it goes through SmemLimit or sets it each time."""
    for f in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, f)) as h:
            text = h.read()
        assert "static bool configured" not in text and "atomic<bool> configured" not in text, f
