"""A kernel's limit of dynamic shared memory with two host threads that ask for different sizes at once: the limit that the
library remembers is never above the one that the kernel has.  The header's function runs against a stand-in for the CUDA
runtime, whose setter lets the second thread in (if nothing keeps it out) before the first one's call returns."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_74_gb300", "csrc")

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include <cuda_runtime.h>
// (the overload for kernels that nvcc's headers have)
static cudaError_t cudaFuncSetAttribute(void (*kernel)(), cudaFuncAttribute attribute, int value) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), attribute, value);
}
#include "sv_ops.h"

static std::atomic<int> limit{0}, sets{0}, device{0};
static std::atomic<bool> large_in{false}, small_in{false};

extern "C" {
cudaError_t CUDARTAPI cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t CUDARTAPI cudaFuncSetAttribute(const void*, cudaFuncAttribute, int value) {
  ++sets;
  limit = value;
  if (value == 160000) {
    large_in = true;
    for (int i = 0; i < 300 && !small_in; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
    std::this_thread::sleep_for(std::chrono::milliseconds(50));  // the other thread notes its size first
  } else {
    small_in = true;
  }
  return cudaSuccess;
}
}

void kernel() {}

int main() {
  std::thread large([] { (void)sv::allow_smem<kernel>(160000); });
  std::thread small([] {
    while (!large_in) std::this_thread::yield();
    (void)sv::allow_smem<kernel>(80000);
  });
  large.join();
  small.join();
  (void)sv::allow_smem<kernel>(160000);  // what a large call does before its launch
  std::printf("limit %d\n", limit.load());
  if (limit < 160000) return 1;
  const int before = sets;
  (void)sv::allow_smem<kernel>(90000);
  if (sets != before) return 2;          // (less than the kernel has: nothing to set)
  device = 1;                            // another device has a limit of its own
  (void)sv::allow_smem<kernel>(90000);
  if (sets != before + 1 || limit != 90000) return 3;
  device = sv::kMaxDevices;              // and one past those that are remembered is set at every call
  (void)sv::allow_smem<kernel>(70000);
  (void)sv::allow_smem<kernel>(70000);
  return sets == before + 3 ? 0 : 4;
}
"""


def test_two_threads_with_two_sizes(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc) or shutil.which("g++") is None:
        pytest.skip("needs g++ and the CUDA headers")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    source, program = tmp_path / "limit.cpp", tmp_path / "limit"
    source.write_text(PROGRAM)
    built = subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", include, "-I", CSRC, str(source), "-o", str(program)],
                           capture_output=True, text=True)
    assert built.returncode == 0, built.stderr
    ran = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert ran.returncode == 0, (ran.returncode, ran.stdout)
