"""csrc/device_once.h by itself, with a fake cudaGetDevice (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "device_once.h"
#include <cstdio>
#include <thread>
#include <vector>
static thread_local int g_device = 0;
static cudaError_t g_status = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = g_device; return g_status; }
#define NEED(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
  dlm::DeviceOnce once;
  int calls = 0;
  cudaError_t result = cudaErrorMemoryAllocation;
  auto f = [&] { ++calls; return result; };
  NEED(once.get(f) == cudaErrorMemoryAllocation && calls == 1);
  NEED(once.get(f) == cudaErrorMemoryAllocation && calls == 2);   // tried again
  result = cudaSuccess;
  NEED(once.get(f) == cudaSuccess && calls == 3);
  result = cudaErrorInvalidValue;
  NEED(once.get(f) == cudaSuccess && calls == 3);                 // remembered
  g_device = 63;
  NEED(once.get(f) == cudaErrorInvalidValue && calls == 4);       // each device by itself
  result = cudaSuccess;
  NEED(once.get(f) == cudaSuccess && once.get(f) == cudaSuccess && calls == 5);
  for (int d : {64, -1}) {
    g_device = d;
    NEED(once.get(f) == cudaErrorInvalidDevice && calls == 5);
  }
  g_device = 1;
  g_status = cudaErrorNoDevice;
  NEED(once.get(f) == cudaErrorNoDevice && calls == 5);
  g_status = cudaSuccess;
  std::vector<std::thread> all;
  for (int i = 0; i < 8; ++i)
    all.emplace_back([&] { g_device = 2; for (int j = 0; j < 1000; ++j) once.get(f); });
  for (auto& t : all) t.join();
  NEED(calls == 6);
  std::puts("fine");
}
"""


def test_device_once(tmp_path):
    if shutil.which("g++") is None or not os.path.exists("/usr/local/cuda/include/cuda_runtime.h"):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I/usr/local/cuda/include",
                    "-I" + os.path.join(ROOT, "masked_block_diffusion_denoise_b200", "csrc"), str(src),
                    "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "fine\n", r.stdout
