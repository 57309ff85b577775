"""The launchers' shared-memory limit (csrc/smem_limit.h) on the host, against a fake runtime: once
per kernel and device, the device's most, from whichever thread; and no launcher sets its own."""

import glob
import os
import subprocess

from conftest import ROOT

CSRC = os.path.join(ROOT, "decode_gemv_epilogue_gb300", "csrc")

FAKE = r"""
#pragma once
typedef int cudaError_t;
enum { cudaSuccess = 0, cudaErrorUnknown = 999 };
enum { cudaDevAttrMaxSharedMemoryPerBlockOptin = 97, cudaFuncAttributeMaxDynamicSharedMemorySize = 8 };
struct cudaFuncAttributes { unsigned long sharedSizeBytes; };
cudaError_t cudaGetDevice(int*);
cudaError_t cudaDeviceGetAttribute(int*, int, int);
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes*, const void*);
cudaError_t cudaFuncSetAttribute(const void*, int, int);
"""

MAIN = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "smem_limit.h"
static thread_local int device = 0;
static std::atomic<int> sets{0}, last{0}, failures{0};
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, int, int) { *v = 232448; return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* f, const void*) { f->sharedSizeBytes = 128; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, int, int v) {
  if (failures.load() > 0) { --failures; return cudaErrorUnknown; }
  std::this_thread::yield();
  ++sets;
  last = v;
  return cudaSuccess;
}
#define CHECK(c) if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; }
int main() {
  static gf::SmemLimit limit;
  failures = 1;
  CHECK(limit.raise(nullptr) == cudaErrorUnknown);  // not remembered
  std::vector<std::thread> t;
  std::atomic<int> bad{0};
  for (int i = 0; i < 16; ++i)
    t.emplace_back([&, i] {
      device = i % 2;
      for (int j = 0; j < 100; ++j) bad += limit.raise(nullptr) != cudaSuccess;
    });
  for (auto& x : t) x.join();
  CHECK(bad == 0 && sets == 2 && last == 232448 - 128);
  device = 70;  // beyond the table: set each time, to the same
  CHECK(limit.raise(nullptr) == cudaSuccess && limit.raise(nullptr) == cudaSuccess && sets == 4 && last == 232448 - 128);
  return 0;
}
"""


def test_limit_is_raised_once(tmp_path):
    (tmp_path / "cuda_runtime.h").write_text(FAKE)
    (tmp_path / "main.cc").write_text(MAIN)
    exe = str(tmp_path / "t")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", str(tmp_path), "-I", CSRC, str(tmp_path / "main.cc"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_no_launcher_sets_a_limit_of_its_own():
    users = [f for f in glob.glob(os.path.join(CSRC, "*")) if "MaxDynamicSharedMemorySize" in open(f).read()]
    assert [os.path.basename(f) for f in users] == ["smem_limit.h"]
