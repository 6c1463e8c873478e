"""State that belongs to a device (a kernel's shared-memory attribute, its occupancy, the multiprocessor count) is
kept by device and not by process.  The host code is compiled against a stand-in for the runtime's current device,
so no GPU is needed."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from block_diffusion_speculative_target_gb300 import build

MAIN = r"""
#include "per_device.h"
#include <cstdio>
#include <thread>
#include <vector>
static thread_local int current = 0;
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = current; return answer; }
#define EXPECT(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
  static dfl::PerDevice smem, sms, shared;
  std::vector<int> set(80, 0);
  auto once = [&](int dev) { current = dev; return smem.once([&] { ++set[dev]; return cudaSuccess; }); };
  for (int rep = 0; rep < 3; ++rep)
    for (int dev : {0, 1, 63, 5}) EXPECT(once(dev) == cudaSuccess);
  EXPECT(set[0] == 1 && set[1] == 1 && set[63] == 1 && set[5] == 1 && set[2] == 0);
  for (int rep = 0; rep < 3; ++rep) EXPECT(once(64) == cudaSuccess);  // past the table: every time
  EXPECT(set[64] == 3);
  // a failure is told and not kept, on its device alone
  current = 7;
  EXPECT(smem.once([] { return cudaErrorInvalidValue; }) == cudaErrorInvalidValue);
  EXPECT(once(7) == cudaSuccess && set[7] == 1);
  answer = cudaErrorNoDevice;
  EXPECT(once(0) == cudaErrorNoDevice);
  answer = cudaSuccess;
  // values differ by device
  for (int rep = 0; rep < 2; ++rep)
    for (int dev : {3, 4}) {
      int n = 0;
      current = dev;
      EXPECT(sms.get(&n, [&](int d, int* v) { *v = rep == 0 ? 100 + d : -1; return cudaSuccess; }) == cudaSuccess);
      EXPECT(n == 100 + dev);
    }
  // from several threads
  std::vector<std::thread> threads;
  std::atomic<int> wrong{0};
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&, t] {
      current = t % 4;
      for (int i = 0; i < 1000; ++i) {
        int n = 0;
        if (shared.get(&n, [](int d, int* v) { *v = d + 1; return cudaSuccess; }) != cudaSuccess || n != t % 4 + 1) ++wrong;
      }
    });
  for (auto& t : threads) t.join();
  EXPECT(wrong == 0);
  std::puts("ok");
}
"""


def test_per_device(tmp_path):
    gxx = shutil.which("g++")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    if not gxx or not os.path.exists(os.path.join(include, "cuda_runtime_api.h")):
        pytest.skip("needs g++ and the toolkit's headers")
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(MAIN)
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", str(src), "-o", str(exe), "-I", build.CSRC, "-I", include],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_no_launch_keeps_a_flag_of_the_process():
    """Every kernel attribute is set through PerDevice, and no function remembers that it was."""
    found = 0
    for path in glob.glob(os.path.join(build.CSRC, "*.cu")):
        text = open(path).read()
        for m in re.finditer("cudaFuncSetAttribute", text):
            found += 1
            assert re.search(r"\.(once|get)\([^;]*$", text[:m.start()]), (path, text[m.start() - 200:m.start()])
        assert not re.search(r"static (bool|int) \w+ = (false|0)[;,]\s*(\\\s*)?\n\s*if \(", text), path
    assert found >= 4
