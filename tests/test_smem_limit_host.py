"""Host threads whose first calls need different amounts of shared memory: the limit that
a kernel is left with, against a stand-in for the runtime's call. No GPU is used."""

import os
import subprocess

from speculative_decoding_tree_build_gb300.build import CSRC, NVCC_FLAGS, _nvcc

PROGRAM = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <thread>
#include "tv_common.cuh"

// The runtime's limit of one kernel. The large call's return is held back until the small
// call is through, as far as it comes (half a second at most).
static std::mutex m;
static std::condition_variable changed;
static int limit = 0, calls = 0;
static bool large_set = false, small_done = false;
constexpr int kLarge = 81920, kSmall = 20;

extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int value) {
  std::unique_lock<std::mutex> held(m);
  ++calls;
  if (value == kSmall) changed.wait_for(held, std::chrono::milliseconds(500), [] { return large_set; });
  limit = value;
  if (value == kLarge) {
    large_set = true;
    changed.notify_all();
    changed.wait_for(held, std::chrono::milliseconds(500), [] { return small_done; });
  }
  return cudaSuccess;
}

static void kernel() {}
static tv::SmemLimit limits;

int main() {
  auto need = [](int bytes) { return tv::ensure_smem(kernel, bytes, limits, 3); };
  std::thread large([&] { need(kLarge); });
  std::thread small([&] {
    {
      std::unique_lock<std::mutex> held(m);          // the large call has passed its first check
      changed.wait_for(held, std::chrono::milliseconds(500), [] { return large_set; });
    }
    need(kSmall);
    const std::lock_guard<std::mutex> held(m);
    small_done = true;
    changed.notify_all();
  });
  large.join();
  small.join();
  need(kLarge);
  need(kSmall);
  std::printf("%d %d\n", limit, calls);
  return 0;
}
"""



def test_the_largest_limit_stays(tmp_path):
    source, program = tmp_path / "limit.cu", tmp_path / "limit"
    source.write_text(PROGRAM)
    nvcc = _nvcc()
    lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")
    subprocess.run([nvcc, *NVCC_FLAGS, "-I", CSRC, "-cudart", "shared", "-Xlinker", "-rpath=" + lib, "-o", str(program),
                    str(source), "-lpthread"], check=True, capture_output=True)
    out = subprocess.run([str(program)], check=True, capture_output=True, text=True, timeout=60).stdout
    limit, calls = out.split()
    assert int(limit) == 81920 and int(calls) <= 2
