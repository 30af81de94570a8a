"""The shared memory that a kernel is opted in to, when two host threads ask for different amounts at once:
prepare_launch compiled against a stand-in for the runtime's call (no GPU)."""
import subprocess

import pytest

from exact_io_aware_23_gb300 import _build

PROGRAM = r"""
#include <cuda.h>
#include <cuda_runtime.h>

#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>

static std::mutex mu;
static std::condition_variable cv;
static int attribute = 0;                  // what the runtime has been told last
static bool small_is_in = false, large_is_done = false;

static cudaError_t set_attribute(void (*)(), cudaFuncAttribute, int bytes) {
  std::unique_lock<std::mutex> lock(mu);
  if (bytes < 1000) {                      // the small request is overtaken by the large one, if that can be
    small_is_in = true;
    cv.notify_all();
    cv.wait_for(lock, std::chrono::milliseconds(500), [] { return large_is_done; });
  }
  attribute = bytes;
  large_is_done = large_is_done || bytes >= 1000;
  cv.notify_all();
  return cudaSuccess;
}
static cudaError_t get_device(int* d) { *d = 0; return cudaSuccess; }
#define cudaFuncSetAttribute set_attribute
#define cudaGetDevice get_device
#include "fa_sm103.cuh"

static void kernel() {}

int main() {
  static fa::LaunchSetup setup;
  std::thread small([] { fa::prepare_launch(setup, kernel, 16); });
  std::thread large([] {
    {
      std::unique_lock<std::mutex> lock(mu);
      cv.wait(lock, [] { return small_is_in; });
    }
    fa::prepare_launch(setup, kernel, 190000);
  });
  small.join();
  large.join();
  fa::prepare_launch(setup, kernel, 190000);
  std::printf("%d\n", attribute);
  fa::prepare_launch(setup, kernel, 100);  // never lowered
  std::printf("%d\n", attribute);
  return 0;
}
"""


def test_a_smaller_request_does_not_undo_a_larger_one(tmp_path):
    try:
        nvcc = _build._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    src, exe = tmp_path / "setup.cu", tmp_path / "setup"
    src.write_text(PROGRAM)
    r = subprocess.run([nvcc, *_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.INCLUDE, "-I", _build.CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout.split() == ["190000", "190000"], out
