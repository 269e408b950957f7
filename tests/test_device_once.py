"""Kernel attributes belong to a device: csrc/device_once.h on the host, over a
cudaGetDevice of the test's own, and that every launcher goes through it."""

import glob
import os
import re
import subprocess

import pytest

from gqa_attention_kv_decode_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "device_once.h"

static thread_local int current = 0;
static thread_local cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = current; return answer; }

static int ran[4], failing = -1;
static gqa::DeviceOnce once;
static cudaError_t use(int dev) {
  current = dev;
  return once.run([&] {
    ++ran[dev < 4 ? dev : 3];
    return dev == failing ? cudaErrorInvalidValue : cudaSuccess;
  });
}
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  CHECK(use(0) == cudaSuccess && use(0) == cudaSuccess && ran[0] == 1);
  CHECK(use(1) == cudaSuccess && ran[1] == 1);               // a second device is set up too
  CHECK(use(0) == cudaSuccess && ran[0] == 1);
  failing = 2;                                               // a failure is this device's alone
  CHECK(use(2) == cudaErrorInvalidValue && use(0) == cudaSuccess && use(1) == cudaSuccess);
  failing = -1;                                              // and is not kept
  CHECK(use(2) == cudaSuccess && ran[2] == 2 && use(2) == cudaSuccess && ran[2] == 2);
  CHECK(use(200) == cudaSuccess && use(200) == cudaSuccess && ran[3] == 2);
  answer = cudaErrorNoDevice;
  CHECK(once.run([] { return cudaSuccess; }) == cudaErrorNoDevice);
  answer = cudaSuccess;
  static gqa::DeviceOnce many;
  std::vector<int> count(8, 0);                              // each entry is touched under the lock
  std::vector<std::thread> threads;
  for (int t = 0; t < 16; ++t)
    threads.emplace_back([&, t] {
      for (int d = 0; d < 8; ++d) {
        current = (d + t) % 8;
        many.run([&] { ++count[current]; return cudaSuccess; });
      }
    });
  for (auto& t : threads) t.join();
  for (int n : count) CHECK(n == 1);
  std::printf("ok\n");
  return 0;
}
"""


def test_setup_runs_once_on_each_device(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, "-isystem", cuda, str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert (out.returncode, out.stdout.strip()) == (0, "ok")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(build.CSRC, "*.cu"))), ids=os.path.basename)
def test_launchers_set_attributes_per_device(path):
    """No attribute is set once for the whole process."""
    text = open(path).read()
    assert "call_once" not in text
    calls = [m.start() for m in re.finditer(r"cudaFuncSetAttribute\(", text)]
    starts = [m.start() for m in re.finditer(r"once\.run\(\[&\] \{", text)]
    for at in calls:
        before = [s for s in starts if s < at]
        assert before and "});" not in text[before[-1]:at]
