"""Numbers asked of a device, kept for each device and kernel (csrc/device_once.h on the host, over
a cudaGetDevice of the test's own), and that what is kept belongs to one kernel."""

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
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

static gqa::DeviceAnswers<3> one, other;
static int asked = 0;
static int get(gqa::DeviceAnswers<3>& a, int dev, int i, int says, cudaError_t e = cudaSuccess) {
  current = dev;
  return a.get(i, [&](int& n) { ++asked; n = says; return e; });
}

int main() {
  CHECK(get(one, 0, 0, 76) == 76 && asked == 1);
  CHECK(get(one, 0, 0, 5) == 76 && asked == 1);                              // kept
  CHECK(get(one, 0, 1, 36) == 36 && get(one, 0, 2, 0) == 0 && asked == 3);   // each question for itself
  CHECK(get(one, 0, 2, 9) == 0 && asked == 3);                               // (none is an answer too)
  CHECK(get(other, 0, 0, 14) == 14 && asked == 4);                           // another kernel's is another
  CHECK(get(one, 1, 0, 20) == 20 && asked == 5 && get(one, 0, 0, 1) == 76);  // another device's too
  CHECK(get(other, 2, 1, 50, cudaErrorInvalidValue) == 0 && asked == 6);     // a failure counts as none,
  CHECK(get(other, 2, 1, 51) == 51 && asked == 7 && get(other, 2, 1, 8) == 51);  // and is not kept
  CHECK(get(one, 200, 0, 3) == 3 && get(one, 200, 0, 4) == 4 && get(one, -1, 0, 6) == 6);
  answer = cudaErrorNoDevice;
  asked = 0;
  CHECK(get(one, 0, 0, 7) == 0 && asked == 0);
  answer = cudaSuccess;
  CHECK(get(one, 0, 0, 7) == 76);
  std::vector<std::thread> threads;
  for (int t = 0; t < 16; ++t)
    threads.emplace_back([] {
      for (int d = 10; d < 60; ++d) {
        current = d;
        one.get(d % 3, [&](int& n) { n = d; return cudaSuccess; });
      }
    });
  for (auto& t : threads) t.join();
  for (int d = 10; d < 60; ++d) CHECK(get(one, d, d % 3, -1) == d);
  std::printf("ok\n");
  return 0;
}
"""


def test_answers_belong_to_a_device_and_a_kernel(tmp_path):
    src, exe = tmp_path / "answers.cpp", tmp_path / "answers"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, "-isystem", cuda, str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert (out.returncode, out.stdout.strip()) == (0, "ok")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))), ids=os.path.basename)
def test_nothing_is_kept_by_a_kernels_type(path):
    """A function over a kernel's type is the same one for all kernels with the same parameters: what it
    keeps would be the first one's."""
    text = open(path).read()
    for m in re.finditer(r"template <typename Kern[^>]*>\n(.*?)\n}\n", text, re.S):
        assert not re.search(r"^\s*static (?!constexpr)", m.group(1), re.M), m.group(1)[:80]
