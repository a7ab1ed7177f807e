"""A kernel's dynamic shared memory limit belongs to a device: a process that
launches on a second GPU has to set it there too.  Without a GPU: the library's
helper compiled against a stand-in for the two runtime calls that it makes."""

import glob
import os
import re
import subprocess

from head_split_kv_decode_b200 import build as BUILD

PROGRAM = r"""
#include "kernels.h"
#include <cstdio>
static int device = 0, sets = 0;
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { ++sets; return answer; }
static void kernel(int) {}
#define CHECK(x) if (!(x)) { std::printf("failed: %s\n", #x); return 1; }
int main() {
  static bool done[duo::kMaxDevices] = {};
  auto call = [&](int d) { device = d; return duo::allow_dynamic_smem(kernel, 100000, done); };
  CHECK(call(0) == cudaSuccess && sets == 1);
  CHECK(call(0) == cudaSuccess && sets == 1);       // once on a device
  CHECK(call(1) == cudaSuccess && sets == 2);       // and once on the next
  CHECK(call(0) == cudaSuccess && call(1) == cudaSuccess && sets == 2);
  answer = cudaErrorInvalidValue;
  CHECK(call(2) == cudaErrorInvalidValue && sets == 3);
  answer = cudaSuccess;
  CHECK(call(2) == cudaSuccess && sets == 4);       // a refusal is not remembered as done
  CHECK(call(2) == cudaSuccess && sets == 4);
  CHECK(call(duo::kMaxDevices) == cudaSuccess && call(duo::kMaxDevices) == cudaSuccess && sets == 6);
  return 0;
}
"""


def test_limit_is_set_on_each_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(BUILD._nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-I" + BUILD.CSRC, "-I" + cuda, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_every_launch_goes_through_it():
    for path in glob.glob(os.path.join(BUILD.CSRC, "*")):
        text = open(path).read()
        assert len(re.findall("cudaFuncSetAttribute", text)) == (os.path.basename(path) == "kernels.h"), path
