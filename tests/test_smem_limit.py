"""A kernel's shared memory limit belongs to a device: a process that launches
on several raises it on each of them.  The header is compiled against fakes of
the two runtime calls, so no GPU is needed."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from collective_all_reduce_rank_gb300 import build

MAIN = r"""
#include <cstdio>
#include <map>
#include <utility>
#include "smem_limit.h"

static int current = 0, calls = 0;
static bool refuse = false;
static std::map<std::pair<int, const void*>, int> limits;

cudaError_t cudaGetDevice(int* d) { *d = current; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  ++calls;
  if (refuse || a != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaErrorInvalidValue;
  limits[{current, f}] = v;
  return cudaSuccess;
}

template <int N> void kernel(int*) {}

#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }

int main() {
  using rra::raise_smem;
  for (int device : {0, 1, 63, 64, 200}) {
    current = device;
    for (int again = 0; again < 3; ++again) CHECK(raise_smem<kernel<1>>(1000 + device) == cudaSuccess);
    CHECK((limits[{device, (const void*)kernel<1>}] == 1000 + device));
  }
  CHECK(calls == 3 + 2 * 3);  // once on each device that is kept, every time past them
  current = 1;
  CHECK((limits.count({1, (const void*)kernel<2>}) == 0));  // of another kernel
  refuse = true;
  CHECK(raise_smem<kernel<2>>(7) == cudaErrorInvalidValue);  // a refusal is no success the next time
  refuse = false;
  CHECK(raise_smem<kernel<2>>(7) == cudaSuccess && (limits[{1, (const void*)kernel<2>}] == 7));
  return 0;
}
"""


def test_the_limit_is_raised_on_every_device(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(MAIN)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    cmd = [cxx, "-std=c++17", "-I", build.CSRC, "-I", cuda, "-I", "/usr/local/cuda/include", str(src), "-o", str(exe)]
    p = subprocess.run(cmd, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    p = subprocess.run([str(exe)], capture_output=True, text=True)
    assert p.returncode == 0, p.stdout


def test_no_launcher_keeps_it_for_the_process():
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        text = open(path).read()
        assert not re.search(r"static const cudaError_t \w+\s*=\s*cudaFuncSetAttribute", text), path
