"""Kernels' shared-memory limits are raised on every device that runs them
(csrc/smem_limit.h), checked against a runtime that the test fakes.  No GPU."""

import glob
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_nf4_quantized_26_b200", "csrc")

PROGRAM = r"""
#include "smem_limit.h"
#include <cstdio>
static int device, calls;
static cudaError_t answer;
static const void* kernel;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void* k, cudaFuncAttribute a, int v) {
  ++calls;
  kernel = k;
  return a == cudaFuncAttributeMaxDynamicSharedMemorySize && v == 99000 ? answer : cudaErrorInvalidValue;
}
static void one(int) {}
static int go(int dev, uint64_t& done) {
  device = dev;
  return static_cast<int>(qnf4::allow_smem(one, 99000, done));
}
int main() {
  uint64_t a = 0, b = 0;
  int bad = 0;
  bad += go(0, a) != 0 || calls != 1 || kernel != reinterpret_cast<const void*>(one);
  bad += go(0, a) != 0 || calls != 1;   // once is enough
  bad += go(1, a) != 0 || calls != 2;   // another device has its own limit
  bad += go(0, a) != 0 || calls != 2;
  bad += go(0, b) != 0 || calls != 3;   // and so has another kernel
  answer = cudaErrorInvalidValue;
  bad += go(2, a) == 0 || calls != 4;   // a refusal is reported and not remembered
  answer = cudaSuccess;
  bad += go(2, a) != 0 || calls != 5;
  std::printf("%d\n", bad);
  return bad;
}
"""


def test_limit_is_raised_once_per_kernel_and_device(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, "-I", inc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_every_limit_is_raised_there():
    """No launcher keeps a flag of its own, which would hold for one device only."""
    users = 0
    for f in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(f).read()
        if os.path.basename(f) != "smem_limit.h":
            assert "cudaFuncSetAttribute" not in text, f
            users += text.count("allow_smem(")
    assert users > 0
