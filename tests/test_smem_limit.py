"""The shared-memory limit of a kernel is raised on every device it is launched on.

The helper is compiled with a fake of the two runtime calls that it makes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a16_int4_quantized_gb300", "csrc")

PROGRAM = r"""
#include "smem_limit.h"
#include <cassert>
#include <cstdio>

static int device = 0, calls = 0, last_device = -1, last_bytes = 0;
static cudaError_t get_error = cudaSuccess, set_error = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return get_error; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute a, int bytes) {
    assert(a == cudaFuncAttributeMaxDynamicSharedMemorySize);
    ++calls;
    last_device = device;
    last_bytes = bytes;
    return set_error;
}

int main() {
    w4::SmemLimit one, two;
    int k = 0;
    for (int round = 0; round < 3; ++round)
        for (device = 0; device < 64; device += 7) assert(one.raise(&k, 100000) == cudaSuccess);
    assert(calls == 10 && last_device == 63 && last_bytes == 100000);  // once for each of ten devices
    device = 0;
    assert(two.raise(&k, 5) == cudaSuccess && calls == 11 && last_bytes == 5);  // another kernel
    device = 1;
    set_error = cudaErrorInvalidValue;  // a failure is not remembered as done, nor for good
    assert(two.raise(&k, 5) == cudaErrorInvalidValue && two.raise(&k, 5) == cudaErrorInvalidValue && calls == 13);
    set_error = cudaSuccess;
    assert(two.raise(&k, 5) == cudaSuccess && two.raise(&k, 5) == cudaSuccess && calls == 14);
    get_error = cudaErrorNoDevice;
    assert(two.raise(&k, 5) == cudaErrorNoDevice && calls == 14);
    get_error = cudaSuccess;
    device = 64;  // beyond what is kept
    assert(two.raise(&k, 5) == cudaSuccess && two.raise(&k, 5) == cudaSuccess && calls == 16);
    std::puts("ok");
}
"""


def test_once_for_each_device(tmp_path):
    cxx = shutil.which("g++") or pytest.skip("no C++ compiler")
    from w4a16_int4_quantized_gb300 import build
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    src = tmp_path / "t.cpp"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, "-I", cuda, str(src), "-o", str(tmp_path / "t")], check=True)
    assert subprocess.run([str(tmp_path / "t")], check=True, capture_output=True, text=True).stdout == "ok\n"


def test_every_launch_goes_through_it():
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f)) as h:
            n = h.read().count("cudaFuncSetAttribute(")
        assert n == (1 if f == "smem_limit.h" else 0), f
