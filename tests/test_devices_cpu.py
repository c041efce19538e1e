"""Kernel attributes belong to a device: a process that uses a second GPU sets
them there too.  Checked without one, against a fake of the runtime's current
device."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_tensor_core_persistent_gb300", "csrc")

PROGRAM = r"""
#include "host.h"
#include <cstdio>

static int current = 0;
static cudaError_t current_error = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = current; return current_error; }

#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
    static tcg::host::OncePerDevice once;
    int calls[3] = {0, 0, 0};
    cudaError_t outcome[3] = {cudaSuccess, cudaErrorInvalidValue, cudaSuccess};
    auto set_up = [&] { ++calls[current]; return outcome[current]; };
    for (int round = 0; round < 3; ++round)
        for (current = 0; current < 3; ++current) CHECK(once(set_up) == outcome[current]);
    for (int d = 0; d < 3; ++d) CHECK(calls[d] == 1);    // once on each, one device's error kept from the others
    static tcg::host::OncePerDevice other;
    current = 2;
    CHECK(other(set_up) == cudaSuccess && calls[2] == 2);
    current = -1;
    CHECK(other(set_up) == cudaErrorInvalidDevice);
    current = tcg::host::kMaxDevices;
    CHECK(other(set_up) == cudaErrorInvalidDevice);
    current = 0;
    current_error = cudaErrorNoDevice;
    CHECK(other(set_up) == cudaErrorNoDevice && calls[0] == 1);
    printf("ok\n");
    return 0;
}
"""


def cuda_include():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    return path if os.path.exists(os.path.join(path, "cuda_runtime.h")) else "/usr/local/cuda/include"


def test_set_up_runs_once_on_each_device(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-w", "-pthread", "-I", CSRC, "-I", cuda_include(), "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout


def test_every_kernel_attribute_is_set_per_device():
    found = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"cudaFuncSetAttribute", text):
            found += 1
            before = text[:m.start()]
            assert before.rfind("OncePerDevice once") > before.rfind("once_flag"), f"{name}: an attribute set once per process"
    assert found >= 2
