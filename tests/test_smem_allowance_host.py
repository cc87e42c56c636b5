"""The shared-memory allowance of a kernel (csrc/hostops.h) with two host
threads asking for different sizes at once: the attribute that is set last
has to be the largest, since the record says that no call needs to set it
again.  Compiled with a fake of the two CUDA calls, which lets the larger
request wait inside its call until the smaller one has had its chance."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "scaled_fp8_linear_gb300", "csrc")

SOURCE = r"""
#include <atomic>
#include <chrono>
#include <cstdarg>
#include <cstdio>
#include <thread>
#include "hostops.h"

static std::atomic<int> attribute{0}, calls{0};
static std::atomic<bool> large_is_in{false};
static int device = 0;

namespace fp8 { int set_error(int status, const char*, ...) { return status; } }
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return ""; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes) {
    ++calls;
    attribute = bytes;   // sets the limit, lower or higher
    if (bytes > 100000) {
        large_is_in = true;
        std::this_thread::sleep_for(std::chrono::milliseconds(300));
    }
    return cudaSuccess;
}
}

static void kernel() {}

static int ask(fp8::host::SmemAllowance& a, int bytes) {
    return fp8::host::allow_smem(reinterpret_cast<const void*>(&kernel), bytes, a);
}

int main() {
    static fp8::host::SmemAllowance a;
    std::thread large([&] { ask(a, 196608); });
    while (!large_is_in) std::this_thread::yield();
    std::thread small([&] { ask(a, 24576); });   // while the other is in its call
    large.join();
    small.join();
    if (attribute != 196608) { std::printf("attribute %d\n", attribute.load()); return 1; }
    const int before = calls;
    if (ask(a, 65536) || ask(a, 196608) || calls != before) return 2;   // known: no call
    if (ask(a, 200000) || attribute != 200000) return 3;                // larger: raised
    if (ask(a, 24576) || attribute != 200000) return 4;                 // smaller: stays
    device = 3;
    if (ask(a, 50000) || attribute != 50000) return 5;                  // each device its own
    return 0;
}
"""


def test_two_threads(tmp_path):
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cxx = shutil.which("g++")
    if not cxx or not os.path.exists(os.path.join(cuda, "include", "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "allow.cpp", tmp_path / "allow"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-I", os.path.join(cuda, "include"),
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout)
