"""The limit of a kernel's dynamic shared memory under calls from several threads, against a stand-in for the CUDA runtime."""
import os
import shutil
import subprocess

import pytest

from gated_delta_rule_27_gb300 import build

# The runtime keeps the size that was set last.  A thread that sets the small size is held up until another has asked
# for the large one, or for a fifth of a second.
PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "kda_smem.cuh"

static void kernel() {}
static std::atomic<int> limit{0}, asked{0};
static std::atomic<bool> small_is_in{false}, large_is_set{false};

extern "C" cudaError_t cudaGetDevice(int *device) { *device = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int bytes) {
    asked++;
    if (bytes == 50000) {
        small_is_in = true;
        for (int i = 0; i < 200 && !large_is_set; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
    }
    limit = bytes;
    if (bytes == 150000) large_is_set = true;
    return cudaSuccess;
}

int main() {
    std::thread small([] { kda::allow_smem<kernel>(50000); });
    while (!small_is_in) std::this_thread::yield();
    std::thread large([] { kda::allow_smem<kernel>(150000); });
    small.join();
    large.join();
    const int before = asked;
    const cudaError_t e = kda::allow_smem<kernel>(100000);  // fits the larger: nothing is asked, and nothing may be lower
    std::printf("%d %d %d\n", (int)e, (int)limit, asked - before);
}
"""


def test_a_smaller_size_never_replaces_a_larger_one(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    source, program = tmp_path / "smem.cpp", tmp_path / "smem"
    source.write_text(PROGRAM)
    include = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", include, "-I", build.CSRC, str(source), "-o", str(program)], check=True)
    out = subprocess.run([str(program)], capture_output=True, text=True, timeout=60, check=True).stdout.split()
    assert out == ["0", "150000", "0"]
