"""CPU checks that the per-kernel records of the host side (the shared-memory
limit) hold when two host threads plan their first launches at once.  A small
program compiled against csrc/pa_internal.h stands in for the CUDA runtime with
fakes that bring the threads into the order that hurts; its waits are bounded."""
import subprocess
from pathlib import Path

import pytest

from pagedattention_decode_paged_gb300 import _build

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

#include <cuda_runtime.h>

static cudaError_t cudaFuncSetAttribute(void (*)(int), cudaFuncAttribute, int bytes);

#include "pa_internal.h"

static std::atomic<int> limit{0}, step{0};

// up to a quarter of a second for `want`
static void wait_for(int want) {
    for (int i = 0; i < 250 && step.load() < want; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
}

extern "C" cudaError_t CUDARTAPI cudaGetDevice(int *dev) { *dev = 0; return cudaSuccess; }
// The larger size is set first; its caller goes on once the smaller one is set too.
static cudaError_t cudaFuncSetAttribute(void (*)(int), cudaFuncAttribute, int bytes) {
    if (bytes == 2000) {
        limit = bytes;
        step = 1;
        wait_for(2);
    } else {
        limit = bytes;
        step = 2;
    }
    return cudaSuccess;
}

static void kern(int) {}

int main() {
    std::atomic<int> configured[64] = {};
    cudaError_t small = cudaErrorUnknown, large = cudaErrorUnknown;
    std::thread a([&] { large = pa::ensure_smem_limit(kern, 2000, configured); });
    std::thread b([&] { wait_for(1); small = pa::ensure_smem_limit(kern, 1000, configured); });
    a.join();
    b.join();
    printf("limit %d recorded %d status %d %d\n", limit.load(), configured[0].load(), (int)small, (int)large);
    return 0;
}
"""


@pytest.fixture(scope="module")
def said(tmp_path_factory):
    d = tmp_path_factory.mktemp("threads")
    src = d / "t.cpp"
    src.write_text(PROGRAM)
    exe = d / "t"
    cuda = Path(_build._nvcc()).resolve().parent.parent / "include"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{cuda}", f"-I{_build.INCLUDE}", f"-I{_build.CSRC}", str(src),
                    "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=120).stdout


def test_a_recorded_limit_is_the_kernels_limit(said):
    assert "limit 2000 recorded 2000 status 0 0" in said, said
