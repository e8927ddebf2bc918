"""CPU checks that the per-kernel records of the host side (the shared-memory
limit, the resident CTAs) hold when two host threads plan launches at once.  A small
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
static cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, void (*)(int), int, size_t smem);

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

static cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, void (*)(int), int, size_t smem) {
    *n = smem == 1000 ? 3 : 1;
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

    // what an int does not hold is refused, not cut to what it holds
    printf("huge %d\n", (int)(pa::ensure_smem_limit(kern, ((size_t)1 << 32) + 8, configured) == cudaErrorInvalidValue));

    // two sizes asked for in turn, by two threads: each gets the answer to its own
    static std::atomic<int64_t> cache[64];
    std::atomic<int> wrong{0}, ready{0};
    auto ask = [&](size_t smem, int want) {
        ++ready;
        for (int i = 0; i < 1000000 && ready.load() < 2; ++i) {}
        for (int i = 0; i < 300000; ++i) {
            int n = 0;
            if (pa::resident_ctas(kern, 32, smem, cache, &n) != cudaSuccess || n != want) ++wrong;
        }
    };
    std::thread c([&] { ask(1000, 3); }), d([&] { ask(2000, 1); });
    c.join();
    d.join();
    printf("wrong %d\n", wrong.load());
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


def test_resident_ctas_are_those_of_the_size_asked_for(said):
    assert "wrong 0" in said, said


def test_sizes_past_an_int_are_refused(said):
    assert "huge 1" in said, said
