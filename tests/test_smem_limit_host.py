"""Two host threads raise one kernel's shared-memory limit at once, the CUDA
calls replaced by stand-ins on the host (no GPU): whichever of them is slow,
the limit that stays is the larger one."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_pq2_ternary_gb300", "csrc")

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <cuda_runtime.h>

static std::atomic<int> g_limit{0}, g_entered{0};
static cudaError_t fake_device(int* dev) { *dev = 0; return cudaSuccess; }
// the smaller size's call takes effect late
template <typename Kern>
static cudaError_t fake_set(Kern, cudaFuncAttribute, int bytes) {
    g_entered.fetch_add(1);
    if (bytes < 200) std::this_thread::sleep_for(std::chrono::milliseconds(300));
    g_limit.store(bytes);
    return cudaSuccess;
}
#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_set
#include "pq2_step.cuh"

int main() {
    static pq2h::SmemLimit lim;
    std::thread small([] { pq2h::raise_smem(lim, 0, 100); });
    while (g_entered.load() == 0) std::this_thread::yield();   // it is in its call
    std::thread large([] { pq2h::raise_smem(lim, 0, 1000); });
    small.join();
    large.join();
    pq2h::raise_smem(lim, 0, 1000);
    pq2h::raise_smem(lim, 0, 500);                             // never down
    std::printf("%d %d\n", g_limit.load(), lim.bytes[0].load());
    return 0;
}
"""


def test_the_larger_limit_stays(tmp_path):
    from gemm_pq2_ternary_gb300 import _build
    try:
        nvcc = _build._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    src, exe = tmp_path / "limit.cu", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, *_build.ARCH, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60, check=True).stdout
    assert out.split() == ["1000", "1000"]
