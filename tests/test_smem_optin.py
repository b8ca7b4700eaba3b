"""The kernels' shared-memory opt-in, kept for each device and set by any host thread: the
header's class against a runtime that records the calls (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SRC = r"""
#include "hsa_internal.h"
#include <cstdio>
#include <thread>
#include <vector>
static thread_local int g_dev = 0;
static std::atomic<int> g_sets[80];
static std::atomic<int> g_fail{0};
extern "C" cudaError_t cudaGetDevice(int *d) { *d = g_dev; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute a, int v)
{
    if (!f || a != cudaFuncAttributeMaxDynamicSharedMemorySize || v != 1234)
        return cudaErrorInvalidValue;
    ++g_sets[g_dev];
    return g_fail ? cudaErrorInvalidDevice : cudaSuccess;
}
static void kern(int) {}
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main()
{
    hsa::SmemOptIn a, b;
    for (int dev : {0, 3, 0, 63, 3, 0}) {
        g_dev = dev;
        CHECK(a.set(kern, 1234) == cudaSuccess);
    }
    CHECK(g_sets[0] == 1 && g_sets[3] == 1 && g_sets[63] == 1);  // once a device
    g_dev = 3;
    CHECK(b.set(kern, 1234) == cudaSuccess && g_sets[3] == 2);   // and a kernel
    g_dev = 70;                                                  // past the bits: every call
    CHECK(a.set(kern, 1234) == cudaSuccess && a.set(kern, 1234) == cudaSuccess && g_sets[70] == 2);
    g_dev = 5;                                                   // a failure is not kept
    g_fail = 1;
    CHECK(a.set(kern, 1234) == cudaErrorInvalidDevice);
    g_fail = 0;
    CHECK(a.set(kern, 1234) == cudaSuccess && a.set(kern, 1234) == cudaSuccess && g_sets[5] == 2);
    std::vector<std::thread> th;
    std::atomic<int> bad{0};
    for (int i = 0; i < 16; ++i)
        th.emplace_back([&, i] {
            g_dev = 8 + i % 4;
            for (int k = 0; k < 1000; ++k)
                bad += a.set(kern, 1234) != cudaSuccess;
        });
    for (auto &t : th)
        t.join();
    CHECK(bad == 0);
    for (int d = 8; d < 12; ++d)
        CHECK(g_sets[d] >= 1 && g_sets[d] <= 4);
    return 0;
}
"""


def test_opt_in_is_kept_for_each_device(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    gxx = shutil.which("g++")
    if not os.path.exists(nvcc) or not gxx:
        pytest.skip("no toolkit")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(SRC)
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", inc, "-I",
                    os.path.join(ROOT, "full_attention_kv_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
