"""Per-device host values (csrc/per_device.h), compiled for the host with a stand-in for cudaGetDevice and run by several
threads under the thread sanitizer: each device has its own value, and first callers that meet do not race."""
import os
import subprocess

import pytest

from expert_offload_serving_router_b200 import build as ftbuild

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
thread_local int dev = 0;
extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* d) { if (dev == 99) return cudaErrorNoDevice; *d = dev; return cudaSuccess; }
using namespace ftmoe;
int main() {
    static PerDeviceCount count;
    static PerDeviceOnce once;
    std::atomic<int> bad{0}, asked{0}, ran{0}, refused{0};
    std::vector<std::thread> ts;
    for (int i = 0; i < 8; ++i)
        ts.emplace_back([&, i] {
            for (int r = 0; r < 2000; ++r) {
                dev = (i + r) % 3;
                if (count([&] { ++asked; return 100 + dev; }) != 100 + dev) ++bad;
                if (once([&] { ++ran; return dev == 2 ? cudaErrorInvalidValue : cudaSuccess; }) !=
                    (dev == 2 ? cudaErrorInvalidValue : cudaSuccess)) ++bad;
            }
        });
    for (auto& t : ts) t.join();
    // devices that have no slot: asked each time
    for (int d : {99, kDeviceTable + 5}) { dev = d; for (int r = 0; r < 2; ++r) if (count([&] { ++refused; return 7; }) != 7) ++bad; }
    std::printf("%d %d %d %d\n", bad.load(), asked.load(), ran.load(), refused.load());
}
"""


@pytest.mark.parametrize("flags", [[], ["-fsanitize=thread"]])
def test_per_device_values_by_many_threads(tmp_path, flags):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(ftbuild.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-pthread", *flags, "-I", ftbuild.CSRC, "-I", cuda, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "data race" not in r.stderr, r.stderr[-2000:]
    bad, asked, ran, refused = map(int, r.stdout.split())
    assert bad == 0
    assert 3 <= asked <= 24                  # once a device, or once for each thread that met the others there
    assert ran > 2 * 2000                    # a setup that failed is tried again by every call
    assert refused == 4
