// Host-side values that belong to a device: set up or queried once for each, by any host thread.
#pragma once
#include <cuda_runtime_api.h>

#include <atomic>

namespace ftmoe {

constexpr int kDeviceTable = 64;      // devices past it repeat the work on every call, which is correct, only slower

inline int device_slot() {
    int d = -1;
    return cudaGetDevice(&d) == cudaSuccess && d >= 0 && d < kDeviceTable ? d : -1;
}

// One-time setup per device: a kernel's cudaFuncSetAttribute values belong to the current device's copy of it.
// Threads that meet before the first is done each run it.
struct PerDeviceOnce {
    std::atomic<bool> done[kDeviceTable] = {};
    template <typename Fn>
    cudaError_t operator()(Fn&& fn) {
        const int d = device_slot();
        if (d >= 0 && done[d].load(std::memory_order_acquire)) return cudaSuccess;
        const cudaError_t e = fn();
        if (e == cudaSuccess && d >= 0) done[d].store(true, std::memory_order_release);
        return e;
    }
};

// A positive number asked of the current device.
struct PerDeviceCount {
    std::atomic<int> n[kDeviceTable] = {};
    template <typename Fn>
    int operator()(Fn&& fn) {
        const int d = device_slot();
        int v = d >= 0 ? n[d].load(std::memory_order_relaxed) : 0;
        if (v) return v;
        v = fn();
        if (d >= 0) n[d].store(v, std::memory_order_relaxed);
        return v;
    }
};

}  // namespace ftmoe
