// device_guard.h -- the entry points' way onto their own device.
#pragma once
#include <cuda_runtime.h>

namespace dsq {

// Makes `device` current for the scope and restores the caller's device.  A
// failure is the entry point's to return: the runtime's last error is cleared,
// or the caller's next launch check would report it.
struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int device) {
        ok = cudaGetDevice(&prev) == cudaSuccess && (prev == device || cudaSetDevice(device) == cudaSuccess);
        if (!ok) cudaGetLastError();
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

}  // namespace dsq
