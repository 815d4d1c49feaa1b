// s6_host.cuh -- host-side helpers of the library's entry points (argument
// checks, device selection), shared by its translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "s6.h"

namespace s6 {
namespace host {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

inline size_t io_size(int io) { return io == S6_BF16 ? 2 : 4; }

inline int launch_status(cudaError_t e) { return e == cudaSuccess ? S6_OK : S6_ERR_CUDA; }

// Every entry point restores the calling thread's current device before it
// returns: use_stream_device below may switch it to the stream's device.
struct DeviceRestore {
    int prev = -1;
    DeviceRestore() {
        if (cudaGetDevice(&prev) != cudaSuccess)
            prev = -1;
    }
    ~DeviceRestore() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev)
            cudaSetDevice(prev);
    }
    DeviceRestore(const DeviceRestore &) = delete;
    DeviceRestore &operator=(const DeviceRestore &) = delete;
};

// Make the device that owns `stream` current for this library's runtime before
// any launch (the caller's framework may have selected it through another
// runtime instance in the same process).  The legacy and per-thread default
// streams keep the current device.
inline int use_stream_device(cudaStream_t stream) {
    if (stream == nullptr || stream == cudaStreamLegacy || stream == cudaStreamPerThread)
        return S6_OK;
    // a stream being captured into a graph: the capture already runs on the
    // current device, and device queries on it would invalidate the capture
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess)
        return S6_ERR_CUDA;
    if (cap != cudaStreamCaptureStatusNone)
        return S6_OK;
    int dev = -1, cur = -1;
    if (cudaStreamGetDevice(stream, &dev) != cudaSuccess || cudaGetDevice(&cur) != cudaSuccess)
        return S6_ERR_CUDA;
    if (dev != cur && cudaSetDevice(dev) != cudaSuccess)
        return S6_ERR_CUDA;
    return S6_OK;
}

inline int device_sm_count() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 148;
    if (!cached[dev]) {
        int n = 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        cached[dev] = n > 0 ? n : 148;
    }
    return cached[dev];
}

}  // namespace host
}  // namespace s6
