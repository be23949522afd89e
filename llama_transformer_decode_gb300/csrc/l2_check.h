// Host side of the entry points that need no handle: argument checks, the device a call runs on.
#pragma once
#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cuda_runtime.h>

#include "../../include/l2.h"
#include "l2_kernels.h"

namespace l2 {

inline int refuse(int code, const char *fmt, ...) {
    char buf[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return set_call_error(code, buf);
}

inline int elt_size(int dtype) { return dtype == L2_F32 ? 4 : 2; }

// Makes the pool's device current for the call and puts the caller's back.
struct DeviceGuard {
    int before = -1;
    ~DeviceGuard() {
        if (before >= 0) cudaSetDevice(before);
    }
    bool enter(int device) {
        int cur = 0;
        if (cudaGetDevice(&cur) != cudaSuccess) return false;
        if (cur == device) return true;
        if (cudaSetDevice(device) != cudaSuccess) return false;
        before = cur;
        return true;
    }
};

// Device memory of one device (*device -1: any, and it is set), aligned to `align` bytes.
inline int check_ptr(const char *who, const char *name, const void *p, unsigned align, int *device) {
    if (!p) return refuse(L2_EINVAL, "%s: %s is NULL", who, name);
    if (reinterpret_cast<uintptr_t>(p) & (align - 1)) return refuse(L2_EINVAL, "%s: %s must be %u-byte aligned", who, name, align);
    cudaPointerAttributes a{};
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess || (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)) {
        cudaGetLastError();
        return refuse(L2_EINVAL, "%s: %s must be device memory", who, name);
    }
    if (*device < 0) *device = a.device;
    if (a.device != *device) return refuse(L2_EINVAL, "%s: %s is on device %d, the call's other memory on %d", who, name, a.device, *device);
    return L2_OK;
}

// Whether rows of `width` elements at every combination of the strides have memory of their own: each stride, in ascending
// order, is at least what the smaller ones span.
inline bool rows_apart(const long long *strides, const int *counts, int dims, long long width) {
    constexpr long long kFar = 1ll << 62;
    long long span = width;
    unsigned done = 0;
    for (int k = 0; k < dims; ++k) {
        int at = -1;  // the next stride; dimensions of one index are never stepped
        for (int i = 0; i < dims; ++i)
            if (counts[i] > 1 && !(done >> i & 1) && (at < 0 || strides[i] < strides[at])) at = i;
        if (at < 0) return true;
        done |= 1u << at;
        if (strides[at] < span) return false;
        span = strides[at] > kFar / counts[at] ? kFar : span + strides[at] * (counts[at] - 1);
    }
    return true;
}

inline int finish(const char *who, cudaError_t e) {
    if (e == cudaSuccess) return L2_OK;
    cudaGetLastError();
    return refuse(L2_ECUDA, "%s: %s (%s)", who, cudaGetErrorString(e), cudaGetErrorName(e));
}

// A row stride of the caller's tensors, in elements: whole 16-byte words.
inline int check_stride(const char *who, const char *name, long long stride, int steps, int es) {
    if (steps > 1 && (stride * es % 16 || stride < 0 || stride > (1ll << 40)))
        return refuse(L2_EINVAL, "%s: %s %lld must not be negative and a multiple of 16 bytes", who, name, stride);
    return L2_OK;
}

inline int sm_count(int device) {
    static std::atomic<int> counts[64];
    if (device < 0 || device >= 64) return 0;
    int n = counts[device].load(std::memory_order_relaxed);
    if (!n && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) == cudaSuccess)
        counts[device].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace l2
