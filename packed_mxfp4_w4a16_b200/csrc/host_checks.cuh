// host_checks.cuh — argument checks shared by the host side of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_mxfp4.h"

namespace moe {

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

constexpr int kAnyDevice = -2;

// p must be memory of GPU `device` (or kAnyDevice), `align`-byte aligned (a
// power of two).
inline int check_device_memory(int device, const void *p, size_t align) {
    if (!p) return MOE_ERR_ARG;
    if (((uintptr_t)p) & (align - 1)) return MOE_ERR_ALIGN;
    cudaPointerAttributes a;
    cudaError_t e = cudaPointerGetAttributes(&a, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_NOT_DEVICE;
    }
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) return MOE_ERR_NOT_DEVICE;
    if (device != kAnyDevice && a.device != device) return MOE_ERR_NOT_DEVICE;
    return MOE_OK;
}

// The current device and its SM count; UNSUPPORTED when it is not sm_100.
inline int current_device_ok(int *dev, int *sms) {
    int d = -1;
    if (cudaGetDevice(&d) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    int major = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    if (major != 10) return MOE_ERR_UNSUPPORTED;
    if (dev) *dev = d;
    if (sms) *sms = n;
    return MOE_OK;
}

inline int cuda_rc(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    cudaGetLastError();
    return MOE_ERR_CUDA;
}

}  // namespace moe
