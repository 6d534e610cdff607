// Host-side helpers shared by the library's translation units.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "mamba_ssm.h"
#include "ssm_device.cuh"

namespace mamba {

// Read and clear the device status word of block_ops.cu (device synchronised).
bool block_ops_take_status(int* code);

namespace {

constexpr int kMaxDevices = 64;

inline int dtype_bytes(int32_t dt) { return dt == MAMBA_BF16 ? 2 : 4; }
inline bool dtype_ok(int32_t dt) { return dt == MAMBA_F32 || dt == MAMBA_BF16; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Do two buffers of `bytes` overlap without being the same?
inline bool partly_overlap(const void* a, const void* b, size_t bytes) {
    if (a == nullptr || b == nullptr || a == b) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bytes && y < x + bytes;
}

// SM count of the current device, cached per device.
inline int current_sm_count(int* device_out) {
    static int cached[kMaxDevices] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (device_out) *device_out = dev;
    if (dev >= 0 && dev < kMaxDevices && cached[dev] > 0) return cached[dev];
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    if (dev >= 0 && dev < kMaxDevices) cached[dev] = sms;
    return sms;
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

template <typename Kernel>
cudaError_t ensure_smem_attr(Kernel kernel, int bytes, bool* done_per_device, int dev) {
    if (dev >= 0 && dev < kMaxDevices && done_per_device[dev]) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done_per_device[dev] = true;
    return e;
}

// Read and clear this translation unit's device status word.
inline bool take_device_status(int* code) {
    const int zero = 0;
    return cudaMemcpyFromSymbol(code, g_device_status, sizeof(int)) == cudaSuccess &&
           cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) == cudaSuccess;
}

}  // namespace
}  // namespace mamba
