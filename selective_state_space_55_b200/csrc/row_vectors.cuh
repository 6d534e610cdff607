// Eight consecutive time steps per lane of a row whose start need not be aligned.
//
// Rows are (batch, dim, seqlen) chains.  With an odd length only some rows
// start on a 16-byte boundary, so the warp's 256-step tiles are laid over
// addresses instead of steps: a row that starts m elements past a boundary is
// cut at steps -m, 256 - m, ...  Every lane's eight steps then sit on aligned
// vectors; the lanes at the row's two ends, and tensors whose own start lies
// elsewhere, move element by element.
#pragma once

#include "ssm_device.cuh"

namespace mamba {

constexpr int kLaneSteps = 8;
constexpr int kWarpSteps = 32 * kLaneSteps;

// Elements between p and the 16-byte boundary at or below it.
template <typename T>
__device__ __forceinline__ int row_phase(const T* p) {
    return (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
}

// Steps t0 .. t0+7 of `row`; steps outside [lo, hi) give `fill` and are not
// read.  Vector loads when the eight are inside and row + t0 is aligned.
template <typename T>
__device__ __forceinline__ void load_steps(const T* row, int64_t t0, int64_t lo, int64_t hi,
                                           float fill, float (&v)[8]) {
    const T* p = row + t0;
    if (t0 >= lo && t0 + 8 <= hi && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        if constexpr (sizeof(T) == 2) {
            unpack16(*reinterpret_cast<const uint4*>(p), v);
        } else {
            const float4 a = reinterpret_cast<const float4*>(p)[0];
            const float4 b = reinterpret_cast<const float4*>(p)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = (t0 + i >= lo && t0 + i < hi) ? DType<T>::load(p + i) : fill;
    }
}

template <typename T>
__device__ __forceinline__ void store_steps(T* row, int64_t t0, int64_t lo, int64_t hi,
                                            const float (&v)[8]) {
    T* p = row + t0;
    if (t0 >= lo && t0 + 8 <= hi && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(p) = pack16(v);
        } else {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t0 + i >= lo && t0 + i < hi) DType<T>::store(p + i, v[i]);
    }
}

}  // namespace mamba
