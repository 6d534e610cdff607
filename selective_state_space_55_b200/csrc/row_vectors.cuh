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

// Steps of a row count in 32 bits, tile borders a little beyond its end included.
constexpr int64_t kMaxRowSteps = ((int64_t)1 << 31) - (1 << 16);
constexpr int kLaneSteps = 8;
constexpr int kWarpSteps = 32 * kLaneSteps;

// Elements between p and the 16-byte boundary at or below it.
template <typename T>
__device__ __forceinline__ int row_phase(const T* p) {
    return (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
}

// The bytes of a tensor: from its first element to behind its last.  A vector
// at the end of a row may reach into the next row or a gap; inside these bounds
// that is memory of the same tensor, and what it holds is thrown away.
struct Span {
    const unsigned char *begin, *end;
    __device__ __forceinline__ bool holds(const void* p, int bytes) const {
        const unsigned char* q = static_cast<const unsigned char*>(p);
        return q >= begin && q + bytes <= end;
    }
};

template <typename T>
__device__ __forceinline__ void unpack_steps(const uint4 (&raw)[sizeof(T) / 2], float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        unpack16(raw[0], v);
    } else {
        float a[4], b[4];
        unpack16(raw[0], a);
        unpack16(raw[1], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
}

// Eight aligned elements.
template <typename T>
__device__ __forceinline__ void load_eight(const T* p, float (&v)[8]) {
    uint4 raw[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
    unpack_steps<T>(raw, v);
}

// Steps t0 .. t0+7 of `row`; steps outside [lo, hi) give 0.  Vector loads when
// row + t0 is aligned and the tensor holds all eight.
template <typename T>
__device__ __forceinline__ void load_steps(const T* row, int t0, int lo, int hi, const Span& span,
                                           float (&v)[8]) {
    const T* p = row + t0;
    const bool some = t0 + 8 > lo && t0 < hi;
    if (some && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && span.holds(p, 8 * (int)sizeof(T))) {
        load_eight(p, v);
        if (t0 < lo || t0 + 8 > hi)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t0 + i < lo || t0 + i >= hi) v[i] = 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = (t0 + i >= lo && t0 + i < hi) ? DType<T>::load(p + i) : 0.0f;
    }
}

// Pairs of values, one per row of two that a warp works on side by side.
__device__ __forceinline__ float2 shfl_up2(float2 v, int o, int width = 32) {
    return make_float2(__shfl_up_sync(0xffffffffu, v.x, o, width), __shfl_up_sync(0xffffffffu, v.y, o, width));
}

__device__ __forceinline__ float2 shfl_down2(float2 v, int o, int width = 32) {
    return make_float2(__shfl_down_sync(0xffffffffu, v.x, o, width), __shfl_down_sync(0xffffffffu, v.y, o, width));
}

__device__ __forceinline__ float2 shfl2(float2 v, int lane, int width = 32) {
    return make_float2(__shfl_sync(0xffffffffu, v.x, lane, width), __shfl_sync(0xffffffffu, v.y, lane, width));
}

template <typename T>
__device__ __forceinline__ void store_eight(T* p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = pack16(v);
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

template <typename T>
__device__ __forceinline__ void store_steps(T* row, int t0, int lo, int hi,
                                            const float (&v)[8]) {
    T* p = row + t0;
    if (t0 >= lo && t0 + 8 <= hi && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        store_eight(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t0 + i >= lo && t0 + i < hi) DType<T>::store(p + i, v[i]);
    }
}

// 16 bytes global -> shared, asynchronous, part of the thread's open group.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}

__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Wait until at most kN of this thread's committed groups are under way.
template <int kN>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

template <typename T>
__device__ __forceinline__ void store_steps2(T* row0, int t0, int lo0, int hi0, T* row1, int64_t t1,
                                             int64_t lo1, int64_t hi1, const float2 (&v)[8]) {
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = v[i].x;
        b[i] = v[i].y;
    }
    store_steps(row0, t0, lo0, hi0, a);
    store_steps(row1, t1, lo1, hi1, b);
}

}  // namespace mamba
