// Layer norm with the residual add, forward and backward (sm_100a).
//
// Per row of dim elements (root-mean-square form: mean = 0):
//
//   s = x + residual;  mean, var = moments of s;  rstd = (var + eps)^-1/2
//   out = (s - mean) rstd w + b
//
// and, with xh = (s - mean) rstd, q = dout w, c1 = sum(q) / dim (0 in the
// root-mean-square form), c2 = sum(q xh) / dim,
//
//   ds = rstd (q - c1 - xh c2) + dresidual_out;  dw = sum_rows dout xh;  db = sum_rows dout.
//
// All of it is HBM-bound: a few operations per element against 4 to 16 bytes.
// A row stays in the registers of one team of threads (a warp, or a CTA of
// dim / 8 threads), so each tensor crosses HBM once; the variance is summed
// from (s - mean)^2 in a second reduction over the registers, so an offset far
// above the spread costs no digits.  The backward's column sums stay in the
// registers of the thread that owns the columns while the CTA walks its rows;
// each CTA leaves one partial row per sum, and a second launch adds the
// partial rows in a fixed order (no atomics: results repeat bit for bit).
#pragma once

#include "ssm_device.cuh"

namespace mamba {

constexpr int kNormElems = 8;            // consecutive elements per thread and chunk
constexpr int kNormWarpDim = 512;        // dims up to here: one warp per row
constexpr int kNormCtaDim = 8192;        // dims up to here: one CTA per row, in registers
constexpr int kNormRowsPerCta = 8;       // rows side by side in a CTA, one warp each
constexpr int kNormWideThreads = 1024;   // wider rows: threads of a CTA that re-reads the row

struct NormParams {
    const void* x;              // fwd: x; bwd: s
    const void* residual;       // fwd, or null
    const float* weight;        // or null (ones)
    const float* bias;          // or null
    void* out;                  // fwd
    void* residual_out;         // fwd, or null
    float* mean;                // fwd, or null
    float* rstd;
    const float* mean_in;       // bwd; null in the root-mean-square form
    const float* rstd_in;
    const void* dout;           // bwd
    const void* dresidual_out;  // bwd, or null
    void* dx;                   // bwd
    void* dresidual;            // bwd, or null
    float* partial;             // bwd: [ctas][sums][dim], or null
    int64_t rows;
    int64_t x_stride, residual_stride, out_stride, residual_out_stride;   // fwd
    int64_t dx_stride, dresidual_stride;                                  // bwd (s: x_stride,
                                                // dout: out_stride, dresidual_out: residual_out_stride)
    float eps;
    int dim;
    int rms;
    int res_f32;                // residual, residual_out, s, dresidual_out, dresidual are fp32
    int has_dw, has_db;
};

// Column of element i of chunk c for thread tid of a team of n: with vectors,
// 8 neighbours per thread; without, neighbouring threads take neighbouring
// columns so that 2- and 4-byte accesses still coalesce.
template <bool kVec>
__device__ __forceinline__ int norm_col(int c, int i, int tid, int n) {
    return kVec ? (c * n + tid) * kNormElems + i : (c * kNormElems + i) * n + tid;
}

template <typename T>
__device__ __forceinline__ void load8_vec(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        unpack16(*reinterpret_cast<const uint4*>(p), v);
    } else {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

template <typename T>
__device__ __forceinline__ void store8_vec(T* p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = pack16(v);
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// Chunk c of a row (columns beyond dim read as `fill`).
template <typename T, bool kVec>
__device__ __forceinline__ void norm_load(const T* row, int dim, int c, int tid, int n, float fill,
                                          float (&v)[8]) {
    if constexpr (kVec) {
        const int col = norm_col<true>(c, 0, tid, n);
        if (col < dim) load8_vec(row + col, v);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fill;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = norm_col<false>(c, i, tid, n);
            v[i] = col < dim ? DType<T>::load(row + col) : fill;
        }
    }
}

template <typename T, bool kVec>
__device__ __forceinline__ void norm_store(T* row, int dim, int c, int tid, int n,
                                           const float (&v)[8]) {
    if constexpr (kVec) {
        const int col = norm_col<true>(c, 0, tid, n);
        if (col < dim) store8_vec(row + col, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = norm_col<false>(c, i, tid, n);
            if (col < dim) DType<T>::store(row + col, v[i]);
        }
    }
}

// The residual stream's tensors: fp32, or the type of x.
template <typename IoT, bool kVec>
__device__ __forceinline__ void norm_load_res(const void* base, int64_t offset, int f32, int dim,
                                              int c, int tid, int n, float (&v)[8]) {
    if (f32) norm_load<float, kVec>(static_cast<const float*>(base) + offset, dim, c, tid, n, 0.0f, v);
    else norm_load<IoT, kVec>(static_cast<const IoT*>(base) + offset, dim, c, tid, n, 0.0f, v);
}

template <typename IoT, bool kVec>
__device__ __forceinline__ void norm_store_res(void* base, int64_t offset, int f32, int dim, int c,
                                               int tid, int n, const float (&v)[8]) {
    if (f32) norm_store<float, kVec>(static_cast<float*>(base) + offset, dim, c, tid, n, v);
    else norm_store<IoT, kVec>(static_cast<IoT*>(base) + offset, dim, c, tid, n, v);
}

// Sums of kN values over the team (the warp, or the CTA when blockDim.x > 32);
// every thread gets them.  `buf` is [2][32 kN] shared floats used in turn, so
// one barrier per call is enough.
template <int kN>
__device__ __forceinline__ void team_sum(float (&v)[kN], float* buf, int& turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (blockDim.x > 32) {
        float* b = buf + turn * 32 * kN;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < kN; ++k) b[warp * kN + k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kN; ++k) v[k] = lane < warps ? b[lane * kN + k] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        turn ^= 1;
    }
}

// Forward, the row in registers: blockDim.x threads per row, blockDim.y rows
// side by side (more than one only with warps), kV chunks of 8 per thread.
template <typename IoT, int kV, bool kVec>
__global__ void __launch_bounds__(kV == 1 ? 1024 : 32 * kNormRowsPerCta, 1)
    layer_norm_fwd_kernel(const __grid_constant__ NormParams p) {
    __shared__ float buf[2 * 32];
    const int tid = threadIdx.x, n = blockDim.x;
    int turn = 0;
    float w[kV][8], b[kV][8];
#pragma unroll
    for (int c = 0; c < kV; ++c) {
        if (p.weight != nullptr) norm_load<float, kVec>(p.weight, p.dim, c, tid, n, 0.0f, w[c]);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) w[c][i] = 1.0f;
        if (p.bias != nullptr) norm_load<float, kVec>(p.bias, p.dim, c, tid, n, 0.0f, b[c]);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) b[c][i] = 0.0f;
    }
    const float inv_dim = 1.0f / (float)p.dim;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < p.rows; row += step) {
        float s[kV][8];
        const IoT* x = static_cast<const IoT*>(p.x) + row * p.x_stride;
#pragma unroll
        for (int c = 0; c < kV; ++c) norm_load<IoT, kVec>(x, p.dim, c, tid, n, 0.0f, s[c]);
        if (p.residual != nullptr) {
#pragma unroll
            for (int c = 0; c < kV; ++c) {
                float r[8];
                norm_load_res<IoT, kVec>(p.residual, row * p.residual_stride, p.res_f32, p.dim, c,
                                         tid, n, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[c][i] += r[i];
            }
        }
        if (p.residual_out != nullptr)
#pragma unroll
            for (int c = 0; c < kV; ++c)
                norm_store_res<IoT, kVec>(p.residual_out, row * p.residual_out_stride, p.res_f32,
                                          p.dim, c, tid, n, s[c]);
        float mean = 0.0f;
        if (!p.rms) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < kV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[0] += s[c][i];
            team_sum(sum, buf, turn);
            mean = sum[0] * inv_dim;
        }
        float sq[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < kV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = s[c][i] - mean;
                s[c][i] = d;
                if (norm_col<kVec>(c, i, tid, n) < p.dim) sq[0] = fmaf(d, d, sq[0]);
            }
        team_sum(sq, buf, turn);
        const float rstd = 1.0f / sqrtf(fmaf(sq[0], inv_dim, p.eps));
        if (tid == 0) {
            if (p.mean != nullptr) p.mean[row] = mean;
            if (p.rstd != nullptr) p.rstd[row] = rstd;
        }
        IoT* out = static_cast<IoT*>(p.out) + row * p.out_stride;
#pragma unroll
        for (int c = 0; c < kV; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[c][i] = fmaf(s[c][i] * rstd, w[c][i], b[c][i]);
            norm_store<IoT, kVec>(out, p.dim, c, tid, n, s[c]);
        }
    }
}

// Forward for rows wider than a CTA's registers: the row is read three times,
// the second and third from L2.
template <typename IoT, bool kVec>
__global__ void __launch_bounds__(kNormWideThreads)
    layer_norm_fwd_wide_kernel(const __grid_constant__ NormParams p) {
    __shared__ float buf[2 * 32];
    const int tid = threadIdx.x, n = blockDim.x;
    const int chunks = (p.dim + n * kNormElems - 1) / (n * kNormElems);
    const float inv_dim = 1.0f / (float)p.dim;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const IoT* x = static_cast<const IoT*>(p.x) + row * p.x_stride;
        auto load = [&](int c, float (&s)[8]) {
            norm_load<IoT, kVec>(x, p.dim, c, tid, n, 0.0f, s);
            if (p.residual != nullptr) {
                float r[8];
                norm_load_res<IoT, kVec>(p.residual, row * p.residual_stride, p.res_f32, p.dim, c,
                                         tid, n, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] += r[i];
            }
        };
        float s[8];
        float mean = 0.0f;
        if (!p.rms) {
            float sum[1] = {0.0f};
            for (int c = 0; c < chunks; ++c) {
                load(c, s);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[0] += s[i];
            }
            team_sum(sum, buf, turn);
            mean = sum[0] * inv_dim;
        }
        float sq[1] = {0.0f};
        for (int c = 0; c < chunks; ++c) {
            load(c, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = s[i] - mean;
                if (norm_col<kVec>(c, i, tid, n) < p.dim) sq[0] = fmaf(d, d, sq[0]);
            }
        }
        team_sum(sq, buf, turn);
        const float rstd = 1.0f / sqrtf(fmaf(sq[0], inv_dim, p.eps));
        if (tid == 0) {
            if (p.mean != nullptr) p.mean[row] = mean;
            if (p.rstd != nullptr) p.rstd[row] = rstd;
        }
        IoT* out = static_cast<IoT*>(p.out) + row * p.out_stride;
        for (int c = 0; c < chunks; ++c) {
            load(c, s);
            // each thread stores only the columns it has already read for the last time
            if (p.residual_out != nullptr)
                norm_store_res<IoT, kVec>(p.residual_out, row * p.residual_out_stride, p.res_f32,
                                          p.dim, c, tid, n, s);
            float w[8], b[8];
            if (p.weight != nullptr) norm_load<float, kVec>(p.weight, p.dim, c, tid, n, 0.0f, w);
            if (p.bias != nullptr) norm_load<float, kVec>(p.bias, p.dim, c, tid, n, 0.0f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] = fmaf((s[i] - mean) * rstd, p.weight != nullptr ? w[i] : 1.0f,
                            p.bias != nullptr ? b[i] : 0.0f);
            norm_store<IoT, kVec>(out, p.dim, c, tid, n, s);
        }
    }
}

// Backward, the row in registers; teams as in the forward.  Every CTA writes
// its column sums to partial[blockIdx.x] (dw then db, those asked for).
template <typename IoT, int kV, bool kVec>
__global__ void __launch_bounds__(kV == 1 ? 1024 : 32 * kNormRowsPerCta, 1)
    layer_norm_bwd_kernel(const __grid_constant__ NormParams p) {
    __shared__ float buf[2 * 64];
    extern __shared__ float cols[];          // several rows per CTA: [blockDim.y][2][dim]
    const int tid = threadIdx.x, n = blockDim.x;
    int turn = 0;
    float w[kV][8], dw[kV][8], db[kV][8];
#pragma unroll
    for (int c = 0; c < kV; ++c) {
        if (p.weight != nullptr) norm_load<float, kVec>(p.weight, p.dim, c, tid, n, 0.0f, w[c]);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) w[c][i] = 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = db[c][i] = 0.0f;
    }
    const float inv_dim = 1.0f / (float)p.dim;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < p.rows; row += step) {
        const float mean = p.rms ? 0.0f : p.mean_in[row];
        const float rstd = p.rstd_in[row];
        float xh[kV][8], q[kV][8];
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            norm_load_res<IoT, kVec>(p.x, row * p.x_stride, p.res_f32, p.dim, c, tid, n, xh[c]);
            norm_load<IoT, kVec>(static_cast<const IoT*>(p.dout) + row * p.out_stride, p.dim, c, tid,
                                 n, 0.0f, q[c]);
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float h = (xh[c][i] - mean) * rstd;
                xh[c][i] = h;
                dw[c][i] = fmaf(q[c][i], h, dw[c][i]);
                db[c][i] += q[c][i];
                q[c][i] *= w[c][i];
                if (norm_col<kVec>(c, i, tid, n) < p.dim) {
                    sum[0] += q[c][i];
                    sum[1] = fmaf(q[c][i], h, sum[1]);
                }
            }
        team_sum(sum, buf, turn);
        const float c1 = p.rms ? 0.0f : sum[0] * inv_dim;
        const float c2 = sum[1] * inv_dim;
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            float ds[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) ds[i] = rstd * (q[c][i] - fmaf(xh[c][i], c2, c1));
            if (p.dresidual_out != nullptr) {
                float r[8];
                norm_load_res<IoT, kVec>(p.dresidual_out, row * p.residual_out_stride, p.res_f32,
                                         p.dim, c, tid, n, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) ds[i] += r[i];
            }
            norm_store<IoT, kVec>(static_cast<IoT*>(p.dx) + row * p.dx_stride, p.dim, c, tid, n, ds);
            if (p.dresidual != nullptr)
                norm_store_res<IoT, kVec>(p.dresidual, row * p.dresidual_stride, p.res_f32, p.dim, c,
                                          tid, n, ds);
        }
    }
    if (p.partial == nullptr) return;
    float* part = p.partial + (int64_t)blockIdx.x * (p.has_dw + p.has_db) * p.dim;
    float* part_db = part + (p.has_dw ? p.dim : 0);
    if (blockDim.y == 1) {
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            if (p.has_dw) norm_store<float, kVec>(part, p.dim, c, tid, n, dw[c]);
            if (p.has_db) norm_store<float, kVec>(part_db, p.dim, c, tid, n, db[c]);
        }
        return;
    }
    float* mine = cols + threadIdx.y * 2 * p.dim;
#pragma unroll
    for (int c = 0; c < kV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = norm_col<kVec>(c, i, tid, n);
            if (col < p.dim) {
                mine[col] = dw[c][i];
                mine[p.dim + col] = db[c][i];
            }
        }
    __syncthreads();
    for (int j = threadIdx.y * 32 + tid; j < 2 * p.dim; j += 32 * blockDim.y) {
        float sum = 0.0f;
        for (int y = 0; y < (int)blockDim.y; ++y) sum += cols[y * 2 * p.dim + j];
        if (j < p.dim) {
            if (p.has_dw) part[j] = sum;
        } else if (p.has_db) {
            part_db[j - p.dim] = sum;
        }
    }
}

// Backward for wider rows: ds with the row read twice ...
template <typename IoT, bool kVec>
__global__ void __launch_bounds__(kNormWideThreads)
    layer_norm_bwd_wide_kernel(const __grid_constant__ NormParams p) {
    __shared__ float buf[2 * 64];
    const int tid = threadIdx.x, n = blockDim.x;
    const int chunks = (p.dim + n * kNormElems - 1) / (n * kNormElems);
    const float inv_dim = 1.0f / (float)p.dim;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float mean = p.rms ? 0.0f : p.mean_in[row];
        const float rstd = p.rstd_in[row];
        auto load = [&](int c, float (&xh)[8], float (&q)[8]) {
            norm_load_res<IoT, kVec>(p.x, row * p.x_stride, p.res_f32, p.dim, c, tid, n, xh);
            norm_load<IoT, kVec>(static_cast<const IoT*>(p.dout) + row * p.out_stride, p.dim, c, tid,
                                 n, 0.0f, q);
            float w[8];
            if (p.weight != nullptr) norm_load<float, kVec>(p.weight, p.dim, c, tid, n, 0.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xh[i] = (xh[i] - mean) * rstd;
                if (p.weight != nullptr) q[i] *= w[i];
            }
        };
        float xh[8], q[8];
        float sum[2] = {0.0f, 0.0f};
        for (int c = 0; c < chunks; ++c) {
            load(c, xh, q);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (norm_col<kVec>(c, i, tid, n) < p.dim) {
                    sum[0] += q[i];
                    sum[1] = fmaf(q[i], xh[i], sum[1]);
                }
        }
        team_sum(sum, buf, turn);
        const float c1 = p.rms ? 0.0f : sum[0] * inv_dim;
        const float c2 = sum[1] * inv_dim;
        for (int c = 0; c < chunks; ++c) {
            load(c, xh, q);
            float ds[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) ds[i] = rstd * (q[i] - fmaf(xh[i], c2, c1));
            if (p.dresidual_out != nullptr) {
                float r[8];
                norm_load_res<IoT, kVec>(p.dresidual_out, row * p.residual_out_stride, p.res_f32,
                                         p.dim, c, tid, n, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) ds[i] += r[i];
            }
            norm_store<IoT, kVec>(static_cast<IoT*>(p.dx) + row * p.dx_stride, p.dim, c, tid, n, ds);
            if (p.dresidual != nullptr)
                norm_store_res<IoT, kVec>(p.dresidual, row * p.dresidual_stride, p.res_f32, p.dim, c,
                                          tid, n, ds);
        }
    }
}

// ... and their column sums: thread (x, y) walks rows y, y + step, ... of
// column block x, one column per thread; row slice gridDim.y writes partial[y].
constexpr int kNormColThreads = 256;

template <typename IoT>
__global__ void __launch_bounds__(kNormColThreads)
    layer_norm_bwd_cols_kernel(const __grid_constant__ NormParams p) {
    const int col = blockIdx.x * kNormColThreads + threadIdx.x;
    if (col >= p.dim) return;
    float dw = 0.0f, db = 0.0f;
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const int64_t si = row * p.x_stride + col;
        const float s = p.res_f32 ? static_cast<const float*>(p.x)[si]
                                  : DType<IoT>::load(static_cast<const IoT*>(p.x) + si);
        const float d = DType<IoT>::load(static_cast<const IoT*>(p.dout) + row * p.out_stride + col);
        const float mean = p.rms ? 0.0f : p.mean_in[row];
        dw = fmaf(d, (s - mean) * p.rstd_in[row], dw);
        db += d;
    }
    float* part = p.partial + (int64_t)blockIdx.y * (p.has_dw + p.has_db) * p.dim;
    if (p.has_dw) part[col] = dw;
    if (p.has_db) part[(p.has_dw ? p.dim : 0) + col] = db;
}

// ---------------------------------------------------------------- column sums

// Sums the rows of partial[rows][cols] in a fixed order: columns below `split`
// go to first[], the others to second[] (either may be null).  A CTA takes 32
// columns; its 32 warps take rows y, y + 32, ... and are added in order.
constexpr int kColSumThreads = 1024;

static __global__ void __launch_bounds__(kColSumThreads)
    column_sum_kernel(const float* __restrict__ partial, int64_t rows, int64_t cols, int64_t split,
                      float* first, float* second) {
    __shared__ float acc[32][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (col < cols) {
#pragma unroll 8
        for (int64_t r = y; r < rows; r += 32) sum += partial[r * cols + col];
    }
    acc[y][lane] = sum;
    __syncthreads();
    if (y == 0 && col < cols) {
        float total = 0.0f;
#pragma unroll
        for (int k = 0; k < 32; ++k) total += acc[k][lane];
        if (col < split) {
            if (first != nullptr) first[col] = total;
        } else if (second != nullptr) {
            second[col - split] = total;
        }
    }
}

}  // namespace mamba
