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
// A row stays in the registers of one team of warps, kV chunks of 8 elements per
// lane, so each tensor crosses HBM once and all of a row's loads are under way
// together; the fewer warps share a row, the fewer reductions, barriers and
// addresses per element (2560 columns, 16384 rows bf16: 5 chunks on 2 warps
// against 1 chunk on 10, see the plan).  The variance is summed from
// (s - mean)^2 in a second reduction over the registers, so an offset far above
// the spread costs no digits.  The backward's column sums stay in the registers
// of the lane that owns the columns while the CTA walks its rows; each CTA
// leaves one partial row per sum, and a second launch adds the partial rows in
// a fixed order (no atomics: results repeat bit for bit).
#pragma once

#include "row_vectors.cuh"

namespace mamba {

#ifndef NBAHEAD
#define NBAHEAD 12
#endif
#ifndef NFAHEAD
#define NFAHEAD 2
#endif
constexpr int kNormElems = 8;            // consecutive elements per lane and chunk
constexpr int kNormFwdChunks = 8;        // most chunks per lane, forward and backward
constexpr int kNormBwdChunks = 2;
constexpr int kNormFewChunks = 2;        // up to here a team may have kNormFewWarps warps
constexpr int kNormCtaWarps = 8;         // warps of a CTA: whole teams side by side
constexpr int kNormFewWarps = 16;        // of a team with few chunks per lane
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

// The team's size again, in a way that keeps the element path's 8 kV addresses
// per tensor from being kept in registers from row to row.
template <bool kVec>
__device__ __forceinline__ int norm_opaque(int n) {
    if constexpr (!kVec) asm volatile("" : "+r"(n));
    return n;
}

// Chunk c of a row as it lies in memory (columns from dim on: 0).
template <typename T, bool kVec>
struct NormRaw {
    uint4 q[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* row, int dim, int c, int tid, int n) {
        const int col = norm_col<true>(c, 0, tid, n);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            q[i] = col < dim ? reinterpret_cast<const uint4*>(row + col)[i] : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack_steps<T>(q, v); }
};

template <typename T>
struct NormRaw<T, false> {
    float q[8];
    __device__ __forceinline__ void load(const T* row, int dim, int c, int tid, int n) {
        int col = norm_col<false>(c, 0, tid, n);
        const T* at = row + col;
#pragma unroll
        for (int i = 0; i < 8; ++i, col += n, at += n) q[i] = col < dim ? DType<T>::load(at) : 0.0f;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = q[i];
    }
};

template <typename T, bool kVec>
__device__ __forceinline__ void norm_load(const T* row, int dim, int c, int tid, int n, float (&v)[8]) {
    NormRaw<T, kVec> r;
    r.load(row, dim, c, tid, n);
    r.get(v);
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

template <typename T, bool kVec>
__device__ __forceinline__ void norm_store(T* row, int dim, int c, int tid, int n,
                                           const float (&v)[8]) {
    if constexpr (kVec) {
        const int col = norm_col<true>(c, 0, tid, n);
        if (col < dim) store8_vec(row + col, v);
    } else {
        int col = norm_col<false>(c, 0, tid, n);
        T* at = row + col;
#pragma unroll
        for (int i = 0; i < 8; ++i, col += n, at += n)
            if (col < dim) DType<T>::store(at, v[i]);
    }
}

// The residual stream's tensors: fp32, or the type of x.
template <typename IoT, bool kVec>
__device__ __forceinline__ void norm_load_res(const void* base, int64_t offset, int f32, int dim,
                                              int c, int tid, int n, float (&v)[8]) {
    if (f32) norm_load<float, kVec>(static_cast<const float*>(base) + offset, dim, c, tid, n, v);
    else norm_load<IoT, kVec>(static_cast<const IoT*>(base) + offset, dim, c, tid, n, v);
}

template <typename IoT, bool kVec>
__device__ __forceinline__ void norm_store_res(void* base, int64_t offset, int f32, int dim, int c,
                                               int tid, int n, const float (&v)[8]) {
    if (f32) norm_store<float, kVec>(static_cast<float*>(base) + offset, dim, c, tid, n, v);
    else norm_store<IoT, kVec>(static_cast<IoT*>(base) + offset, dim, c, tid, n, v);
}

// Sums of kN values over the team: blockDim.x threads (threadIdx.y numbers the
// CTA's teams); every thread gets them.  `buf` is [2][32 kN] shared floats used
// in turn, so one barrier per call is enough.
template <int kN>
__device__ __forceinline__ void team_sum(float (&v)[kN], float* buf, int& turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (blockDim.x > 32) {
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        float* b = buf + (turn * 32 + threadIdx.y * warps) * kN;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < kN; ++k) b[(threadIdx.x >> 5) * kN + k] = v[k];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
#pragma unroll
        for (int k = 0; k < kN; ++k) v[k] = lane < warps ? b[lane * kN + k] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        turn ^= 1;
    }
}

// A lane's weights: in registers for a single chunk, else in shared memory,
// padded to whole chunks.
template <int kV, bool kVec>
struct NormWeights {
    static constexpr bool kRegs = kV == 1;
    float reg[kRegs ? kV : 1][8];
    const float* shared;

    // `fill` where there are no weights; every thread of the CTA calls it.
    __device__ __forceinline__ void init(const float* w, float fill, float* room, int dim, int tid, int n) {
        shared = room;
        if constexpr (kRegs) {
#pragma unroll
            for (int c = 0; c < kV; ++c) {
                if (w != nullptr) norm_load<float, kVec>(w, dim, c, tid, n, reg[c]);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) reg[c][i] = fill;
            }
        } else {
            const int threads = blockDim.x * blockDim.y, me = threadIdx.y * blockDim.x + threadIdx.x;
            for (int j = me; j < kV * 8 * n; j += threads) room[j] = j < dim ? (w != nullptr ? w[j] : fill) : 0.0f;
        }
    }
    __device__ __forceinline__ void get(int c, int tid, int n, float (&v)[8]) const {
        if constexpr (kRegs) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = reg[c][i];
        } else if constexpr (kVec) {
            const float4* q = reinterpret_cast<const float4*>(shared + norm_col<true>(c, 0, tid, n));
            const float4 a = q[0], b = q[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = shared[norm_col<false>(c, i, tid, n)];
        }
    }
};

// A team's row as it lies in memory.  ResT: the residual stream's type.
template <typename IoT, typename ResT, int kV, bool kVec>
struct NormFwdRow {
    NormRaw<IoT, kVec> x[kV];
    NormRaw<ResT, kVec> r[kV];
    __device__ __forceinline__ void load(const NormParams& p, int64_t row, int tid, int n) {
#pragma unroll
        for (int c = 0; c < kV; ++c)
            x[c].load(static_cast<const IoT*>(p.x) + row * p.x_stride, p.dim, c, tid, n);
        if (p.residual != nullptr)
#pragma unroll
            for (int c = 0; c < kV; ++c)
                r[c].load(static_cast<const ResT*>(p.residual) + row * p.residual_stride, p.dim, c, tid, n);
    }
    // Loads and sum at once: fewer registers than load, then get.
    static __device__ __forceinline__ void fetch(const NormParams& p, int64_t row, int tid, int n, float (&s)[kV][8]) {
        NormRaw<IoT, kVec> x[kV];
#pragma unroll
        for (int c = 0; c < kV; ++c)
            x[c].load(static_cast<const IoT*>(p.x) + row * p.x_stride, p.dim, c, tid, n);
        if (p.residual == nullptr) {
#pragma unroll
            for (int c = 0; c < kV; ++c) x[c].get(s[c]);
            return;
        }
        const ResT* res = static_cast<const ResT*>(p.residual) + row * p.residual_stride;
        NormRaw<ResT, kVec> r[kV];
#pragma unroll
        for (int c = 0; c < kV; ++c) r[c].load(res, p.dim, c, tid, n);
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            float v[8];
            r[c].get(s[c]);
            x[c].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[c][i] += v[i];
        }
    }
    __device__ __forceinline__ void get(const NormParams& p, float (&s)[kV][8]) const {
        if (p.residual == nullptr) {
#pragma unroll
            for (int c = 0; c < kV; ++c) x[c].get(s[c]);
        } else {
#pragma unroll
            for (int c = 0; c < kV; ++c) {
                float v[8];
                x[c].get(v);
                r[c].get(s[c]);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[c][i] += v[i];
            }
        }
    }
};

// Forward, the row in registers: a team of blockDim.x threads per row,
// blockDim.y teams side by side.  With few chunks per lane the next row is
// requested before this one is reduced.
template <typename IoT, typename ResT, int kV, bool kVec>
__global__ void __launch_bounds__(32 * (kV <= kNormFewChunks ? kNormFewWarps : kNormCtaWarps),
                                  kV <= kNormFewChunks ? 1 : 2)
    layer_norm_fwd_kernel(const __grid_constant__ NormParams p) {
    __shared__ float buf[2 * 32];
    extern __shared__ float4 room[];                 // weights and bias, when not in registers
    constexpr bool kAhead = kV <= NFAHEAD;
    const int tid = threadIdx.x;
    int n = blockDim.x, turn = 0;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    NormFwdRow<IoT, ResT, kV, kVec> ahead;
    if (kAhead && row < p.rows) ahead.load(p, row, tid, n);
    NormWeights<kV, kVec> w, b;
    w.init(p.weight, 1.0f, reinterpret_cast<float*>(room), p.dim, tid, n);
    b.init(p.bias, 0.0f, reinterpret_cast<float*>(room) + kV * 8 * n, p.dim, tid, n);
    if constexpr (!NormWeights<kV, kVec>::kRegs) __syncthreads();
    const float inv_dim = 1.0f / (float)p.dim;
    for (; row < p.rows; row += step) {
        n = norm_opaque<kVec>(n);
        float s[kV][8];
        if constexpr (kAhead) {
            ahead.get(p, s);
            if (row + step < p.rows) ahead.load(p, row + step, tid, n);
        } else {
            NormFwdRow<IoT, ResT, kV, kVec>::fetch(p, row, tid, n, s);
        }
        if (p.residual_out != nullptr)
#pragma unroll
            for (int c = 0; c < kV; ++c)
                norm_store<ResT, kVec>(static_cast<ResT*>(p.residual_out) + row * p.residual_out_stride,
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
        for (int c = 0; c < kV; ++c) {
            // columns from dim on hold 0, not the mean: they stay out
            if constexpr (kVec) {
                if (norm_col<true>(c, 0, tid, n) >= p.dim) continue;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[c][i] -= mean;
                if (kVec || norm_col<false>(c, i, tid, n) < p.dim) sq[0] = fmaf(s[c][i], s[c][i], sq[0]);
            }
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
            float wv[8], bv[8];
            w.get(c, tid, n, wv);
            b.get(c, tid, n, bv);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[c][i] = fmaf(s[c][i] * rstd, wv[i], bv[i]);
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
            norm_load<IoT, kVec>(x, p.dim, c, tid, n, s);
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
            if (p.weight != nullptr) norm_load<float, kVec>(p.weight, p.dim, c, tid, n, w);
            if (p.bias != nullptr) norm_load<float, kVec>(p.bias, p.dim, c, tid, n, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] = fmaf((s[i] - mean) * rstd, p.weight != nullptr ? w[i] : 1.0f,
                            p.bias != nullptr ? b[i] : 0.0f);
            norm_store<IoT, kVec>(out, p.dim, c, tid, n, s);
        }
    }
}

template <typename IoT, typename ResT, int kV, bool kVec>
struct NormBwdRow {
    NormRaw<IoT, kVec> d[kV];
    NormRaw<ResT, kVec> s[kV], r[kV];
    float mean, rstd;
    __device__ __forceinline__ void load(const NormParams& p, int64_t row, int tid, int n) {
        mean = p.rms ? 0.0f : p.mean_in[row];
        rstd = p.rstd_in[row];
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            d[c].load(static_cast<const IoT*>(p.dout) + row * p.out_stride, p.dim, c, tid, n);
            s[c].load(static_cast<const ResT*>(p.x) + row * p.x_stride, p.dim, c, tid, n);
        }
    }
    __device__ __forceinline__ void load_res(const NormParams& p, int64_t row, int tid, int n) {
        if (p.dresidual_out == nullptr) return;
#pragma unroll
        for (int c = 0; c < kV; ++c)
            r[c].load(static_cast<const ResT*>(p.dresidual_out) + row * p.residual_out_stride, p.dim, c, tid, n);
    }
};

// Backward, the row in registers; teams as in the forward, the next row
// requested while this one is reduced.  Every CTA writes its column sums to
// partial[blockIdx.x] (dw then db, those asked for), the teams' sums added in
// order.
template <typename IoT, typename ResT, int kV, bool kVec>
__global__ void __launch_bounds__(32 * kNormFewWarps, 1)
    layer_norm_bwd_kernel(const __grid_constant__ NormParams p) {
    __shared__ float buf[2 * 64];
    extern __shared__ float4 room[];         // weights while rows go by, then the teams' column sums
    // registers for the next row: up to 24 of them
    constexpr bool kAhead = kV * (sizeof(IoT) + 2 * sizeof(ResT)) <= NBAHEAD;
    const int tid = threadIdx.x;
    int n = blockDim.x, turn = 0;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    NormBwdRow<IoT, ResT, kV, kVec> ahead;
    if (kAhead && row < p.rows) {
        ahead.load(p, row, tid, n);
        ahead.load_res(p, row, tid, n);
    }
    NormWeights<kV, kVec> w;
    w.init(p.weight, 1.0f, reinterpret_cast<float*>(room), p.dim, tid, n);
    if constexpr (!NormWeights<kV, kVec>::kRegs) __syncthreads();
    float dw[kV][8], db[kV][8];
#pragma unroll
    for (int c = 0; c < kV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = db[c][i] = 0.0f;
    const float inv_dim = 1.0f / (float)p.dim;
    for (; row < p.rows; row += step) {
        n = norm_opaque<kVec>(n);
        NormBwdRow<IoT, ResT, kV, kVec> here;
        if (!kAhead) {
            here.load(p, row, tid, n);
            here.load_res(p, row, tid, n);
        }
        NormBwdRow<IoT, ResT, kV, kVec>& in = kAhead ? ahead : here;
        const float rstd = in.rstd, mean = in.mean;
        float xh[kV][8], q[kV][8];
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            float wv[8];
            in.d[c].get(q[c]);               // 0 from dim on: nothing is added there
            in.s[c].get(xh[c]);
            w.get(c, tid, n, wv);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float h = (xh[c][i] - mean) * rstd;
                xh[c][i] = h;
                dw[c][i] = fmaf(q[c][i], h, dw[c][i]);
                db[c][i] += q[c][i];
                q[c][i] *= wv[i];
                sum[0] += q[c][i];
                sum[1] = fmaf(q[c][i], h, sum[1]);
            }
        }
        if (kAhead && row + step < p.rows) in.load(p, row + step, tid, n);
        team_sum(sum, buf, turn);
        const float c1 = p.rms ? 0.0f : sum[0] * inv_dim;
        const float c2 = sum[1] * inv_dim;
#pragma unroll
        for (int c = 0; c < kV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) q[c][i] = rstd * (q[c][i] - fmaf(xh[c][i], c2, c1));
        if (p.dresidual_out != nullptr)
#pragma unroll
            for (int c = 0; c < kV; ++c) {
                float v[8];
                in.r[c].get(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) q[c][i] += v[i];
            }
        if (kAhead && row + step < p.rows) in.load_res(p, row + step, tid, n);
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            norm_store<IoT, kVec>(static_cast<IoT*>(p.dx) + row * p.dx_stride, p.dim, c, tid, n, q[c]);
            if (p.dresidual != nullptr)
                norm_store<ResT, kVec>(static_cast<ResT*>(p.dresidual) + row * p.dresidual_stride, p.dim, c,
                                       tid, n, q[c]);
        }
    }
    if (p.partial == nullptr) return;
    // [teams' running sums: dw | db], one team after another
    const int width = kV * 8 * n;
    float* sums = reinterpret_cast<float*>(room);
    for (int y = 0; y < (int)blockDim.y; ++y) {
        if (y > 0 || !NormWeights<kV, kVec>::kRegs) __syncthreads();
        if ((int)threadIdx.y != y) continue;
        const bool last = y == (int)blockDim.y - 1;
        float* part = p.partial + (int64_t)blockIdx.x * (p.has_dw + p.has_db) * p.dim;
        float* part_db = part + (p.has_dw ? p.dim : 0);
#pragma unroll
        for (int c = 0; c < kV; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = norm_col<kVec>(c, i, tid, n);
                if (y > 0) {
                    dw[c][i] = sums[col] + dw[c][i];
                    db[c][i] = sums[width + col] + db[c][i];
                }
                if (!last) {
                    sums[col] = dw[c][i];
                    sums[width + col] = db[c][i];
                }
            }
            if (last) {
                if (p.has_dw) norm_store<float, kVec>(part, p.dim, c, tid, n, dw[c]);
                if (p.has_db) norm_store<float, kVec>(part_db, p.dim, c, tid, n, db[c]);
            }
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
                                 n, q);
            float w[8];
            if (p.weight != nullptr) norm_load<float, kVec>(p.weight, p.dim, c, tid, n, w);
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
