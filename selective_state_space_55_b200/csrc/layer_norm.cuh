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
// a fixed order (no atomics: results repeat bit for bit).  With few chunks per lane
// a team's rows come through a ring of bulk copies in shared memory, because the
// registers hold one row only.
//
// Measured, bf16 with a residual (copy rate 6529 GB/s): 32768 x 2560 forward 119 us,
// 5.65 TB/s, 87 %; backward 127 us, 5.29 TB/s, 81 %, the rest being the barriers of
// the two row reductions; 8 x 2560 forward 8 us, latency.  fp32: 248 and 236 us, 83 and
// 87 %.  Columns that are not a multiple of 8 move element by element: 32768 x 2559 203
// and 276 us, 51 and 37 %.  4096 x 16384: forward, 8 chunks per lane on 8 warps, 166 us,
// 50 %; backward, beyond the registers, where s and dout are read three times, 332 us,
// 25 %.
#pragma once

#include "row_vectors.cuh"

namespace mamba {

constexpr int kNormElems = 8;            // consecutive elements per lane and chunk
constexpr int kNormFwdChunks = 8;        // most chunks per lane, forward and backward
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

template <typename T, bool kVec>
__device__ __forceinline__ void norm_store(T* row, int dim, int c, int tid, int n,
                                           const float (&v)[8]) {
    if constexpr (kVec) {
        const int col = norm_col<true>(c, 0, tid, n);
        if (col < dim) store_eight(row + col, v);
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

// A chunk as four pairs, for packed fp32x2 arithmetic, and back.
__device__ __forceinline__ void to_pairs(const float (&v)[8], float2 (&q)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

__device__ __forceinline__ void from_pairs(const float2 (&q)[4], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = q[i].x;
        v[2 * i + 1] = q[i].y;
    }
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
        // the lanes past the warps hold 0: the steps over them can be left out, lane 0's
        // power-of-two neighbourhood holds them all, and the others read its sum
        int reach = 1;
        while (reach < warps) reach <<= 1;
        for (int o = reach >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
#pragma unroll
        for (int k = 0; k < kN; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], 0);
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

// Coming rows of a team in shared memory, brought by bulk copies that one thread
// asks for: a stage holds one row of up to kTensors tensors, each as it lies in
// memory.  `bars` are the team's barriers, one per stage.
constexpr int kNormStages = 4;               // at most

template <int kTensors>
struct NormRing {
    const unsigned char* from[kTensors];     // of the next row to ask for
    int64_t stride[kTensors];                // between a team's rows, bytes
    uint32_t bytes[kTensors], offset[kTensors];
    uint32_t data, stage_bytes, bars, at;    // at: the stage being worked on
    int64_t coming, rows, step;
    int stages, stage;
    uint32_t parity;
    int failed;                              // waits since one ran out, that one included

    // Tensor k (null: there is none) with rows of `dim` elements.
    template <typename T>
    __device__ __forceinline__ void tensor(int k, const void* base, int64_t row, int64_t row_stride, int dim) {
        from[k] = static_cast<const unsigned char*>(base) + row * row_stride * (int64_t)sizeof(T);
        stride[k] = step * row_stride * (int64_t)sizeof(T);
        bytes[k] = base != nullptr ? dim * (uint32_t)sizeof(T) : 0u;
        offset[k] = k == 0 ? 0u : offset[k - 1] + bytes[k - 1];
    }
    // After the tensors; every thread calls it, a barrier of the CTA has to follow.
    __device__ __forceinline__ void init(const float4* room, uint32_t bytes_per_stage, uint32_t team_bars, int n_stages,
                                         int64_t first, int64_t n_rows) {
        stage_bytes = bytes_per_stage;
        data = smem_u32(room) + threadIdx.y * n_stages * bytes_per_stage;
        bars = team_bars;
        at = data;
        stages = n_stages;
        stage = 0;
        parity = 0;
        failed = 0;
        coming = first;
        rows = n_rows;
        if (threadIdx.x == 0) {
            for (int k = 0; k < n_stages; ++k) mbar_init(bars + 8 * k, 1);
            fence_mbar_init();
        }
    }
    // The next row into stage `to`; one thread of the team.
    __device__ __forceinline__ void request(int to) {
        if (coming < rows && failed == 0) {
            const uint32_t bar = bars + 8 * to, dst = data + to * stage_bytes;
            uint32_t total = 0;
#pragma unroll
            for (int k = 0; k < kTensors; ++k) total += bytes[k];
            mbar_arrive_expect_tx(bar, total);
#pragma unroll
            for (int k = 0; k < kTensors; ++k)
                if (bytes[k] != 0u) bulk_load(dst + offset[k], from[k], bytes[k], bar);
        }
        coming += step;
#pragma unroll
        for (int k = 0; k < kTensors; ++k) from[k] += stride[k];
    }
    // A wait that runs out is recorded and the call's outputs are undefined.  Nothing
    // more is asked for then, and one more wait per stage keeps the CTA's shared memory
    // until the copies under way have landed.
    __device__ __forceinline__ void wait() {
        const uint32_t bar = bars + 8 * stage;
        if (failed == 0) {
            if (mbar_wait_bounded(bar, parity)) return;
            record_device_error(MAMBA_ERR_TIMEOUT);
        }
        if (failed < stages) {
            mbar_wait_bounded(bar, parity);
            ++failed;
        }
    }
    // Eight elements of tensor k from column col on; 0 where there are none.
    template <typename T>
    __device__ __forceinline__ void get(int k, int col, int dim, float (&v)[8]) const {
        uint4 q[sizeof(T) / 2];
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            q[i] = make_uint4(0, 0, 0, 0);
            if (col < dim)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w)
                             : "r"(at + offset[k] + col * (uint32_t)sizeof(T) + 16 * i)
                             : "memory");
        }
        unpack_steps<T>(q, v);
    }
    // Every thread of the team has read stage `st` (it comes from a barrier, or is
    // a single warp): it takes the row `stages` further on.
    __device__ __forceinline__ void refill(int st) {
        if (blockDim.x == 32) __syncwarp();
        if (threadIdx.x == 0) request(st);
    }
    __device__ __forceinline__ int before() const { return stage == 0 ? stages - 1 : stage - 1; }
    __device__ __forceinline__ void advance() {
        stage = stage + 1 == stages ? 0 : stage + 1;
        if (stage == 0) parity ^= 1;
        at = data + stage * stage_bytes;
    }
};

// A thread's place in consecutive rows of one tensor, `step` rows apart.
template <typename T>
struct NormWalk {
    T* at;
    int64_t stride;
    __device__ __forceinline__ NormWalk(void* base, int64_t row, int64_t row_stride, int64_t step, int col)
        : at(static_cast<T*>(base) + row * row_stride + col), stride(step * row_stride) {}
    __device__ __forceinline__ void next() { at += stride; }
};

// Loads and sums a row's x and residual at once, all loads first.
template <typename IoT, typename ResT, int kV, bool kVec>
__device__ __forceinline__ void norm_fetch(const NormParams& p, int64_t row, int tid, int n, float (&s)[kV][8]) {
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

// Forward, the row in registers: a team of blockDim.x threads per row,
// blockDim.y teams side by side.  With few chunks per lane and vectors, rows
// come through a ring of `stages`; otherwise a lane's many loads are enough.
template <typename IoT, typename ResT, int kV, bool kVec>
__global__ void __launch_bounds__(32 * (kV <= kNormFewChunks ? kNormFewWarps : kNormCtaWarps),
                                  kV <= kNormFewChunks ? 1 : 2)
    layer_norm_fwd_kernel(const __grid_constant__ NormParams p, int ring_at, int stage_bytes, int stages) {
    __shared__ float buf[2 * 32];
    __shared__ uint64_t bars[kNormCtaWarps][kNormStages];
    extern __shared__ float4 room[];                 // weights and bias, when not in registers; the ring
    constexpr bool kRing = kV <= kNormFewChunks && kVec;
    const int tid = threadIdx.x;
    int n = blockDim.x, turn = 0;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int col = norm_col<kVec>(0, 0, tid, n);
    NormRing<2> ring;                                // x, residual
    if constexpr (kRing) {
        ring.step = step;
        ring.template tensor<IoT>(0, p.x, row, p.x_stride, p.dim);
        ring.template tensor<ResT>(1, p.residual, row, p.residual_stride, p.dim);
        ring.init(room + ring_at, stage_bytes, smem_u32(&bars[threadIdx.y][0]), stages, row, p.rows);
        __syncthreads();
        if (tid == 0)
            for (int k = 0; k < stages; ++k) ring.request(k);
    }
    NormWeights<kV, kVec> w, b;
    w.init(p.weight, 1.0f, reinterpret_cast<float*>(room), p.dim, tid, n);
    b.init(p.bias, 0.0f, reinterpret_cast<float*>(room) + kV * 8 * n, p.dim, tid, n);
    if constexpr (!NormWeights<kV, kVec>::kRegs) __syncthreads();
    const float inv_dim = 1.0f / (float)p.dim;
    for (; row < p.rows; row += step) {
        n = norm_opaque<kVec>(n);
        float s[kV][8];
        if constexpr (kRing) {
            ring.wait();
#pragma unroll
            for (int c = 0; c < kV; ++c) {
                ring.template get<IoT>(0, col + c * n * kNormElems, p.dim, s[c]);
                if (p.residual != nullptr) {
                    float v[8];
                    ring.template get<ResT>(1, col + c * n * kNormElems, p.dim, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[c][i] += v[i];
                }
            }
        } else {
            norm_fetch<IoT, ResT, kV, kVec>(p, row, tid, n, s);
        }
        if (p.residual_out != nullptr)
#pragma unroll
            for (int c = 0; c < kV; ++c)
                norm_store<ResT, kVec>(static_cast<ResT*>(p.residual_out) + row * p.residual_out_stride,
                                       p.dim, c, tid, n, s[c]);
        float2 t[kV][4];
#pragma unroll
        for (int c = 0; c < kV; ++c) to_pairs(s[c], t[c]);
        float mean = 0.0f;
        if (!p.rms) {
            float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < kV; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc = __fadd2_rn(acc, t[c][i]);
            float sum[1] = {acc.x + acc.y};
            team_sum(sum, buf, turn);
            mean = sum[0] * inv_dim;
        }
        const float2 shift = make_float2(-mean, -mean);
        float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < kV; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[c][i] = __fadd2_rn(t[c][i], shift);
            // columns from dim on held 0 and now hold -mean: they stay out
            if constexpr (kVec) {
                if (norm_col<true>(c, 0, tid, n) < p.dim)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc = __ffma2_rn(t[c][i], t[c][i], acc);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (norm_col<false>(c, 2 * i, tid, n) < p.dim) acc.x = fmaf(t[c][i].x, t[c][i].x, acc.x);
                    if (norm_col<false>(c, 2 * i + 1, tid, n) < p.dim) acc.y = fmaf(t[c][i].y, t[c][i].y, acc.y);
                }
            }
        }
        float sq[1] = {acc.x + acc.y};
        team_sum(sq, buf, turn);
        if constexpr (kRing) {
            ring.refill(ring.stage);
            ring.advance();
        }
        const float rstd = 1.0f / sqrtf(fmaf(sq[0], inv_dim, p.eps));
        if (tid == 0) {
            if (p.mean != nullptr) p.mean[row] = mean;
            if (p.rstd != nullptr) p.rstd[row] = rstd;
        }
        const float2 scale = make_float2(rstd, rstd);
        IoT* out = static_cast<IoT*>(p.out) + row * p.out_stride;
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            float v[8];
            float2 wv[4], bv[4];
            w.get(c, tid, n, v);
            to_pairs(v, wv);
            b.get(c, tid, n, v);
            to_pairs(v, bv);
#pragma unroll
            for (int i = 0; i < 4; ++i) t[c][i] = __ffma2_rn(__fmul2_rn(t[c][i], scale), wv[i], bv[i]);
            from_pairs(t[c], v);
            norm_store<IoT, kVec>(out, p.dim, c, tid, n, v);
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

// Backward, the row in registers; teams as in the forward, rows through a ring
// of `stages` (element path: loaded where they are used).  Every CTA writes its
// column sums to partial[blockIdx.x] (dw then db, those asked for), the teams'
// sums added in order.
template <typename IoT, typename ResT, int kV, bool kVec>
__global__ void __launch_bounds__(32 * kNormFewWarps, 1)
    layer_norm_bwd_kernel(const __grid_constant__ NormParams p, int ring_at, int stage_bytes, int stages) {
    __shared__ float buf[2 * 64];
    __shared__ uint64_t bars[kNormCtaWarps][kNormStages];
    extern __shared__ float4 room[];         // weights while rows go by, then the teams' column sums; the ring
    const int tid = threadIdx.x;
    int n = blockDim.x, turn = 0;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int col = norm_col<kVec>(0, 0, tid, n);
    NormRing<3> ring;                        // dout, s, dresidual_out
    if constexpr (kVec) {
        ring.step = step;
        ring.template tensor<IoT>(0, p.dout, row, p.out_stride, p.dim);
        ring.template tensor<ResT>(1, p.x, row, p.x_stride, p.dim);
        ring.template tensor<ResT>(2, p.dresidual_out, row, p.residual_out_stride, p.dim);
        ring.init(room + ring_at, stage_bytes, smem_u32(&bars[threadIdx.y][0]), stages, row, p.rows);
        __syncthreads();
        if (tid == 0)
            for (int k = 0; k < stages; ++k) ring.request(k);
    }
    NormWalk<IoT> dx(p.dx, row, p.dx_stride, step, col);
    NormWalk<ResT> dr(p.dresidual, row, p.dresidual_stride, step, col);
    bool started = false;
    float mean = 0.0f, rstd = 0.0f;
    if (row < p.rows) {
        mean = p.rms ? 0.0f : p.mean_in[row];
        rstd = p.rstd_in[row];
    }
    NormWeights<kV, kVec> w;
    w.init(p.weight, 1.0f, reinterpret_cast<float*>(room), p.dim, tid, n);
    if constexpr (!NormWeights<kV, kVec>::kRegs) __syncthreads();
    float2 dw2[kV][4], db2[kV][4];
#pragma unroll
    for (int c = 0; c < kV; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) dw2[c][i] = db2[c][i] = make_float2(0.0f, 0.0f);
    const float inv_dim = 1.0f / (float)p.dim;
    for (; row < p.rows; row += step) {
        n = norm_opaque<kVec>(n);
        float2 xh[kV][4], q[kV][4];
        if constexpr (kVec) ring.wait();
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            float d[8], x[8];
            if constexpr (kVec) {
                ring.template get<IoT>(0, col + c * n * kNormElems, p.dim, d);
                ring.template get<ResT>(1, col + c * n * kNormElems, p.dim, x);
            } else {
                norm_load<IoT, kVec>(static_cast<const IoT*>(p.dout) + row * p.out_stride, p.dim, c, tid, n, d);
                norm_load<ResT, kVec>(static_cast<const ResT*>(p.x) + row * p.x_stride, p.dim, c, tid, n, x);
            }
            to_pairs(d, q[c]);
            to_pairs(x, xh[c]);
        }
        const float2 scale = make_float2(rstd, rstd), shift = make_float2(-mean, -mean);
        if (row + step < p.rows) {
            mean = p.rms ? 0.0f : p.mean_in[row + step];
            rstd = p.rstd_in[row + step];
        }
        float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
#pragma unroll
        for (int c = 0; c < kV; ++c) {       // dout is 0 from dim on: nothing is added there
            float v[8];
            float2 wv[4];
            w.get(c, tid, n, v);
            to_pairs(v, wv);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 h = __fmul2_rn(__fadd2_rn(xh[c][i], shift), scale);
                xh[c][i] = h;
                dw2[c][i] = __ffma2_rn(q[c][i], h, dw2[c][i]);
                db2[c][i] = __fadd2_rn(db2[c][i], q[c][i]);
                q[c][i] = __fmul2_rn(q[c][i], wv[i]);
                s0 = __fadd2_rn(s0, q[c][i]);
                s1 = __ffma2_rn(q[c][i], h, s1);
            }
        }
        float sum[2] = {s0.x + s0.y, s1.x + s1.y};
        team_sum(sum, buf, turn);
        // past this barrier the row before is done with
        if constexpr (kVec) {
            if (started) ring.refill(ring.before());
            started = true;
        }
        const float c1 = p.rms ? 0.0f : -sum[0] * inv_dim;
        const float c2 = -sum[1] * inv_dim;
#pragma unroll
        for (int c = 0; c < kV; ++c) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[c][i] = __fmul2_rn(scale, __fadd2_rn(q[c][i], __ffma2_rn(xh[c][i], make_float2(c2, c2), make_float2(c1, c1))));
            if (p.dresidual_out != nullptr) {
                float2 r[4];
                if constexpr (kVec)
                    ring.template get<ResT>(2, col + c * n * kNormElems, p.dim, v);
                else
                    norm_load<ResT, kVec>(static_cast<const ResT*>(p.dresidual_out) + row * p.residual_out_stride,
                                          p.dim, c, tid, n, v);
                to_pairs(v, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) q[c][i] = __fadd2_rn(q[c][i], r[i]);
            }
            from_pairs(q[c], v);
            if constexpr (kVec) {
                if (col + c * n * kNormElems < p.dim) {
                    store_eight(dx.at + c * n * kNormElems, v);
                    if (p.dresidual != nullptr) store_eight(dr.at + c * n * kNormElems, v);
                }
            } else {
                norm_store<IoT, kVec>(static_cast<IoT*>(p.dx) + row * p.dx_stride, p.dim, c, tid, n, v);
                if (p.dresidual != nullptr)
                    norm_store<ResT, kVec>(static_cast<ResT*>(p.dresidual) + row * p.dresidual_stride, p.dim, c, tid, n, v);
            }
        }
        if constexpr (kVec) {
            ring.advance();
            dx.next();
            dr.next();
        }
    }
    if (p.partial == nullptr) return;
    float dw[kV][8], db[kV][8];
#pragma unroll
    for (int c = 0; c < kV; ++c) {
        from_pairs(dw2[c], dw[c]);
        from_pairs(db2[c], db[c]);
    }
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
    grid_dependency_wait();          // launched to overlap the kernel that writes the partial rows
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
