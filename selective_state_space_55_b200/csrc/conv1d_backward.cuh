// Backward pass of the short causal convolution (sm_100a).
//
// With pre_t = bias + sum_{k<W} w_k x_{t-W+1+k} and out_t = act(pre_t):
//
//   dpre_t = dout_t act'(pre_t),   silu'(p) = sg (1 + p (1 - sg)), sg = sigmoid(p)
//   dx_s   = sum_k w_k dpre_{s+W-1-k}  (+ dfinal of the last W inputs)
//   dw_k   = sum_{b,t} dpre_t x_{t-W+1+k},   dbias = sum_{b,t} dpre_t
//
// where x at negative times is the initial conv state (its gradient is the
// same sum at those times).  HBM-bound: x and dout are read and dx is written
// once.  A warp owns a stretch of one row and walks it from its end, 256 steps
// at a time, eight per lane: the W-1 inputs before a lane's steps come from the
// lane below by shuffle, the W-1 dpre after them from the lane above, or, for
// the last lane, from the tile done before.  Only at the two ends of a stretch
// are neighbours recomputed.  The weight and bias sums stay in registers until
// the stretch ends; each stretch leaves one partial per sum, and a second
// launch adds the partials in a fixed order.
#pragma once

#include "conv1d.cuh"
#include "row_vectors.cuh"

namespace mamba {

constexpr int kConvBwdWarps = 8;

struct ConvBwdParams {
    const void* x;
    const void* dout;
    const float* weight;       // (dim, W)
    const float* bias;         // (dim) or null
    const void* init;          // (batch, dim, W) or null
    const void* dfinal;        // (batch, dim, W) or null
    void* dx;
    void* dinit;               // (batch, dim, W) or null
    float* partial;            // [batch * stretches][dim W | dim]: weight sums, then bias sums
    int64_t dim, seqlen, chains;
    int64_t stretch_tiles;     // tiles of 256 steps per stretch
    int64_t stretches;         // per row
    int silu;
};

template <int kW>
__device__ __forceinline__ float conv_dpre(float pre, float dout, int silu) {
    if (!silu) return dout;
    const float sg = __fdividef(1.0f, 1.0f + ex2_approx(-pre * kLog2e));
    return dout * sg * fmaf(pre, 1.0f - sg, 1.0f);
}

// dpre at one step, everything read from memory (0 outside the row).
template <typename IoT, int kW>
__device__ __forceinline__ float conv_dpre_at(const ConvBwdParams& p, const IoT* x, const IoT* dout,
                                              const IoT* init, const float (&w)[kW], float b,
                                              int64_t t) {
    if (t < 0 || t >= p.seqlen) return 0.0f;
    float pre = b;
#pragma unroll
    for (int k = 0; k < kW; ++k) {
        const int64_t s = t - (kW - 1) + k;
        const float xs = s >= 0 ? DType<IoT>::load(x + s)
                                : (init != nullptr ? DType<IoT>::load(init + kW + s) : 0.0f);
        pre = fmaf(w[k], xs, pre);
    }
    return conv_dpre<kW>(pre, DType<IoT>::load(dout + t), p.silu);
}

template <typename IoT, int kW>
__global__ void __launch_bounds__(kConvBwdWarps * 32)
    causal_conv1d_bwd_kernel(const __grid_constant__ ConvBwdParams p) {
    constexpr int H = kW > 1 ? kW - 1 : 1;               // neighbours on each side
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kConvBwdWarps + (threadIdx.x >> 5);
    if (unit >= p.chains * p.stretches) return;          // whole warp leaves together
    const int64_t chain = unit / p.stretches, stretch = unit % p.stretches;
    const int64_t d = chain % p.dim, L = p.seqlen;
    const IoT* x = static_cast<const IoT*>(p.x) + chain * L;
    const IoT* dout = static_cast<const IoT*>(p.dout) + chain * L;
    IoT* dx = static_cast<IoT*>(p.dx) + chain * L;
    const IoT* init = p.init != nullptr ? static_cast<const IoT*>(p.init) + chain * kW : nullptr;
    const IoT* dfinal = p.dfinal != nullptr ? static_cast<const IoT*>(p.dfinal) + chain * kW : nullptr;
    float w[kW];
#pragma unroll
    for (int k = 0; k < kW; ++k) w[k] = p.weight[d * kW + k];
    const float b = p.bias != nullptr ? p.bias[d] : 0.0f;

    // Stretch in steps: tiles start at multiples of 256 minus the row's phase.
    const int phase = row_phase(x);
    const int64_t begin = stretch * p.stretch_tiles * kWarpSteps - phase;
    const int64_t end = begin + p.stretch_tiles * kWarpSteps;
    const int64_t lo = begin > 0 ? begin : 0;
    const int64_t hi = end < L ? end : L;

    float dw[kW], db = 0.0f;
#pragma unroll
    for (int k = 0; k < kW; ++k) dw[k] = 0.0f;
    float later[H];                                      // the first H dpre after the tile (lane 31)
#pragma unroll
    for (int i = 0; i < H; ++i) later[i] = 0.0f;
    if (kW > 1 && hi > lo && hi < L) {
        const float mine = lane < kW - 1 ? conv_dpre_at<IoT, kW>(p, x, dout, init, w, b, hi + lane) : 0.0f;
#pragma unroll
        for (int i = 0; i < kW - 1; ++i) later[i] = __shfl_sync(0xffffffffu, mine, i);
    }
    const int64_t tiles = hi > lo ? (hi - begin + kWarpSteps - 1) / kWarpSteps : 0;
    for (int64_t tile = tiles - 1; tile >= 0; --tile) {
        const int64_t t0 = begin + tile * kWarpSteps + lane * kLaneSteps;
        float xv[8], dv[8], before[H];
        load_steps(x, t0, lo, hi, 0.0f, xv);
        load_steps(dout, t0, lo, hi, 0.0f, dv);
#pragma unroll
        for (int i = 0; i < H; ++i) before[i] = 0.0f;
        if (kW > 1) {
            // The kW-1 inputs before t0.  Lane 0, and the lane that holds the row's
            // or the stretch's first steps, read them from memory.
            float mem[H];
            const bool edge = lane == 0 || (t0 - (kW - 1) < lo);
#pragma unroll
            for (int i = 0; i < kW - 1; ++i) {
                mem[i] = 0.0f;
                const int64_t s = t0 - (kW - 1) + i;
                if (edge && s < hi) {
                    if (s >= 0) mem[i] = DType<IoT>::load(x + s);
                    else if (init != nullptr && s >= -kW) mem[i] = DType<IoT>::load(init + kW + s);
                }
            }
#pragma unroll
            for (int i = 0; i < kW - 1; ++i) {
                const float up = __shfl_up_sync(0xffffffffu, xv[8 - (kW - 1) + i], 1);
                before[i] = edge ? mem[i] : up;
            }
            // A lane whose steps start before the row (phase > 0) sees the initial
            // state inside its own eight.
            if (t0 < 0 && init != nullptr)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t s = t0 + i;
                    if (s < 0 && s >= -kW) xv[i] = DType<IoT>::load(init + kW + s);
                }
        }
        float dp[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float pre = b;
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                const int j = i - (kW - 1) + k;
                pre = fmaf(w[k], j >= 0 ? xv[j] : before[kW - 1 + j], pre);
            }
            // steps outside [lo, hi) have dout 0 (pre may be anything there)
            const bool in = t0 + i >= lo && t0 + i < hi;
            dp[i] = in ? conv_dpre<kW>(pre, dv[i], p.silu) : 0.0f;
            db += dp[i];
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                const int j = i - (kW - 1) + k;
                const float xs = j >= 0 ? xv[j] : before[kW - 1 + j];
                if (in) dw[k] = fmaf(dp[i], xs, dw[k]);
            }
        }
        // dpre after this lane's steps: the lane above, or the tile done before.
        float after[H];
#pragma unroll
        for (int i = 0; i < H; ++i) after[i] = 0.0f;
        if (kW > 1) {
#pragma unroll
            for (int i = 0; i < kW - 1; ++i) {
                const float down = __shfl_down_sync(0xffffffffu, dp[i], 1);
                after[i] = lane == 31 ? later[i] : down;
            }
#pragma unroll
            for (int i = 0; i < kW - 1; ++i) later[i] = __shfl_sync(0xffffffffu, dp[i], 0);
        }
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float acc = 0.0f;
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                const int j = i + kW - 1 - k;
                acc = fmaf(w[k], j < 8 ? dp[j] : after[j - 8 < H ? j - 8 : 0], acc);
            }
            o[i] = acc;
        }
        if (dfinal != nullptr && t0 + 8 > L - kW)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t t = t0 + i;
                if (t >= L - kW && t >= 0 && t < L) o[i] += DType<IoT>::load(dfinal + (t + kW - L));
            }
        store_steps(dx, t0, lo, hi, o);
    }
    // Gradient of the initial state: the same sum at times -W .. -1.
    if (p.dinit != nullptr && stretch == 0 && lane < kW) {
        const int64_t s = lane - kW;
        float acc = 0.0f;
#pragma unroll
        for (int k = 0; k < kW; ++k)
            acc = fmaf(w[k], conv_dpre_at<IoT, kW>(p, x, dout, init, w, b, s + kW - 1 - k), acc);
        if (dfinal != nullptr && lane >= L) acc += DType<IoT>::load(dfinal + (lane - L));
        DType<IoT>::store(static_cast<IoT*>(p.dinit) + chain * kW + lane, acc);
    }
    float* part = p.partial + ((chain / p.dim) * p.stretches + stretch) * (kW + 1) * p.dim;
#pragma unroll
    for (int k = 0; k <= kW; ++k) {
        float v = k < kW ? dw[k < kW ? k : 0] : db;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) part[k < kW ? d * kW + k : p.dim * kW + d] = v;
    }
}

}  // namespace mamba
