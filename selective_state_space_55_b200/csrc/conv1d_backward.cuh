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
// once.  A warp owns a stretch of two neighbouring rows (one per half of its
// packed fp32x2 arithmetic) and walks it from its end, 256 steps at a time,
// eight per lane: the W-1 inputs before a lane's steps come from the lane below
// by shuffle, the W-1 dpre after them from the lane above, or, for the last
// lane, from the tile done before.  Only at the two ends of a stretch are
// neighbours recomputed.  Each lane brings its own vectors of the coming tiles
// into shared memory (cp.async), three or four tiles deep, so that loads are
// under way while it computes.  The weight and bias sums stay in registers until
// the stretch ends; each stretch leaves one partial per sum, and a second
// launch adds the partials in a fixed order.
//
// Measured, W = 4 with silu (copy rate 6529 GB/s): 16 x 5120 x 2048 bf16 266 us, 3.78
// TB/s, 58 %; 8 x 5120 x 2048 fp32 252 us, 61 %.  Bound by latency: the ring and the
// registers leave 16 warps per SM, four per scheduler, which use 56 % of the issue
// slots (32 instructions per element) and wait for fixed latencies first.  Rows of odd
// length: 16 x 5120 x 1023 bf16 254 us, 30 %; of a row's five tiles, because it starts
// up to 7 steps past a boundary, the first and the last fetch their neighbours element
// by element and mask their ends.
#pragma once

#include "conv1d.cuh"
#include "row_vectors.cuh"

namespace mamba {

constexpr int kConvBwdWarps = 4;

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
    int64_t pairs;             // of rows
    int64_t stretch_tiles;     // tiles of 256 steps per stretch
    int64_t stretches;         // per row
    int silu;
};

// dout act'(pre) of two rows.
__device__ __forceinline__ float2 conv_dpre2(float2 pre, float2 dout, int silu) {
    if (!silu) return dout;
    const float2 one = make_float2(1.0f, 1.0f);
    const float2 t = __fmul2_rn(pre, make_float2(-kLog2e, -kLog2e));
    const float2 e = __fadd2_rn(make_float2(ex2_approx(t.x), ex2_approx(t.y)), one);
    const float2 sg = make_float2(rcp_approx(e.x), rcp_approx(e.y));
    const float2 rest = __ffma2_rn(sg, make_float2(-1.0f, -1.0f), one);
    return __fmul2_rn(__fmul2_rn(dout, sg), __ffma2_rn(pre, rest, one));
}

// One row of a warp's pair.
template <typename IoT, int kW>
struct ConvRow {
    const IoT *x, *dout, *init, *dfinal;
    IoT* dx;
    int64_t chain, d;
    int begin, lo, hi;                     // begin: the stretch's first step, before the row's start if negative
    bool live;

    __device__ __forceinline__ ConvRow(const ConvBwdParams& p, int64_t c, int64_t stretch) {
        live = c < p.chains;
        chain = live ? c : p.chains - 1;
        d = chain % p.dim;
        const int64_t at = chain * p.seqlen;
        x = static_cast<const IoT*>(p.x) + at;
        dout = static_cast<const IoT*>(p.dout) + at;
        dx = static_cast<IoT*>(p.dx) + at;
        init = p.init != nullptr ? static_cast<const IoT*>(p.init) + chain * kW : nullptr;
        dfinal = p.dfinal != nullptr ? static_cast<const IoT*>(p.dfinal) + chain * kW : nullptr;
        // counted in tiles, because the last stretch may end far behind the row, past 32 bits of steps
        const int phase = row_phase(x), L = (int)p.seqlen, tiles = (L + phase + kWarpSteps - 1) / kWarpSteps;
        const int first = (int)stretch * (int)p.stretch_tiles, end = first + (int)p.stretch_tiles;
        begin = first * kWarpSteps - phase;
        lo = begin > 0 ? begin : 0;
        hi = live ? (end < tiles ? end * kWarpSteps - phase : L) : lo;
    }

    // x_s at any time: the row, the initial state before it, 0 elsewhere
    __device__ __forceinline__ float input(int s, int L) const {
        if (s >= 0) return s < L && live ? DType<IoT>::load(x + s) : 0.0f;
        return init != nullptr && s >= -kW ? DType<IoT>::load(init + kW + s) : 0.0f;
    }

    // dpre at one step, everything read from memory (0 outside the row)
    __device__ __forceinline__ float dpre(const ConvBwdParams& p, const float (&w)[kW], float b, int t) const {
        if (t < 0 || t >= p.seqlen || !live) return 0.0f;
        float pre = b;
#pragma unroll
        for (int k = 0; k < kW; ++k) pre = fmaf(w[k], input(t - (kW - 1) + k, (int)p.seqlen), pre);
        const float g = DType<IoT>::load(dout + t);
        return conv_dpre2(make_float2(pre, 0.0f), make_float2(g, 0.0f), p.silu).x;
    }

    // gradient of the initial state's entry j, and the stretch's sums
    __device__ __forceinline__ void finish(const ConvBwdParams& p, const float (&w)[kW], float b, int64_t stretch,
                                           int lane, const float (&dw)[kW], float db) const {
        if (p.dinit != nullptr && stretch == 0 && lane < kW && live) {
            float acc = 0.0f;
#pragma unroll
            for (int k = 0; k < kW; ++k) acc = fmaf(w[k], dpre(p, w, b, lane - 1 - k), acc);
            if (dfinal != nullptr && lane >= p.seqlen) acc += DType<IoT>::load(dfinal + (lane - p.seqlen));
            DType<IoT>::store(static_cast<IoT*>(p.dinit) + chain * kW + lane, acc);
        }
        float* part = p.partial + ((chain / p.dim) * p.stretches + stretch) * (kW + 1) * p.dim;
#pragma unroll
        for (int k = 0; k <= kW; ++k) {
            float v = k < kW ? dw[k < kW ? k : 0] : db;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0 && live) part[k < kW ? d * kW + k : p.dim * kW + d] = v;
        }
    }
};

// A warp's ring: per stage x and dout of both rows, a lane's vectors side by side.
template <typename IoT>
struct ConvRing {
    static constexpr int kStages = sizeof(IoT) == 2 ? 4 : 3;
    static constexpr int kVecs = (int)sizeof(IoT) / 2;           // of 16 bytes, per lane and tensor
    static constexpr int kBytes = kConvBwdWarps * kStages * 4 * kVecs * 32 * 16;
};

template <typename IoT, int kW>
__global__ void __launch_bounds__(kConvBwdWarps * 32, 4)
    causal_conv1d_bwd_kernel(const __grid_constant__ ConvBwdParams p) {
    constexpr int H = kW > 1 ? kW - 1 : 1;               // neighbours on each side
    using Ring = ConvRing<IoT>;
    extern __shared__ uint4 ring_all[];                  // [warp][stage][x0, x1, dout0, dout1][vector][lane]
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kConvBwdWarps + (threadIdx.x >> 5);
    if (unit >= p.pairs * p.stretches) return;           // whole warp leaves together
    uint4* ring = ring_all + (threadIdx.x >> 5) * (Ring::kStages * 4 * Ring::kVecs * 32);
    const int64_t pair = unit / p.stretches, stretch = unit % p.stretches;
    const int L = (int)p.seqlen;
    const ConvRow<IoT, kW> r0(p, 2 * pair, stretch), r1(p, 2 * pair + 1, stretch);
    const float2 zero = make_float2(0.0f, 0.0f);
    float2 w[kW], dw[kW], db = zero;
#pragma unroll
    for (int k = 0; k < kW; ++k) {
        w[k] = make_float2(p.weight[r0.d * kW + k], p.weight[r1.d * kW + k]);
        dw[k] = zero;
    }
    const float2 b = p.bias != nullptr ? make_float2(p.bias[r0.d], p.bias[r1.d]) : zero;
    float w0[kW], w1[kW];
#pragma unroll
    for (int k = 0; k < kW; ++k) {
        w0[k] = w[k].x;
        w1[k] = w[k].y;
    }

    float2 later[H];                                     // the first H dpre after the tile (lane 31)
#pragma unroll
    for (int i = 0; i < H; ++i) later[i] = zero;
    if (kW > 1 && ((r0.live && r0.hi < L) || (r1.live && r1.hi < L))) {   // a row goes on after the stretch
        const bool ask = lane < kW - 1;
        const float2 mine = make_float2(ask ? r0.dpre(p, w0, b.x, r0.hi + lane) : 0.0f,
                                        ask ? r1.dpre(p, w1, b.y, r1.hi + lane) : 0.0f);
#pragma unroll
        for (int i = 0; i < kW - 1; ++i) later[i] = shfl2(mine, i);
    }
    const int span0 = r0.hi > r0.lo ? r0.hi - r0.begin : 0, span1 = r1.hi > r1.lo ? r1.hi - r1.begin : 0;
    const int tiles = ((span0 > span1 ? span0 : span1) + kWarpSteps - 1) / kWarpSteps;
    const int64_t total = p.chains * p.seqlen * (int64_t)sizeof(IoT);
    const Span xspan{static_cast<const unsigned char*>(p.x), static_cast<const unsigned char*>(p.x) + total};
    const Span dspan{static_cast<const unsigned char*>(p.dout), static_cast<const unsigned char*>(p.dout) + total};
    // A tile travels through the ring when dout's rows lie like x's and the tensors
    // hold all of it (what belongs to other rows is thrown away).
    const bool alike = row_phase(r0.dout) == row_phase(r0.x) && row_phase(r1.dout) == row_phase(r1.x);
    constexpr int kTileBytes = kWarpSteps * (int)sizeof(IoT);
    auto fits = [&](int tile) {
        const int o0 = r0.begin + tile * kWarpSteps, o1 = r1.begin + tile * kWarpSteps;
        return alike && tile >= 0 && xspan.holds(r0.x + o0, kTileBytes) && xspan.holds(r1.x + o1, kTileBytes) &&
               dspan.holds(r0.dout + o0, kTileBytes) && dspan.holds(r1.dout + o1, kTileBytes);
    };
    int ring_lo = 0, ring_hi = tiles;                    // only the tensors' two ends can fall outside
    while (ring_hi > 0 && !fits(ring_hi - 1)) --ring_hi;
    while (ring_lo < ring_hi && !fits(ring_lo)) ++ring_lo;
    auto in_ring = [&](int tile) { return tile >= ring_lo && tile < ring_hi; };
    // Shared address of this lane's words in a stage.
    constexpr int kStageBytes = 4 * Ring::kVecs * 32 * 16;
    const uint32_t mine = smem_u32(ring) + lane * 16;
    auto stage_of = [&](int tile) { return (uint32_t)(tile % Ring::kStages) * kStageBytes; };
    auto request = [&](int tile) {                   // one group per call, empty where nothing is asked for
        if (in_ring(tile)) {
            const uint32_t to = mine + stage_of(tile);
            const int o0 = r0.begin + tile * kWarpSteps + lane * kLaneSteps;
            const int o1 = r1.begin + tile * kWarpSteps + lane * kLaneSteps;
            const IoT* src[4] = {r0.x + o0, r1.x + o1, r0.dout + o0, r1.dout + o1};
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < Ring::kVecs; ++v)
                    copy_async16(to + (j * Ring::kVecs + v) * 512, reinterpret_cast<const uint4*>(src[j]) + v);
        }
        copy_async_commit();
    };
    auto take = [&](uint32_t from, int j, float (&v)[8]) {
        uint4 raw[Ring::kVecs];
#pragma unroll
        for (int k = 0; k < Ring::kVecs; ++k)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(raw[k].x), "=r"(raw[k].y), "=r"(raw[k].z), "=r"(raw[k].w)
                         : "r"(from + (j * Ring::kVecs + k) * 512)
                         : "memory");
        unpack_steps<IoT>(raw, v);
    };
    const bool dx_alike = row_phase(r0.dx) == row_phase(r0.x) && row_phase(r1.dx) == row_phase(r1.x);

#pragma unroll
    for (int k = 0; k < Ring::kStages - 1; ++k) request(tiles - 1 - k);
    for (int tile = tiles - 1; tile >= 0; --tile) {
        copy_async_wait<Ring::kStages - 3>();            // this tile and the one before it are here
        __syncwarp();
        const int b0 = r0.begin + tile * kWarpSteps, b1 = r1.begin + tile * kWarpSteps;
        const int t0 = b0 + lane * kLaneSteps, t1 = b1 + lane * kLaneSteps;
        const bool here = in_ring(tile);
        // all steps inside both rows, none with a final state to add
        const bool inner = here && b0 >= 0 && b1 >= 0 && b0 + kWarpSteps <= r0.hi && b1 + kWarpSteps <= r1.hi &&
                           (p.dfinal == nullptr || (b0 + kWarpSteps <= L - kW && b1 + kWarpSteps <= L - kW));
        const uint32_t from = mine + stage_of(tile);
        float2 xv[8], dp[8], before[H], after[H];
        {
            float v0[8], v1[8], g0[8], g1[8];
            if (here) {
                take(from, 0, v0);
                take(from, 1, v1);
                take(from, 2, g0);
                take(from, 3, g1);
            } else {
                load_steps(r0.x, t0, r0.lo, r0.hi, xspan, v0);
                load_steps(r1.x, t1, r1.lo, r1.hi, xspan, v1);
                load_steps(r0.dout, t0, r0.lo, r0.hi, dspan, g0);
                load_steps(r1.dout, t1, r1.lo, r1.hi, dspan, g1);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xv[i] = make_float2(v0[i], v1[i]);
                dp[i] = make_float2(g0[i], g1[i]);
            }
        }
        if (!inner) {
            // before the row's start: the initial state; behind its end: nothing
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (t0 + i < 0 || t0 + i >= r0.hi) xv[i].x = t0 + i < 0 ? r0.input(t0 + i, L) : 0.0f;
                if (t1 + i < 0 || t1 + i >= r1.hi) xv[i].y = t1 + i < 0 ? r1.input(t1 + i, L) : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < H; ++i) before[i] = after[i] = zero;
        if constexpr (kW > 1) {
            // the last steps of the tile before, for lane 0: lane 31's words of its stage
            float2 edge[H];
            if (inner && in_ring(tile - 1)) {
                const uint32_t last = smem_u32(ring) + 31 * 16 + stage_of(tile - 1);
                float e0[8], e1[8];
                take(last, 0, e0);
                take(last, 1, e1);
#pragma unroll
                for (int i = 0; i < kW - 1; ++i) edge[i] = make_float2(e0[8 - (kW - 1) + i], e1[8 - (kW - 1) + i]);
            } else {
#pragma unroll
                for (int i = 0; i < kW - 1; ++i) {
                    const int s0 = b0 - (kW - 1) + i, s1 = b1 - (kW - 1) + i;
                    edge[i] = make_float2(lane == 0 && s0 < r0.hi ? r0.input(s0, L) : 0.0f,
                                          lane == 0 && s1 < r1.hi ? r1.input(s1, L) : 0.0f);
                }
            }
#pragma unroll
            for (int i = 0; i < kW - 1; ++i) {
                const float2 up = shfl_up2(xv[8 - (kW - 1) + i], 1);
                before[i] = make_float2(lane == 0 ? edge[i].x : up.x, lane == 0 ? edge[i].y : up.y);
            }
        }
        __syncwarp();                                    // the slots read above are free again
        request(tile - (Ring::kStages - 1));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float2 pre = b;
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                const int j = i - (kW - 1) + k;
                pre = __ffma2_rn(w[k], j >= 0 ? xv[j] : before[kW - 1 + j], pre);
            }
            dp[i] = conv_dpre2(pre, dp[i], p.silu);
        }
        if (!inner) {                                    // outside: what was read there counts for nothing
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (t0 + i < r0.lo || t0 + i >= r0.hi) dp[i].x = 0.0f;
                if (t1 + i < r1.lo || t1 + i >= r1.hi) dp[i].y = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            db = __fadd2_rn(db, dp[i]);
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                const int j = i - (kW - 1) + k;
                dw[k] = __ffma2_rn(dp[i], j >= 0 ? xv[j] : before[kW - 1 + j], dw[k]);
            }
        }
        // dpre after this lane's steps: the lane above; for lane 31, what lane 0 had one tile later
        if constexpr (kW > 1) {
#pragma unroll
            for (int i = 0; i < kW - 1; ++i) {
                const float2 next = shfl2(dp[i], (lane + 1) & 31);
                after[i] = make_float2(lane == 31 ? later[i].x : next.x, lane == 31 ? later[i].y : next.y);
                later[i] = next;
            }
        }
        float2 o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i] = __fmul2_rn(w[kW - 1], dp[i]);
#pragma unroll
            for (int k = 0; k < kW - 1; ++k) {
                const int j = i + kW - 1 - k;
                o[i] = __ffma2_rn(w[k], j < 8 ? dp[j] : after[j - 8 < H ? j - 8 : 0], o[i]);
            }
        }
        if (inner && dx_alike) {
            float v0[8], v1[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v0[i] = o[i].x;
                v1[i] = o[i].y;
            }
            store_eight(r0.dx + t0, v0);
            store_eight(r1.dx + t1, v1);
        } else {
            if (p.dfinal != nullptr)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int f0 = t0 + i + kW - L, f1 = t1 + i + kW - L;
                    if (f0 >= 0 && f0 < kW && t0 + i >= 0) o[i].x += DType<IoT>::load(r0.dfinal + f0);
                    if (f1 >= 0 && f1 < kW && t1 + i >= 0) o[i].y += DType<IoT>::load(r1.dfinal + f1);
                }
            store_steps2(r0.dx, t0, r0.lo, r0.hi, r1.dx, t1, r1.lo, r1.hi, o);
        }
    }
    float s0[kW], s1[kW];
#pragma unroll
    for (int k = 0; k < kW; ++k) {
        s0[k] = dw[k].x;
        s1[k] = dw[k].y;
    }
    r0.finish(p, w0, b.x, stretch, lane, s0, db.x);
    r1.finish(p, w1, b.y, stretch, lane, s1, db.y);
}

}  // namespace mamba
