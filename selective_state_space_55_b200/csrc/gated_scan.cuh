// Gated linear recurrence, forward, backward and one token (sm_100a).
//
// Per chain (batch row b, channel d), with f_t = gate_t + bias_d:
//
//   sigmoid gate   a_t = 1 - g_t, u_t = g_t x_t, g_t = sigmoid(f_t)
//   log decay      a_t = exp(f_t), u_t = x_t
//   h_t = a_t h_{t-1} + u_t,   out_t = h_t
//
// and, backwards in time with l_t = dLoss/dh_t and r_t = a_t l_t,
//
//   l_t = dout_t + r_{t+1}   (l_{L-1} += dlast_state)
//   sigmoid gate   dx_t = g_t l_t,  dgate_t = l_t (x_t - h_{t-1}) g_t a_t
//   log decay      dx_t = l_t,      dgate_t = l_t a_t h_{t-1}
//   dbias = sum dgate,  dinitial_state = r_0.
//
// Steps outside a sequence (t >= seqlens[b]) count as a = 1, u = 0, dout = 0:
// they pass the state on, and out, dgate and dx are 0 there, whatever the
// padding holds.
//
// Both directions are scans of affine maps h -> A h + H, composed in any
// grouping.  Forward and backward are HBM-bound streams (3 and 5 tensors) as
// long as the step's arithmetic (two special-function operations for the
// sigmoid, one for the log decay) and the joins stay below the issue rate.
//
// Layout (batch, seqlen, dim): a warp takes a block of 64 steps of 64 channels
// (a lane two neighbours: rows of 128 or 256 bytes per access), up to 8 warps
// side by side in time make a segment of 512 steps.  Phase one walks the block
// and keeps only its map; the segment's maps are composed through shared
// memory; segments of a chain are joined by a look-back in fixed groups of 8,
// so that every state is composed in the same order whatever the timing.  Phase
// two walks the block again from its true start: its inputs come from L1 and
// L2 (a segment is 128 KB in bf16, some 70 MB over all resident CTAs), so HBM
// sees each input once.  The steps' arithmetic is done twice in exchange, in
// packed fp32x2.  Segments are handed out by a counter, the earliest steps of
// all chains first, so that every segment's predecessors belong to CTAs that
// are running or done; the wait is bounded all the same.
//
// Layout (batch, dim, seqlen): a lane takes 8 consecutive steps of one chain,
// the warp composes its lanes' maps by shuffles, and 1 to 8 warps per chain
// share a tile through shared memory.  Chains are plentiful here (one per
// channel instead of one per 64), so a chain stays with its warps and nothing
// waits.
#pragma once

#include "row_vectors.cuh"

namespace mamba {

constexpr int kGatedBlock = 64;                             // steps per warp
constexpr int kGatedWarps = 8;                              // blocks per segment, at most
constexpr int kGatedChannels = 64;                          // per CTA, two per lane
constexpr int kGatedThreads = kGatedWarps * 32;
constexpr int kGatedJoin = 8;                               // segments folded from one known state
static_assert(kGatedBlock == MAMBA_GATED_CHECKPOINT_STEPS, "checkpoints are the states entering blocks");

struct GatedStrides { int64_t batch, row; };

struct GatedParams {
    const void* gate;
    const void* x;
    const float* bias;            // (dim) or null
    const float* h0;              // (batch, dim) or null
    const int32_t* seqlens;       // (batch) or null
    void* out;                    // fwd (null: states only)
    float* last;                  // fwd, (batch, dim) or null
    const void* dout;             // bwd
    const float* dlast;           // bwd, (batch, dim) or null
    void* dgate;                  // bwd
    void* dx;                     // bwd
    float* dh0;                   // bwd, (batch, dim) or null
    float* bias_partial;          // bwd: [batch * segments][dim] (seqlen fastest: [batch][dim]) or null
    // (batch, seqlen, dim)
    float* enter;                 // [batch][blocks][dim], states entering blocks; fwd: written or null
    float4* maps;                 // [groups][segments][32]: a lane's two (A, H) pairs
    float2* states;               // [groups][segments / kGatedJoin][32]: states entering a join group
    unsigned int* flags;          // [groups][segments]: 0, 1 = map published, 2 = state published
    unsigned int* ticket;         // null: one segment per chain, one CTA per segment
    // (batch, dim, seqlen), bwd: states entering tiles, [chains][tiles]
    float* chain_states;
    GatedStrides gate_s, x_s, out_s, dgate_s, dx_s;          // out_s: out, or dout
    int64_t batch, dim, seqlen, chains;
    int64_t blocks;               // of 64 steps, per chain
    int64_t segments;             // per chain
    int64_t groups_per_row;       // 64-channel groups per batch row
    int64_t groups;
    int64_t items;                // groups * segments
    int64_t tiles;                // (batch, dim, seqlen): per chain
    int withhold;                 // test only: publish nothing
};

constexpr unsigned int kGatedPollLimit = 1u << 19;

// g and a of the sigmoid gate from f log2(e); a = 1 - g to fp32 on both sides.
// With e = exp(-|f|), small = e / (1 + e) is the smaller of the two and the
// other is 1 - small, rounded to nearest: a decay close to 1 is applied over
// about 1 / g steps, and a biased rounding would grow with that memory.
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void sigmoid_gate2(float2 f2, float2& g, float2& a) {
    const float2 one = make_float2(1.0f, 1.0f);
    const float2 e = make_float2(ex2_approx(-fabsf(f2.x)), ex2_approx(-fabsf(f2.y)));
    const float2 d = __fadd2_rn(e, one);
    const float2 small = __fmul2_rn(e, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
    const float2 big = __ffma2_rn(small, make_float2(-1.0f, -1.0f), one);
    g = make_float2(f2.x < 0.0f ? small.x : big.x, f2.y < 0.0f ? small.y : big.y);
    a = make_float2(f2.x < 0.0f ? big.x : small.x, f2.y < 0.0f ? big.y : small.y);
}

// Decay a and input gain g of two gates (gate values f, bias times log2(e)).
template <bool kLog>
__device__ __forceinline__ void gated_gains2(float2 f, float2 bias2, float2& g, float2& a) {
    const float2 f2 = __ffma2_rn(f, make_float2(kLog2e, kLog2e), bias2);
    if constexpr (kLog) {
        a = exp2_near_one_exact2(f2);
        g = make_float2(1.0f, 1.0f);
    } else {
        sigmoid_gate2(f2, g, a);
    }
}

// One gate.
template <bool kLog>
__device__ __forceinline__ void gated_gains(float f, float bias, float& g, float& a) {
    float2 g2, a2;
    gated_gains2<kLog>(make_float2(f, f), make_float2(bias * kLog2e, bias * kLog2e), g2, a2);
    g = g2.x;
    a = a2.x;
}

template <bool kLog>
__device__ __forceinline__ void gated_terms(float f, float bias, float x, float& a, float& u) {
    float g;
    gated_gains<kLog>(f, bias, g, a);
    u = kLog ? x : g * x;
}

// Decay and input term.
template <bool kLog>
__device__ __forceinline__ void gated_terms2(float2 f, float2 bias2, float2 x, float2& a, float2& u) {
    float2 g;
    gated_gains2<kLog>(f, bias2, g, a);
    u = kLog ? x : __fmul2_rn(g, x);
}

__device__ __forceinline__ int64_t gated_length(const GatedParams& p, int64_t b) {
    if (p.seqlens == nullptr) return p.seqlen;
    const int64_t n = p.seqlens[b];
    return n < 0 ? 0 : (n > p.seqlen ? p.seqlen : n);
}

__device__ __forceinline__ unsigned int load_acquire(const unsigned int* p) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void store_release(unsigned int* p, unsigned int v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// ------------------------------------------------ (batch, seqlen, dim) layout

// Two neighbouring channels of one step; raw bits so that a tile can be
// requested while the previous one is being worked on.  kVec: both lie in one
// aligned word; otherwise element by element (c1 says whether the second exists).
template <typename IoT> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    uint32_t v;
    __device__ __forceinline__ float2 get() const {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
};
template <> struct Pair<float> {
    float2 v;
    __device__ __forceinline__ float2 get() const { return v; }
};

template <typename IoT, bool kVec>
__device__ __forceinline__ Pair<IoT> load_pair(const IoT* p, bool c0, bool c1) {
    Pair<IoT> r;
    if constexpr (sizeof(IoT) == 2) {
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
        if constexpr (kVec) r.v = c0 ? *reinterpret_cast<const uint32_t*>(p) : 0u;
        else r.v = (c0 ? (uint32_t)q[0] : 0u) | ((c1 ? (uint32_t)q[1] : 0u) << 16);
    } else {
        if constexpr (kVec) r.v = c0 ? *reinterpret_cast<const float2*>(p) : make_float2(0.0f, 0.0f);
        else r.v = make_float2(c0 ? p[0] : 0.0f, c1 ? p[1] : 0.0f);
    }
    return r;
}

template <typename IoT, bool kVec>
__device__ __forceinline__ void store_pair(IoT* p, bool c0, bool c1, float2 v) {
    if constexpr (kVec) {
        if (!c0) return;
        if constexpr (sizeof(IoT) == 2) *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v.x, v.y);
        else *reinterpret_cast<float2*>(p) = v;
    } else {
        if (c0) DType<IoT>::store(p, v.x);
        if (c1) DType<IoT>::store(p + 1, v.y);
    }
}

// An fp32 pair of a (.., dim) array.
template <bool kVec>
__device__ __forceinline__ float2 load_f2(const float* p, bool c0, bool c1) {
    if constexpr (kVec) return c0 ? __ldcg(reinterpret_cast<const float2*>(p)) : make_float2(0.0f, 0.0f);
    else return make_float2(c0 ? __ldcg(p) : 0.0f, c1 ? __ldcg(p + 1) : 0.0f);
}

template <bool kVec>
__device__ __forceinline__ void store_f2(float* p, bool c0, bool c1, float2 v) {
    store_pair<float, kVec>(p, c0, c1, v);
}

// Where a warp's block lies: item = position * groups + group, positions in the
// order of the scan (kReverse: the last segment of a chain first).
struct GatedBlockAt {
    int64_t b, group, pos, segment, block, t, d;    // t: first step; d: this lane's first channel
    int left, rows;                                 // steps inside the sequence, inside the tensor
};

template <bool kReverse>
__device__ __forceinline__ GatedBlockAt gated_block(const GatedParams& p, int64_t item, int warp, int lane) {
    GatedBlockAt at;
    at.pos = item / p.groups;
    at.group = item - at.pos * p.groups;
    at.segment = kReverse ? p.segments - 1 - at.pos : at.pos;
    at.b = at.group / p.groups_per_row;
    at.d = (at.group - at.b * p.groups_per_row) * kGatedChannels + 2 * lane;
    at.block = at.segment * (blockDim.x >> 5) + warp;
    at.t = at.block * kGatedBlock;
    const int64_t n = gated_length(p, at.b) - at.t, rows = p.seqlen - at.t;
    at.left = (int)(n < 0 ? 0 : (n > kGatedBlock ? kGatedBlock : n));
    at.rows = (int)(rows < 0 ? 0 : (rows > kGatedBlock ? kGatedBlock : rows));
    return at;
}

// kN steps of two channels; steps from `left` on are not read and give 0.
template <typename IoT, bool kVec, int kN>
__device__ __forceinline__ void load_pairs(Pair<IoT> (&r)[kN], const IoT* p, int64_t stride, int left,
                                           bool c0, bool c1) {
    if (left >= kN) {
#pragma unroll
        for (int i = 0; i < kN; ++i) r[i] = load_pair<IoT, kVec>(p + i * stride, c0, c1);
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) r[i] = load_pair<IoT, kVec>(p + i * stride, i < left && c0, i < left && c1);
    }
}

// Publishing: every lane has written its part; lane 0 raises the flag.
__device__ __forceinline__ void gated_publish(const GatedParams& p, unsigned int* flag, int lane,
                                              unsigned int value) {
    __syncwarp();
    if (lane == 0 && !p.withhold) {
        __threadfence();
        store_release(flag, value);
    }
}

// The state entering segment `pos` of a chain (positions in scan order) for
// this lane's two channels; called by one warp with the segment's own map.
// Positions form groups of kGatedJoin.  The last of a group publishes the state
// that leaves it, the others their maps; a segment waits for the state entering
// its group and the maps of the group's earlier segments, and folds them in
// order.  `start` is the state entering position 0.
__device__ __forceinline__ float2 gated_join(const GatedParams& p, int64_t group, int64_t pos, int lane,
                                             float4 map, float2 start) {
    const int64_t join = pos / kGatedJoin, first = join * kGatedJoin;
    const int before = (int)(pos - first);
    unsigned int* flags = p.flags + group * p.segments;
    float4* maps = p.maps + (group * p.segments) * 32 + lane;
    const int64_t joins = (p.segments + kGatedJoin - 1) / kGatedJoin;
    float2* states = p.states + (group * joins) * 32 + lane;
    const bool closes = before == kGatedJoin - 1;
    if (!closes && pos + 1 < p.segments) {
        __stcg(maps + pos * 32, map);
        gated_publish(p, flags + pos, lane, 1u);
    }
    // lane l < before waits for the map of segment first + l, lane kGatedJoin for the state
    const bool wait_map = lane < before, wait_state = lane == kGatedJoin && join > 0;
    const unsigned int* mine = flags + (wait_map ? first + lane : first - 1);
    bool ready = !(wait_map || wait_state);
    unsigned int poll = 0;
    for (; poll < kGatedPollLimit; ++poll) {
        if (!ready) ready = load_acquire(mine) >= (wait_state ? 2u : 1u);
        if (__all_sync(0xffffffffu, ready)) break;
    }
    float2 h = start;
    if (poll == kGatedPollLimit) {
        if (lane == 0) record_device_error(MAMBA_ERR_TIMEOUT);
    } else {
        float4 m[kGatedJoin - 1];
#pragma unroll
        for (int i = 0; i < kGatedJoin - 1; ++i)
            m[i] = i < before ? __ldcg(maps + (first + i) * 32) : make_float4(1.0f, 0.0f, 1.0f, 0.0f);
        if (join > 0) h = __ldcg(states + join * 32);
#pragma unroll
        for (int i = 0; i < kGatedJoin - 1; ++i)
            if (i < before) {
                h.x = fmaf(m[i].x, h.x, m[i].y);
                h.y = fmaf(m[i].z, h.y, m[i].w);
            }
    }
    if (closes && pos + 1 < p.segments) {
        __stcg(states + (join + 1) * 32, make_float2(fmaf(map.x, h.x, map.y), fmaf(map.z, h.y, map.w)));
        gated_publish(p, flags + pos, lane, 2u);
    }
    return h;
}

// The next item of a CTA.  `slot` is written before a barrier and read after it.
__device__ __forceinline__ int64_t gated_first_item(const GatedParams& p, int64_t* slot) {
    if (p.ticket == nullptr) return blockIdx.x;
    if (threadIdx.x == 0) *slot = atomicAdd(p.ticket, 1u);
    __syncthreads();
    return *slot;
}

constexpr int kGatedSub = 8;                 // steps requested at a time

template <typename IoT, bool kLog, bool kVec>
__global__ void __launch_bounds__(kGatedThreads)
    gated_scan_fwd_kernel(const __grid_constant__ GatedParams p) {
    __shared__ float4 maps[kGatedWarps][32];
    __shared__ float2 entering[32];
    __shared__ int64_t first_slot, next_slot;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const float2 zero = make_float2(0.0f, 0.0f), one = make_float2(1.0f, 1.0f);
    int64_t item = gated_first_item(p, &first_slot);
    while (item < p.items) {
        const GatedBlockAt at = gated_block<false>(p, item, warp, lane);
        const bool c0 = at.d < p.dim, c1 = at.d + 1 < p.dim;
        float2 bias2 = p.bias != nullptr ? load_f2<kVec>(p.bias + at.d, c0, c1) : zero;
        bias2 = __fmul2_rn(bias2, make_float2(kLog2e, kLog2e));
        const IoT* gate = static_cast<const IoT*>(p.gate) + at.b * p.gate_s.batch + at.t * p.gate_s.row + at.d;
        const IoT* x = static_cast<const IoT*>(p.x) + at.b * p.x_s.batch + at.t * p.x_s.row + at.d;
        float2 h = p.h0 != nullptr ? load_f2<kVec>(p.h0 + at.b * p.dim + at.d, c0, c1) : zero;
        int64_t following = p.items;
        if (p.blocks > 1) {
            if (threadIdx.x == 0 && p.ticket != nullptr) next_slot = atomicAdd(p.ticket, 1u);
            float2 A = one, H = zero;
            for (int s = 0; s < at.left; s += kGatedSub) {
                Pair<IoT> rf[kGatedSub], rx[kGatedSub];
                load_pairs<IoT, kVec>(rf, gate + s * p.gate_s.row, p.gate_s.row, at.left - s, c0, c1);
                load_pairs<IoT, kVec>(rx, x + s * p.x_s.row, p.x_s.row, at.left - s, c0, c1);
                float2 a[kGatedSub], u[kGatedSub];
#pragma unroll
                for (int i = 0; i < kGatedSub; ++i)
                    gated_terms2<kLog>(rf[i].get(), bias2, rx[i].get(), a[i], u[i]);
                if (at.left - s < kGatedSub)
#pragma unroll
                    for (int i = 0; i < kGatedSub; ++i)
                        if (s + i >= at.left) a[i] = one;       // u is 0: x was not read
#pragma unroll
                for (int i = 0; i < kGatedSub; ++i) {
                    H = __ffma2_rn(a[i], H, u[i]);
                    A = __fmul2_rn(A, a[i]);
                }
            }
            maps[warp][lane] = make_float4(A.x, H.x, A.y, H.y);
            __syncthreads();
            if (p.ticket != nullptr) {
                following = next_slot;
                if (warp == 0) {
                    float2 At = one, Ht = zero;
                    for (int v = 0; v < warps; ++v) {
                        const float4 m = maps[v][lane];
                        Ht = __ffma2_rn(make_float2(m.x, m.z), Ht, make_float2(m.y, m.w));
                        At = __fmul2_rn(At, make_float2(m.x, m.z));
                    }
                    entering[lane] = gated_join(p, at.group, at.pos, lane, make_float4(At.x, Ht.x, At.y, Ht.y), h);
                }
            }
            float2 Ap = one, Hp = zero;
            for (int v = 0; v < warp; ++v) {
                const float4 m = maps[v][lane];
                Hp = __ffma2_rn(make_float2(m.x, m.z), Hp, make_float2(m.y, m.w));
                Ap = __fmul2_rn(Ap, make_float2(m.x, m.z));
            }
            if (p.ticket != nullptr) {
                __syncthreads();
                h = entering[lane];
            }
            h = __ffma2_rn(Ap, h, Hp);
        }
        if (at.rows > 0 && p.enter != nullptr)
            store_f2<kVec>(p.enter + (at.b * p.blocks + at.block) * p.dim + at.d, c0, c1, h);
        if (p.out != nullptr) {
            IoT* out = static_cast<IoT*>(p.out) + at.b * p.out_s.batch + at.t * p.out_s.row + at.d;
            int s = 0;
            for (; s < at.left; s += kGatedSub) {
                Pair<IoT> rf[kGatedSub], rx[kGatedSub];
                load_pairs<IoT, kVec>(rf, gate + s * p.gate_s.row, p.gate_s.row, at.left - s, c0, c1);
                load_pairs<IoT, kVec>(rx, x + s * p.x_s.row, p.x_s.row, at.left - s, c0, c1);
                float2 a[kGatedSub], u[kGatedSub];
#pragma unroll
                for (int i = 0; i < kGatedSub; ++i)
                    gated_terms2<kLog>(rf[i].get(), bias2, rx[i].get(), a[i], u[i]);
                IoT* o = out + s * p.out_s.row;
                if (at.left - s >= kGatedSub) {
#pragma unroll
                    for (int i = 0; i < kGatedSub; ++i) {
                        h = __ffma2_rn(a[i], h, u[i]);
                        store_pair<IoT, kVec>(o + i * p.out_s.row, c0, c1, h);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kGatedSub; ++i) {
                        const bool in = s + i < at.left;
                        if (in) h = __ffma2_rn(a[i], h, u[i]);
                        if (s + i < at.rows) store_pair<IoT, kVec>(o + i * p.out_s.row, c0, c1, in ? h : zero);
                    }
                }
            }
            for (; s < at.rows; ++s) store_pair<IoT, kVec>(out + s * p.out_s.row, c0, c1, zero);
            if (p.last != nullptr && at.block == p.blocks - 1)
                store_f2<kVec>(p.last + at.b * p.dim + at.d, c0, c1, h);
        }
        item = following;
    }
}

// Backward.  Phase one walks a block forward from its checkpoint, keeps the
// state every kGatedBack steps in shared memory and accumulates the block's map
// of r, R = sum_t (prod_{s <= t} a_s) dout_t; phase two walks it backward.
constexpr int kGatedBack = 4;

template <typename IoT, bool kLog, bool kVec>
__global__ void __launch_bounds__(kGatedThreads, 2)
    gated_scan_bwd_kernel(const __grid_constant__ GatedParams p) {
    __shared__ float4 maps[kGatedWarps][32];
    __shared__ float2 entering[32];
    __shared__ float2 bias_sums[kGatedWarps][32];
    __shared__ float2 kept[kGatedWarps][kGatedBlock / kGatedBack][32];
    __shared__ int64_t first_slot, next_slot;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const float2 zero = make_float2(0.0f, 0.0f), one = make_float2(1.0f, 1.0f);
    int64_t item = gated_first_item(p, &first_slot);
    while (item < p.items) {
        const GatedBlockAt at = gated_block<true>(p, item, warp, lane);
        const bool c0 = at.d < p.dim, c1 = at.d + 1 < p.dim;
        float2 bias2 = p.bias != nullptr ? load_f2<kVec>(p.bias + at.d, c0, c1) : zero;
        bias2 = __fmul2_rn(bias2, make_float2(kLog2e, kLog2e));
        const IoT* gate = static_cast<const IoT*>(p.gate) + at.b * p.gate_s.batch + at.t * p.gate_s.row + at.d;
        const IoT* x = static_cast<const IoT*>(p.x) + at.b * p.x_s.batch + at.t * p.x_s.row + at.d;
        const IoT* dout = static_cast<const IoT*>(p.dout) + at.b * p.out_s.batch + at.t * p.out_s.row + at.d;
        int64_t following = p.items;
        if (threadIdx.x == 0 && p.ticket != nullptr) next_slot = atomicAdd(p.ticket, 1u);
        float2 h = at.rows > 0 ? load_f2<kVec>(p.enter + (at.b * p.blocks + at.block) * p.dim + at.d, c0, c1) : zero;
        float2 P = one, R = zero;
        for (int s = 0; s < at.left; s += kGatedSub) {
            Pair<IoT> rf[kGatedSub], rx[kGatedSub], rd[kGatedSub];
            load_pairs<IoT, kVec>(rf, gate + s * p.gate_s.row, p.gate_s.row, at.left - s, c0, c1);
            load_pairs<IoT, kVec>(rx, x + s * p.x_s.row, p.x_s.row, at.left - s, c0, c1);
            load_pairs<IoT, kVec>(rd, dout + s * p.out_s.row, p.out_s.row, at.left - s, c0, c1);
#pragma unroll
            for (int i = 0; i < kGatedSub; ++i) {
                if (i % kGatedBack == 0) kept[warp][(s + i) / kGatedBack][lane] = h;
                float2 a, u;
                gated_terms2<kLog>(rf[i].get(), bias2, rx[i].get(), a, u);
                if (s + i >= at.left) a = one;
                h = __ffma2_rn(a, h, u);
                P = __fmul2_rn(P, a);
                R = __ffma2_rn(P, rd[i].get(), R);
            }
        }
        maps[warp][lane] = make_float4(P.x, R.x, P.y, R.y);
        __syncthreads();
        float2 r = p.dlast != nullptr ? load_f2<kVec>(p.dlast + at.b * p.dim + at.d, c0, c1) : zero;
        if (p.ticket != nullptr) {
            following = next_slot;
            if (warp == 0) {
                float2 At = one, Rt = zero;
                for (int v = warps - 1; v >= 0; --v) {
                    const float4 m = maps[v][lane];
                    Rt = __ffma2_rn(make_float2(m.x, m.z), Rt, make_float2(m.y, m.w));
                    At = __fmul2_rn(At, make_float2(m.x, m.z));
                }
                entering[lane] = gated_join(p, at.group, at.pos, lane, make_float4(At.x, Rt.x, At.y, Rt.y), r);
            }
        }
        float2 Ap = one, Rp = zero;
        for (int v = warps - 1; v > warp; --v) {
            const float4 m = maps[v][lane];
            Rp = __ffma2_rn(make_float2(m.x, m.z), Rp, make_float2(m.y, m.w));
            Ap = __fmul2_rn(Ap, make_float2(m.x, m.z));
        }
        if (p.ticket != nullptr) {
            __syncthreads();
            r = entering[lane];
        }
        r = __ffma2_rn(Ap, r, Rp);

        float2 db = zero;
        IoT* dgate = static_cast<IoT*>(p.dgate) + at.b * p.dgate_s.batch + at.t * p.dgate_s.row + at.d;
        IoT* dx = static_cast<IoT*>(p.dx) + at.b * p.dx_s.batch + at.t * p.dx_s.row + at.d;
        for (int s = at.left; s < at.rows; ++s) {
            store_pair<IoT, kVec>(dgate + s * p.dgate_s.row, c0, c1, zero);
            store_pair<IoT, kVec>(dx + s * p.dx_s.row, c0, c1, zero);
        }
        for (int s = (at.left - 1) & ~(kGatedBack - 1); s >= 0; s -= kGatedBack) {
            const int left = at.left - s;
            Pair<IoT> rf[kGatedBack], rx[kGatedBack], rd[kGatedBack];
            load_pairs<IoT, kVec>(rf, gate + s * p.gate_s.row, p.gate_s.row, left, c0, c1);
            load_pairs<IoT, kVec>(rx, x + s * p.x_s.row, p.x_s.row, left, c0, c1);
            load_pairs<IoT, kVec>(rd, dout + s * p.out_s.row, p.out_s.row, left, c0, c1);
            float2 a[kGatedBack], g[kGatedBack], before[kGatedBack];
            h = kept[warp][s / kGatedBack][lane];
#pragma unroll
            for (int i = 0; i < kGatedBack; ++i) {
                gated_gains2<kLog>(rf[i].get(), bias2, g[i], a[i]);
                before[i] = h;
                h = __ffma2_rn(a[i], h, kLog ? rx[i].get() : __fmul2_rn(g[i], rx[i].get()));
            }
#pragma unroll
            for (int i = kGatedBack - 1; i >= 0; --i)
                if (i < left) {
                    const float2 l = __fadd2_rn(rd[i].get(), r);
                    r = __fmul2_rn(a[i], l);
                    float2 df, dv;
                    if constexpr (kLog) {
                        dv = l;
                        df = __fmul2_rn(r, before[i]);
                    } else {
                        const float2 diff = __ffma2_rn(before[i], make_float2(-1.0f, -1.0f), rx[i].get());
                        dv = __fmul2_rn(g[i], l);
                        df = __fmul2_rn(__fmul2_rn(g[i], r), diff);
                    }
                    db = __fadd2_rn(db, df);
                    store_pair<IoT, kVec>(dgate + (s + i) * p.dgate_s.row, c0, c1, df);
                    store_pair<IoT, kVec>(dx + (s + i) * p.dx_s.row, c0, c1, dv);
                }
        }
        if (p.dh0 != nullptr && at.block == 0) store_f2<kVec>(p.dh0 + at.b * p.dim + at.d, c0, c1, r);
        if (p.bias_partial != nullptr) {
            bias_sums[warp][lane] = db;
            __syncthreads();
            if (warp == 0) {
                float2 sum = zero;
                for (int v = 0; v < warps; ++v) sum = __fadd2_rn(sum, bias_sums[v][lane]);
                store_f2<kVec>(p.bias_partial + (at.b * p.segments + at.segment) * p.dim + at.d, c0, c1, sum);
            }
        }
        item = following;
    }
}

// ------------------------------------------------ (batch, dim, seqlen) layout

// Inclusive compositions over the first lanes of a team of `width` lanes
// (kReverse: from the team's last lane down): on return (A, H) is the map of
// every lane before this one in scan order, (At, Ht) of the whole team.
template <bool kReverse>
__device__ __forceinline__ void team_scan(float& A, float& H, float& At, float& Ht, int lane, int width) {
    const int rank = lane & (width - 1);
    const int first = kReverse ? width - 1 : 0;
    for (int o = 1; o < width; o <<= 1) {
        const float Ao = kReverse ? __shfl_down_sync(0xffffffffu, A, o, width) : __shfl_up_sync(0xffffffffu, A, o, width);
        const float Ho = kReverse ? __shfl_down_sync(0xffffffffu, H, o, width) : __shfl_up_sync(0xffffffffu, H, o, width);
        if (kReverse ? rank + o < width : rank >= o) {
            H = fmaf(A, Ho, H);
            A *= Ao;
        }
    }
    At = __shfl_sync(0xffffffffu, A, width - 1 - first, width);
    Ht = __shfl_sync(0xffffffffu, H, width - 1 - first, width);
    const float Ae = kReverse ? __shfl_down_sync(0xffffffffu, A, 1, width) : __shfl_up_sync(0xffffffffu, A, 1, width);
    const float He = kReverse ? __shfl_down_sync(0xffffffffu, H, 1, width) : __shfl_up_sync(0xffffffffu, H, 1, width);
    A = rank == first ? 1.0f : Ae;
    H = rank == first ? 0.0f : He;
}

// Composes the maps of the kWarps warps that share a chain: (A, H) gains the
// maps of the warps before this one in scan order, (At, Ht) becomes the map of
// the whole tile.  `buf` is [kGatedWarps] shared pairs; two of them used in turn.
template <int kWarps, bool kReverse>
__device__ __forceinline__ void join_warps(float& A, float& H, float& At, float& Ht, float2* buf,
                                           int warp, int lane) {
    if constexpr (kWarps > 1) {
        if (lane == 0) buf[warp] = make_float2(At, Ht);
        __syncthreads();
        const int base = warp / kWarps * kWarps, rank = warp - base;
        float2 mine = make_float2(1.0f, 0.0f), all = make_float2(1.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const int v = kReverse ? kWarps - 1 - k : k;
            if (v == rank) mine = all;
            const float2 m = buf[base + v];
            all.y = fmaf(m.x, all.y, m.y);
            all.x *= m.x;
        }
        H = fmaf(A, mine.y, H);
        A *= mine.x;
        At = all.x;
        Ht = all.y;
    }
}

// A lane's place: kWarps warps per chain; with one, `width` lanes per chain.
template <int kWarps>
struct GatedChainAt {
    int64_t chain, b, d, n, step;     // step: time steps per tile
    int64_t offset;                   // first step of this lane in tile 0, before the phase
    bool live;
    __device__ __forceinline__ GatedChainAt(const GatedParams& p, int warp, int lane, int width) {
        if (kWarps > 1) {
            chain = (int64_t)blockIdx.x * (kGatedWarps / kWarps) + warp / kWarps;
            offset = (warp % kWarps) * kWarpSteps + lane * kLaneSteps;
            step = kWarps * kWarpSteps;
        } else {
            const int64_t teams = 32 / width;
            chain = ((int64_t)blockIdx.x * kGatedWarps + warp) * teams + lane / width;
            offset = (lane & (width - 1)) * kLaneSteps;
            step = (int64_t)width * kLaneSteps;
        }
        live = chain < p.chains;
        if (!live) chain = p.chains - 1;
        b = chain / p.dim;
        d = chain - b * p.dim;
        n = live ? gated_length(p, b) : 0;
    }
};

template <typename IoT, bool kLog, int kWarps>
__global__ void __launch_bounds__(kGatedThreads)
    gated_scan_rows_fwd_kernel(const __grid_constant__ GatedParams p, int width) {
    __shared__ float2 buf[2][kGatedWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const GatedChainAt<kWarps> at(p, warp, lane, width);
    const IoT* gate = static_cast<const IoT*>(p.gate) + at.b * p.gate_s.batch + at.d * p.gate_s.row;
    const IoT* x = static_cast<const IoT*>(p.x) + at.b * p.x_s.batch + at.d * p.x_s.row;
    IoT* out = static_cast<IoT*>(p.out) + at.b * p.out_s.batch + at.d * p.out_s.row;
    const int64_t hi = at.live ? p.seqlen : 0;
    const float bias = p.bias != nullptr ? p.bias[at.d] : 0.0f;
    float carry = p.h0 != nullptr ? p.h0[at.chain] : 0.0f;
    const int64_t shift = at.offset - row_phase(gate);
    for (int64_t tile = 0; tile < p.tiles; ++tile) {
        const int64_t t0 = tile * at.step + shift;
        float a[8], u[8], x8[8];
        load_steps(gate, t0, 0, at.n, 0.0f, a);
        load_steps(x, t0, 0, at.n, 0.0f, x8);
        float A = 1.0f, H = 0.0f, At, Ht;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            gated_terms<kLog>(a[i], bias, x8[i], a[i], u[i]);
            if (t0 + i < 0 || t0 + i >= at.n) {
                a[i] = 1.0f;
                u[i] = 0.0f;
            }
            H = fmaf(a[i], H, u[i]);
            A *= a[i];
        }
        team_scan<false>(A, H, At, Ht, lane, width);
        join_warps<kWarps, false>(A, H, At, Ht, buf[tile & 1], warp, lane);
        float h = fmaf(A, carry, H);
        carry = fmaf(At, carry, Ht);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h = fmaf(a[i], h, u[i]);
            u[i] = t0 + i < at.n ? h : 0.0f;
        }
        store_steps(out, t0, 0, hi, u);
    }
    if (p.last != nullptr && at.live && at.offset == 0) p.last[at.chain] = carry;
}

// Backward: with more than one tile per chain, a first sweep keeps the states
// entering the tiles; the second runs from the last tile to the first and reads
// gate and x again (from L2 while the chains in flight fit there).
template <typename IoT, bool kLog, int kWarps>
__global__ void __launch_bounds__(kGatedThreads)
    gated_scan_rows_bwd_kernel(const __grid_constant__ GatedParams p, int width) {
    __shared__ float2 buf[2][kGatedWarps];
    __shared__ float2 back[2][kGatedWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const GatedChainAt<kWarps> at(p, warp, lane, width);
    const IoT* gate = static_cast<const IoT*>(p.gate) + at.b * p.gate_s.batch + at.d * p.gate_s.row;
    const IoT* x = static_cast<const IoT*>(p.x) + at.b * p.x_s.batch + at.d * p.x_s.row;
    const IoT* dout = static_cast<const IoT*>(p.dout) + at.b * p.out_s.batch + at.d * p.out_s.row;
    IoT* dgate = static_cast<IoT*>(p.dgate) + at.b * p.dgate_s.batch + at.d * p.dgate_s.row;
    IoT* dx = static_cast<IoT*>(p.dx) + at.b * p.dx_s.batch + at.d * p.dx_s.row;
    const int64_t hi = at.live ? p.seqlen : 0;
    const float bias = p.bias != nullptr ? p.bias[at.d] : 0.0f;
    const int64_t shift = at.offset - row_phase(gate);
    float* states = p.chain_states + at.chain * p.tiles;
    float carry = p.h0 != nullptr ? p.h0[at.chain] : 0.0f;
    for (int64_t tile = 0; tile + 1 < p.tiles; ++tile) {
        const int64_t t0 = tile * at.step + shift;
        float f[8], x8[8];
        load_steps(gate, t0, 0, at.n, 0.0f, f);
        load_steps(x, t0, 0, at.n, 0.0f, x8);
        float A = 1.0f, H = 0.0f, At, Ht;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float a, u;
            gated_terms<kLog>(f[i], bias, x8[i], a, u);
            if (t0 + i < 0 || t0 + i >= at.n) {
                a = 1.0f;
                u = 0.0f;
            }
            H = fmaf(a, H, u);
            A *= a;
        }
        team_scan<false>(A, H, At, Ht, lane, width);
        join_warps<kWarps, false>(A, H, At, Ht, buf[tile & 1], warp, lane);
        if (at.live && at.offset == 0) states[tile] = carry;
        carry = fmaf(At, carry, Ht);
    }
    if (kWarps > 1) __syncthreads();
    else __syncwarp();
    float r_carry = p.dlast != nullptr ? p.dlast[at.chain] : 0.0f;
    float db = 0.0f;
    for (int64_t tile = p.tiles - 1; tile >= 0; --tile) {
        const int64_t t0 = tile * at.step + shift;
        float a[8], g[8], x8[8], d8[8], before[8];
        load_steps(gate, t0, 0, at.n, 0.0f, a);
        load_steps(x, t0, 0, at.n, 0.0f, x8);
        load_steps(dout, t0, 0, at.n, 0.0f, d8);
        if (tile + 1 < p.tiles) carry = states[tile];
        float A = 1.0f, H = 0.0f, At, Ht;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            gated_gains<kLog>(a[i], bias, g[i], a[i]);
            if (t0 + i < 0 || t0 + i >= at.n) {
                a[i] = 1.0f;
                g[i] = 0.0f;
            }
            H = fmaf(a[i], H, g[i] * x8[i]);
            A *= a[i];
        }
        float B = A, R = 0.0f, Bt, Rt;
#pragma unroll
        for (int i = 7; i >= 0; --i) R = a[i] * (d8[i] + R);
        team_scan<false>(A, H, At, Ht, lane, width);
        team_scan<true>(B, R, Bt, Rt, lane, width);
        // the reverse join's barrier covers the forward one's buffer as well
        join_warps<kWarps, false>(A, H, At, Ht, buf[tile & 1], warp, lane);
        join_warps<kWarps, true>(B, R, Bt, Rt, back[tile & 1], warp, lane);
        float h = fmaf(A, carry, H);
        float r = fmaf(B, r_carry, R);
        r_carry = fmaf(Bt, r_carry, Rt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            before[i] = h;
            h = fmaf(a[i], h, g[i] * x8[i]);
        }
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            const float l = d8[i] + r;
            r = a[i] * l;
            const bool in = t0 + i >= 0 && t0 + i < at.n;
            const float df = kLog ? r * before[i] : g[i] * r * (x8[i] - before[i]);
            const float dv = kLog ? l : g[i] * l;
            d8[i] = in ? df : 0.0f;
            x8[i] = in ? dv : 0.0f;
            db += d8[i];
        }
        store_steps(dgate, t0, 0, hi, d8);
        store_steps(dx, t0, 0, hi, x8);
    }
    if (p.dh0 != nullptr && at.live && at.offset == 0) p.dh0[at.chain] = r_carry;
    if (p.bias_partial != nullptr) {
        for (int o = width / 2; o > 0; o >>= 1) db += __shfl_xor_sync(0xffffffffu, db, o, width);
        if constexpr (kWarps > 1) {
            __syncthreads();
            if (lane == 0) buf[0][warp].x = db;
            __syncthreads();
            db = 0.0f;
            const int base = warp / kWarps * kWarps;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) db += buf[0][base + v].x;
        }
        if (at.live && at.offset == 0) p.bias_partial[at.chain] = db;
    }
}

// ------------------------------------------------------------------ one token

struct GatedUpdateParams {
    float* state;                 // (batch, dim), in place
    const void* gate;
    const void* x;
    const float* bias;            // (dim) or null
    void* out;
    int64_t gate_stride, x_stride, out_stride;     // between batch rows
    int64_t batch, dim;
    int64_t per_row;              // threads per row
};

constexpr int kGatedUpdateThreads = 128;

// kN channels per thread (8: vectors; 1: any alignment and size).  One read
// and one write of the fp32 state beside gate, x and out: HBM-bound for large
// batches, launch latency below.
template <typename IoT, bool kLog, int kN>
__global__ void __launch_bounds__(kGatedUpdateThreads)
    gated_update_kernel(const __grid_constant__ GatedUpdateParams p) {
    const int64_t i = (int64_t)blockIdx.x * kGatedUpdateThreads + threadIdx.x;
    const int64_t b = i / p.per_row;
    if (b >= p.batch) return;
    const int64_t d = (i - b * p.per_row) * kN;
    float* state = p.state + b * p.dim + d;
    const IoT* gate = static_cast<const IoT*>(p.gate) + b * p.gate_stride + d;
    const IoT* x = static_cast<const IoT*>(p.x) + b * p.x_stride + d;
    IoT* out = static_cast<IoT*>(p.out) + b * p.out_stride + d;
    if constexpr (kN == 8) {
        float h[8], f[8], v[8], bias[8];
        load_steps(state, 0, 0, 8, 0.0f, h);
        load_steps(gate, 0, 0, 8, 0.0f, f);
        load_steps(x, 0, 0, 8, 0.0f, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) bias[k] = 0.0f;
        if (p.bias != nullptr) load_steps(p.bias + d, 0, 0, 8, 0.0f, bias);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float a, u;
            gated_terms<kLog>(f[k], bias[k], v[k], a, u);
            h[k] = fmaf(a, h[k], u);
        }
        store_steps(state, 0, 0, 8, h);
        store_steps(out, 0, 0, 8, h);
    } else {
        float a, u;
        gated_terms<kLog>(DType<IoT>::load(gate), p.bias != nullptr ? p.bias[d] : 0.0f,
                          DType<IoT>::load(x), a, u);
        const float h = fmaf(a, *state, u);
        *state = h;
        DType<IoT>::store(out, h);
    }
}

}  // namespace mamba
