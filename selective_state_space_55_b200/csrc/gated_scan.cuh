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
// Layout (batch, seqlen, dim), what TMA cannot move (odd strides or bases) and the
// backward of few chains: a warp takes a block of 64 steps of 128 channels (a lane
// four neighbours: rows of 256 or 512 bytes per access), up to 8 warps side by side
// in time make a segment of 512 steps.  Phase one walks the block and keeps only its
// map; the segment's maps are composed through shared memory; segments of a chain
// are joined by a look-back in fixed groups of 24, so that every state is composed
// in the same order whatever the timing.  Phase two walks the block again from its
// true start: its inputs come from L2 (a segment is 256 KB in bf16), so HBM sees
// each input once.  The steps' arithmetic is done twice in exchange, in packed
// fp32x2.  Segments are handed out by a counter, the earliest steps of all chains
// first, so that every segment's predecessors belong to CTAs that are running or
// done; the wait is bounded all the same.  What TMA can move has kernels of its own
// (gated_chain.cuh).  Measured, bf16: 1 x 131072 x 1536 backward 555 us, 56 % of the
// copy rate (without checkpoints 792); 8 x 2047 x 4095 forward 500 us, 12 %, backward
// 1217 us, 9 %, where rows start anywhere: every element is a load of its own, twice,
// and a store of its own.
//
// Layout (batch, dim, seqlen): a lane takes 8 consecutive steps of two neighbouring
// chains, the warp composes its lanes' maps by shuffles, and 1 to 8 warps share a
// tile of a pair through shared memory.  Chains are plentiful here (one per channel
// instead of one per 64), so a chain stays with its warps and nothing waits; the
// warps walk pair after pair, the next tile on its way by cp.async.  Bound by issue (75
// and 65 % of the slots on 8 x 4096 x 1024: the scan across lanes and the addresses of
// every tile, beside the steps' arithmetic): 8 x 4096 x 2048 bf16 forward 98 us, 63 % of
// the copy rate, backward 229 us, 45 %.  A backward row that needs a second tile pays a
// sweep for it: 2047 steps, whose rows start up to 7 past a boundary, take 381 us.
#pragma once

#include "row_vectors.cuh"

namespace mamba {

constexpr int kGatedBlock = 64;                             // steps per warp
constexpr int kGatedWarps = 8;                              // blocks per segment, at most
constexpr int kGatedChannels = 128;                         // per CTA, four per lane
constexpr int kGatedThreads = kGatedWarps * 32;
constexpr int kRowWarps = 8;                                // per pair of chains in (batch, dim, seqlen), at most
constexpr int kRowThreads = kRowWarps * 32;
constexpr int kGatedJoin = 24;                              // segments folded from one known state
static_assert(kGatedJoin < 32, "one lane per map and one for the state");
static_assert(kGatedBlock == MAMBA_GATED_CHECKPOINT_STEPS, "checkpoints are the states entering blocks");

struct GatedStrides { int64_t batch, row; };

// What the segments of the chains hand on: `segments` per group of channels.
struct GatedLinks {
    float4* maps;                 // [groups][segments][pairs][32]: a lane's maps
    float2* states;               // [groups][segments / kGatedJoin][pairs][32]: states entering a join group
    unsigned int* flags;          // [groups][segments]: 0, 1 = map published, 2 = state published
    unsigned int* failed;         // 0, or 1 once a wait of this call has run out
    int64_t segments;
    int withhold;                 // test only: publish nothing
};

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
    GatedLinks links;
    unsigned int* ticket;         // null: one segment per chain, one CTA per segment
    // (batch, dim, seqlen), bwd: states entering tiles, [chains][tiles]
    float* chain_states;
    GatedStrides gate_s, x_s, out_s, dgate_s, dx_s;          // out_s: out, or dout
    int64_t batch, dim, seqlen, chains;
    int64_t blocks;               // of 64 steps, per chain
    int64_t segments;             // per chain
    int64_t groups_per_row;       // 128-channel groups per batch row
    int64_t groups;
    int64_t items;                // groups * segments
    int64_t tiles;                // (batch, dim, seqlen): per chain
};

// A wait that runs out (some 0.3 s) is recorded, and marked for the call: every
// other wait of the call looks at the mark now and then, and the CTAs leave instead
// of waiting as long for each item that is left.
constexpr unsigned int kGatedPollLimit = 1u << 19;
constexpr unsigned int kGatedPollsPerLook = 64;

// g and a of the sigmoid gate from f log2(e).  With e = exp(-f): g = 1 / (1 + e),
// and a = e g for f >= 0, 1 - g (rounded to nearest) for f < 0: there a is close
// to 1, it is applied over about 1 / g steps, and a biased rounding would grow
// with that memory.  e = inf gives g = 0, a = 1.
__device__ __forceinline__ void sigmoid_gate2(float2 f2, float2& g, float2& a) {
    const float2 one = make_float2(1.0f, 1.0f);
    const float2 e = make_float2(ex2_approx(-f2.x), ex2_approx(-f2.y));
    const float2 d = __fadd2_rn(e, one);
    g = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    const float2 small = __fmul2_rn(e, g);
    const float2 big = __ffma2_rn(g, make_float2(-1.0f, -1.0f), one);
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

// Loads from L2 of what other CTAs hand on, and of the start states (whose buffer
// the last states may share).  They stay on their side of the waits, barriers and
// publications around them: the cached-load intrinsics do not promise that.
__device__ __forceinline__ float load_ordered(const float* p) {
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ float2 load_ordered(const float2* p) {
    float2 v;
    asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ float4 load_ordered(const float4* p) {
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Time to look whether another wait of this call has run out?
__device__ __forceinline__ bool gated_look(unsigned int poll) {
    return poll % kGatedPollsPerLook == kGatedPollsPerLook - 1;
}

__device__ __forceinline__ void gated_give_up(unsigned int* failed) {
    record_device_error(MAMBA_ERR_TIMEOUT);
    store_release(failed, 1u);
}

// ------------------------------------------------ (batch, seqlen, dim) layout

constexpr int kGatedPairs = kGatedChannels / 64;            // pairs of channels per lane

// A lane's channels of one step, as fp32 pairs.  kVec: four neighbours in one
// aligned word; otherwise channels lane, lane + 32, ... so that single elements
// still coalesce.
struct Channels {
    int64_t d;                    // this lane's first channel
    int live;                     // how many of its channels exist
};

template <bool kVec>
__device__ __forceinline__ Channels gated_channels(int64_t first, int64_t dim, int lane) {
    Channels c;
    const int64_t left = dim - first;
    if constexpr (kVec) {         // dim is a multiple of 4: all or none
        c.d = first + 4 * lane;
        c.live = c.d < dim ? 4 : 0;
    } else {
        c.d = first + lane;
        c.live = left <= lane ? 0 : (int)((left - lane + 31) / 32);
        c.live = c.live > 4 ? 4 : c.live;
    }
    return c;
}

template <typename IoT> struct Quad;
template <> struct Quad<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ float2 get(int k) const {
        const uint32_t w = k == 0 ? v.x : v.y;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};
template <> struct Quad<float> {
    float4 v;
    __device__ __forceinline__ float2 get(int k) const {
        return k == 0 ? make_float2(v.x, v.y) : make_float2(v.z, v.w);
    }
};

template <typename IoT, bool kVec>
__device__ __forceinline__ Quad<IoT> load_quad(const IoT* p, int live) {
    Quad<IoT> r;
    if constexpr (sizeof(IoT) == 2) {
        if constexpr (kVec) {
            r.v = live > 0 ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
        } else {
            const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
            r.v.x = (live > 0 ? (uint32_t)q[0] : 0u) | ((live > 1 ? (uint32_t)q[32] : 0u) << 16);
            r.v.y = (live > 2 ? (uint32_t)q[64] : 0u) | ((live > 3 ? (uint32_t)q[96] : 0u) << 16);
        }
    } else {
        if constexpr (kVec)
            r.v = live > 0 ? *reinterpret_cast<const float4*>(p) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        else
            r.v = make_float4(live > 0 ? p[0] : 0.0f, live > 1 ? p[32] : 0.0f, live > 2 ? p[64] : 0.0f,
                              live > 3 ? p[96] : 0.0f);
    }
    return r;
}

template <typename IoT, bool kVec>
__device__ __forceinline__ void store_quad(IoT* p, int live, float2 a, float2 b) {
    if constexpr (kVec) {
        if (live == 0) return;
        if constexpr (sizeof(IoT) == 2)
            *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y));
        else
            *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
    } else {
        if (live > 0) DType<IoT>::store(p, a.x);
        if (live > 1) DType<IoT>::store(p + 32, a.y);
        if (live > 2) DType<IoT>::store(p + 64, b.x);
        if (live > 3) DType<IoT>::store(p + 96, b.y);
    }
}

// kN steps; steps from `left` on are not read and give 0.
template <typename IoT, bool kVec, int kN>
__device__ __forceinline__ void load_quads(Quad<IoT> (&r)[kN], const IoT* p, int64_t stride, int left, int live) {
    if (left >= kN) {
#pragma unroll
        for (int i = 0; i < kN; ++i) r[i] = load_quad<IoT, kVec>(p + i * stride, live);
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) r[i] = load_quad<IoT, kVec>(p + i * stride, i < left ? live : 0);
    }
}

// Affine maps of a lane's four channels.
struct Maps { float2 A[kGatedPairs], H[kGatedPairs]; };
static_assert(kGatedPairs == 2, "four channels per lane");

__device__ __forceinline__ Maps identity_maps() {
    Maps m;
#pragma unroll
    for (int k = 0; k < kGatedPairs; ++k) {
        m.A[k] = make_float2(1.0f, 1.0f);
        m.H[k] = make_float2(0.0f, 0.0f);
    }
    return m;
}

// first, then second
__device__ __forceinline__ Maps compose(const Maps& first, const Maps& second) {
    Maps m;
#pragma unroll
    for (int k = 0; k < kGatedPairs; ++k) {
        m.A[k] = __fmul2_rn(second.A[k], first.A[k]);
        m.H[k] = __ffma2_rn(second.A[k], first.H[k], second.H[k]);
    }
    return m;
}

struct MapStore { float4 A, H; };

__device__ __forceinline__ MapStore pack_maps(const Maps& m) {
    return {make_float4(m.A[0].x, m.A[0].y, m.A[1].x, m.A[1].y), make_float4(m.H[0].x, m.H[0].y, m.H[1].x, m.H[1].y)};
}

__device__ __forceinline__ Maps unpack_maps(const float4& A, const float4& H) {
    Maps m;
    m.A[0] = make_float2(A.x, A.y);
    m.A[1] = make_float2(A.z, A.w);
    m.H[0] = make_float2(H.x, H.y);
    m.H[1] = make_float2(H.z, H.w);
    return m;
}

// Where a warp's block lies: item = position * groups + group, positions in the
// order of the scan (kReverse: the last segment of a chain first).
struct GatedBlockAt {
    int64_t b, group, pos, segment, block, t;
    Channels c;
    int left, rows;                                 // steps inside the sequence, inside the tensor
};

template <bool kReverse, bool kVec>
__device__ __forceinline__ GatedBlockAt gated_block(const GatedParams& p, int64_t item, int warp, int lane) {
    GatedBlockAt at;
    at.pos = item / p.groups;
    at.group = item - at.pos * p.groups;
    at.segment = kReverse ? p.segments - 1 - at.pos : at.pos;
    at.b = at.group / p.groups_per_row;
    at.c = gated_channels<kVec>((at.group - at.b * p.groups_per_row) * kGatedChannels, p.dim, lane);
    at.block = at.segment * (blockDim.x >> 5) + warp;
    at.t = at.block * kGatedBlock;
    const int64_t n = gated_length(p, at.b) - at.t, rows = p.seqlen - at.t;
    at.left = (int)(n < 0 ? 0 : (n > kGatedBlock ? kGatedBlock : n));
    at.rows = (int)(rows < 0 ? 0 : (rows > kGatedBlock ? kGatedBlock : rows));
    return at;
}

// Publishing: every lane has written its part; lane 0 raises the flag.
__device__ __forceinline__ void gated_publish(const GatedLinks& links, unsigned int* flag, int lane,
                                              unsigned int value) {
    __syncwarp();
    if (lane == 0 && !links.withhold) {
        __threadfence();
        store_release(flag, value);
    }
}

// The state entering segment `pos` of a chain (positions in scan order) for
// this lane's kP pairs of channels; called by one warp with the segment's own
// map (A, H).  Positions form groups of kGatedJoin.  The last of a group
// publishes the state that leaves it, the others their maps; a segment waits for
// the state entering its group and the maps of the group's earlier segments, and
// folds them in order.  h is the state entering position 0 and becomes the one
// entering pos.  False when the wait, or another of the call, ran out.
template <int kP>
__device__ __forceinline__ bool gated_join(const GatedLinks& links, int64_t group, int64_t pos, int lane,
                                           const float2 (&A)[kP], const float2 (&H)[kP], float2 (&h)[kP]) {
    const int64_t join = pos / kGatedJoin, first = join * kGatedJoin;
    const int before = (int)(pos - first);
    unsigned int* flags = links.flags + group * links.segments;
    float4* maps = links.maps + (group * links.segments) * (32 * kP) + lane;
    const int64_t joins = (links.segments + kGatedJoin - 1) / kGatedJoin;
    float2* states = links.states + (group * joins) * (32 * kP) + lane;
    const bool closes = before == kGatedJoin - 1;
    if (!closes && pos + 1 < links.segments) {
#pragma unroll
        for (int k = 0; k < kP; ++k)
            __stcg(maps + (pos * kP + k) * 32, make_float4(A[k].x, A[k].y, H[k].x, H[k].y));
        gated_publish(links, flags + pos, lane, 1u);
    }
    // lane l < before waits for the map of segment first + l, lane kGatedJoin for the state
    const bool wait_map = lane < before, wait_state = lane == kGatedJoin && join > 0;
    const unsigned int* mine = flags + (wait_map ? first + lane : first - 1);
    bool ready = !(wait_map || wait_state);
    unsigned int poll = 0;
    for (; poll < kGatedPollLimit; ++poll) {
        if (!ready) ready = load_acquire(mine) >= (wait_state ? 2u : 1u);
        if (__all_sync(0xffffffffu, ready)) break;
        if (gated_look(poll) && __any_sync(0xffffffffu, load_acquire(links.failed) != 0u)) return false;
    }
    if (poll == kGatedPollLimit) {
        if (lane == 0) gated_give_up(links.failed);
        return false;
    }
    __syncwarp();                                // what a lane has acquired, the warp may read
    if (join > 0)
#pragma unroll
        for (int k = 0; k < kP; ++k) h[k] = load_ordered(states + (join * kP + k) * 32);
    constexpr int kBatch = 8;                    // maps asked for together
    for (int c = 0; c < before; c += kBatch) {
        float4 m[kBatch][kP];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int k = 0; k < kP; ++k)
                m[i][k] = c + i < before ? load_ordered(maps + ((first + c + i) * kP + k) * 32)
                                         : make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int k = 0; k < kP; ++k)
                h[k] = __ffma2_rn(make_float2(m[i][k].x, m[i][k].y), h[k], make_float2(m[i][k].z, m[i][k].w));
    }
    if (closes && pos + 1 < links.segments) {
#pragma unroll
        for (int k = 0; k < kP; ++k) __stcg(states + ((join + 1) * kP + k) * 32, __ffma2_rn(A[k], h[k], H[k]));
        gated_publish(links, flags + pos, lane, 2u);
    }
    return true;
}

// The first item of a CTA.
__device__ __forceinline__ int64_t gated_first_item(const GatedParams& p, int64_t* slot) {
    if (p.ticket == nullptr) return blockIdx.x;
    if (threadIdx.x == 0) *slot = atomicAdd(p.ticket, 1u);
    __syncthreads();
    return *slot;
}

// Joins the warps' maps (in shared memory) and the segments': h, the state
// entering position 0 of the chain, becomes the one entering this warp's block.
// False, for the whole CTA, when a wait ran out: it takes no further item.
template <bool kReverse>
__device__ __forceinline__ bool gated_enter(const GatedParams& p, const GatedBlockAt& at, int warp, int lane,
                                            const float4 (&sA)[kGatedWarps][32], const float4 (&sH)[kGatedWarps][32],
                                            float4 (&entering)[32], float2 (&h)[kGatedPairs]) {
    const int warps = blockDim.x >> 5;
    bool lost = false;
    const int rank = kReverse ? warps - 1 - warp : warp;             // in scan order
    if (p.ticket != nullptr && warp == 0) {
        Maps all = identity_maps();
        for (int v = 0; v < warps; ++v) {
            const int w = kReverse ? warps - 1 - v : v;
            all = compose(all, unpack_maps(sA[w][lane], sH[w][lane]));
        }
        float2 e[kGatedPairs] = {h[0], h[1]};
        // a wait that ran out is recorded; the call's outputs are undefined then
        lost = !gated_join<kGatedPairs>(p.links, at.group, at.pos, lane, all.A, all.H, e);
        entering[lane] = make_float4(e[0].x, e[0].y, e[1].x, e[1].y);
    }
    Maps mine = identity_maps();
    for (int v = 0; v < rank; ++v) {
        const int w = kReverse ? warps - 1 - v : v;
        mine = compose(mine, unpack_maps(sA[w][lane], sH[w][lane]));
    }
    if (p.ticket != nullptr) {
        if (__syncthreads_or(lost)) return false;
        const float4 e = entering[lane];
        h[0] = make_float2(e.x, e.y);
        h[1] = make_float2(e.z, e.w);
    }
#pragma unroll
    for (int k = 0; k < kGatedPairs; ++k) h[k] = __ffma2_rn(mine.A[k], h[k], mine.H[k]);
    return true;
}

template <bool kVec>
__device__ __forceinline__ void load_state(const float* base, int64_t row, int64_t dim, const Channels& c,
                                           float2 (&h)[kGatedPairs]) {
    if (base == nullptr) {
        h[0] = h[1] = make_float2(0.0f, 0.0f);
        return;
    }
    const Quad<float> q = load_quad<float, kVec>(base + row * dim + c.d, c.live);
    h[0] = q.get(0);
    h[1] = q.get(1);
}

constexpr int kGatedSub = 4;                 // steps requested at a time

// Walks `left` steps, kGatedSub at a time.
template <typename IoT, typename Load, typename Work>
__device__ __forceinline__ void walk_block(int left, Load load, Work work) {
    for (int s = 0; s < left; s += kGatedSub) {
        Quad<IoT> f[kGatedSub], x[kGatedSub];
        load(f, x, s);
        work(f, x, s);
    }
}

template <typename IoT, bool kLog, bool kVec>
__global__ void __launch_bounds__(kGatedThreads, sizeof(IoT) == 2 ? 4 : 2)
    gated_scan_fwd_kernel(const __grid_constant__ GatedParams p) {
    __shared__ float4 sA[kGatedWarps][32], sH[kGatedWarps][32];
    __shared__ float4 entering[32];
    __shared__ int64_t first_slot, next_slot;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2 zero = make_float2(0.0f, 0.0f), one = make_float2(1.0f, 1.0f);
    int64_t item = gated_first_item(p, &first_slot);
    while (item < p.items) {
        const GatedBlockAt at = gated_block<false, kVec>(p, item, warp, lane);
        const int live = at.c.live;
        float2 bias2[kGatedPairs], h[kGatedPairs];
        load_state<kVec>(p.bias, 0, p.dim, at.c, bias2);
        bias2[0] = __fmul2_rn(bias2[0], make_float2(kLog2e, kLog2e));
        bias2[1] = __fmul2_rn(bias2[1], make_float2(kLog2e, kLog2e));
        load_state<kVec>(p.h0, at.b, p.dim, at.c, h);
        const IoT* gate = static_cast<const IoT*>(p.gate) + at.b * p.gate_s.batch + at.t * p.gate_s.row + at.c.d;
        const IoT* x = static_cast<const IoT*>(p.x) + at.b * p.x_s.batch + at.t * p.x_s.row + at.c.d;
        int64_t following = p.items;
        if (p.blocks > 1) {
            int64_t coming = 0;                  // asked for now, needed at the barrier
            if (threadIdx.x == 0 && p.ticket != nullptr) coming = atomicAdd(p.ticket, 1u);
            Maps m = identity_maps();
            const IoT* gs = gate;
            const IoT* xs = x;
            walk_block<IoT>(
                at.left,
                [&](Quad<IoT> (&rf)[kGatedSub], Quad<IoT> (&rx)[kGatedSub], int s) {
                    load_quads<IoT, kVec>(rf, gs, p.gate_s.row, at.left - s, live);
                    load_quads<IoT, kVec>(rx, xs, p.x_s.row, at.left - s, live);
                    gs += kGatedSub * p.gate_s.row;
                    xs += kGatedSub * p.x_s.row;
                },
                [&](const Quad<IoT> (&rf)[kGatedSub], const Quad<IoT> (&rx)[kGatedSub], int s) {
                    float2 a[kGatedSub][kGatedPairs], u[kGatedSub][kGatedPairs];
#pragma unroll
                    for (int i = 0; i < kGatedSub; ++i)
#pragma unroll
                        for (int k = 0; k < kGatedPairs; ++k)
                            gated_terms2<kLog>(rf[i].get(k), bias2[k], rx[i].get(k), a[i][k], u[i][k]);
                    if (at.left - s < kGatedSub)
#pragma unroll
                        for (int i = 0; i < kGatedSub; ++i)
                            if (s + i >= at.left) a[i][0] = a[i][1] = one;       // u is 0: x was not read
#pragma unroll
                    for (int i = 0; i < kGatedSub; ++i)
#pragma unroll
                        for (int k = 0; k < kGatedPairs; ++k) {
                            m.H[k] = __ffma2_rn(a[i][k], m.H[k], u[i][k]);
                            m.A[k] = __fmul2_rn(m.A[k], a[i][k]);
                        }
                });
            const MapStore ms = pack_maps(m);
            sA[warp][lane] = ms.A;
            sH[warp][lane] = ms.H;
            if (threadIdx.x == 0) next_slot = coming;
            __syncthreads();
            if (p.ticket != nullptr) following = next_slot;
            if (!gated_enter<false>(p, at, warp, lane, sA, sH, entering, h)) break;
        }
        if (at.rows > 0 && p.enter != nullptr)
            store_quad<float, kVec>(p.enter + (at.b * p.blocks + at.block) * p.dim + at.c.d, live, h[0], h[1]);
        if (p.out != nullptr) {
            IoT* out = static_cast<IoT*>(p.out) + at.b * p.out_s.batch + at.t * p.out_s.row + at.c.d;
            walk_block<IoT>(
                at.left,
                [&](Quad<IoT> (&rf)[kGatedSub], Quad<IoT> (&rx)[kGatedSub], int s) {
                    load_quads<IoT, kVec>(rf, gate, p.gate_s.row, at.left - s, live);
                    load_quads<IoT, kVec>(rx, x, p.x_s.row, at.left - s, live);
                    gate += kGatedSub * p.gate_s.row;
                    x += kGatedSub * p.x_s.row;
                },
                [&](const Quad<IoT> (&rf)[kGatedSub], const Quad<IoT> (&rx)[kGatedSub], int s) {
                    float2 a[kGatedSub][kGatedPairs], u[kGatedSub][kGatedPairs];
#pragma unroll
                    for (int i = 0; i < kGatedSub; ++i)
#pragma unroll
                        for (int k = 0; k < kGatedPairs; ++k)
                            gated_terms2<kLog>(rf[i].get(k), bias2[k], rx[i].get(k), a[i][k], u[i][k]);
#pragma unroll
                    for (int i = 0; i < kGatedSub; ++i) {
                        const bool in = s + i < at.left;
                        if (in) {
                            h[0] = __ffma2_rn(a[i][0], h[0], u[i][0]);
                            h[1] = __ffma2_rn(a[i][1], h[1], u[i][1]);
                        }
                        if (s + i < at.rows)
                            store_quad<IoT, kVec>(out + i * p.out_s.row, live, in ? h[0] : zero, in ? h[1] : zero);
                    }
                    out += kGatedSub * p.out_s.row;
                });
            int s = (at.left + kGatedSub - 1) / kGatedSub * kGatedSub;
            for (; s < at.rows; ++s, out += p.out_s.row) store_quad<IoT, kVec>(out, live, zero, zero);
            if (p.last != nullptr && at.block == p.blocks - 1)
                store_quad<float, kVec>(p.last + at.b * p.dim + at.c.d, live, h[0], h[1]);
        }
        item = following;
    }
}

// Backward.  Phase one walks a block forward from its checkpoint, keeps the
// state every kGatedSub steps in shared memory and accumulates the block's map
// of r, R = sum_t (prod_{s <= t} a_s) dout_t; phase two walks it backward.
constexpr int kGatedKept = kGatedBlock / kGatedSub;
constexpr int kGatedBwdSmem = kGatedWarps * kGatedKept * 32 * (int)sizeof(float4);

template <typename IoT, bool kLog, bool kVec>
__global__ void __launch_bounds__(kGatedThreads, 2)
    gated_scan_bwd_kernel(const __grid_constant__ GatedParams p) {
    __shared__ float4 sA[kGatedWarps][32], sH[kGatedWarps][32];
    __shared__ float4 entering[32];
    __shared__ int64_t first_slot, next_slot;
    extern __shared__ float4 kept_all[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float4* kept = kept_all + warp * kGatedKept * 32 + lane;
    const float2 zero = make_float2(0.0f, 0.0f), one = make_float2(1.0f, 1.0f);
    int64_t item = gated_first_item(p, &first_slot);
    while (item < p.items) {
        const GatedBlockAt at = gated_block<true, kVec>(p, item, warp, lane);
        const int live = at.c.live;
        float2 bias2[kGatedPairs], h[kGatedPairs];
        load_state<kVec>(p.bias, 0, p.dim, at.c, bias2);
        bias2[0] = __fmul2_rn(bias2[0], make_float2(kLog2e, kLog2e));
        bias2[1] = __fmul2_rn(bias2[1], make_float2(kLog2e, kLog2e));
        const IoT* gate = static_cast<const IoT*>(p.gate) + at.b * p.gate_s.batch + at.t * p.gate_s.row + at.c.d;
        const IoT* x = static_cast<const IoT*>(p.x) + at.b * p.x_s.batch + at.t * p.x_s.row + at.c.d;
        const IoT* dout = static_cast<const IoT*>(p.dout) + at.b * p.out_s.batch + at.t * p.out_s.row + at.c.d;
        int64_t coming = 0;                      // asked for now, needed at the barrier
        if (threadIdx.x == 0 && p.ticket != nullptr) coming = atomicAdd(p.ticket, 1u);
        load_state<kVec>(at.rows > 0 ? p.enter : nullptr, at.b * p.blocks + at.block, p.dim, at.c, h);
        Maps m = identity_maps();
        struct Raw { Quad<IoT> f[kGatedSub], x[kGatedSub], d[kGatedSub]; };
        auto load = [&](Raw& r, int s) {
            load_quads<IoT, kVec>(r.f, gate, p.gate_s.row, at.left - s, live);
            load_quads<IoT, kVec>(r.x, x, p.x_s.row, at.left - s, live);
            load_quads<IoT, kVec>(r.d, dout, p.out_s.row, at.left - s, live);
        };
        auto forward = [&](const Raw& r, int s) {
            kept[s / kGatedSub * 32] = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
#pragma unroll
            for (int i = 0; i < kGatedSub; ++i)
#pragma unroll
                for (int k = 0; k < kGatedPairs; ++k) {
                    float2 a, u;
                    gated_terms2<kLog>(r.f[i].get(k), bias2[k], r.x[i].get(k), a, u);
                    if (s + i >= at.left) a = one;              // u and dout are 0: not read
                    h[k] = __ffma2_rn(a, h[k], u);
                    m.A[k] = __fmul2_rn(m.A[k], a);
                    m.H[k] = __ffma2_rn(m.A[k], r.d[i].get(k), m.H[k]);
                }
        };
        auto move = [&](int steps) {
            gate += steps * p.gate_s.row;
            x += steps * p.x_s.row;
            dout += steps * p.out_s.row;
        };
        // 16-bit inputs: registers for the next steps' loads under way
        constexpr bool kAhead = sizeof(IoT) == 2;
        Raw ra, rb;
        if constexpr (kAhead) {
            if (at.left > 0) load(ra, 0);
            for (int s = 0; s < at.left; s += 2 * kGatedSub) {
                move(kGatedSub);
                if (s + kGatedSub < at.left) load(rb, s + kGatedSub);
                forward(ra, s);
                if (s + kGatedSub >= at.left) break;
                move(kGatedSub);
                if (s + 2 * kGatedSub < at.left) load(ra, s + 2 * kGatedSub);
                forward(rb, s + kGatedSub);
            }
        } else {
            for (int s = 0; s < at.left; s += kGatedSub) {
                Raw raw;
                load(raw, s);
                move(kGatedSub);
                forward(raw, s);
            }
        }
        // the pointers now stand at the block's end, in whole groups of kGatedSub steps
        float2 r[kGatedPairs];
        // before the barrier: dh0 may replace dlast, and block 0 may be done early
        load_state<kVec>(p.dlast, at.b, p.dim, at.c, r);
        const MapStore ms = pack_maps(m);
        sA[warp][lane] = ms.A;
        sH[warp][lane] = ms.H;
        if (threadIdx.x == 0) next_slot = coming;
        __syncthreads();
        const int64_t following = p.ticket != nullptr ? next_slot : p.items;
        // phase two's first loads, under way during the join
        if (kAhead && at.left > 0) {
            move(-kGatedSub);
            load(ra, (at.left - 1) / kGatedSub * kGatedSub);
        }
        if (!gated_enter<true>(p, at, warp, lane, sA, sH, entering, r)) break;

        float2 db[kGatedPairs] = {zero, zero};
        IoT* dgate = static_cast<IoT*>(p.dgate) + at.b * p.dgate_s.batch + at.t * p.dgate_s.row + at.c.d;
        IoT* dx = static_cast<IoT*>(p.dx) + at.b * p.dx_s.batch + at.t * p.dx_s.row + at.c.d;
        for (int s = at.left; s < at.rows; ++s) {
            store_quad<IoT, kVec>(dgate + s * p.dgate_s.row, live, zero, zero);
            store_quad<IoT, kVec>(dx + s * p.dx_s.row, live, zero, zero);
        }
        const int top = (at.left + kGatedSub - 1) / kGatedSub * kGatedSub;
        dgate += top * p.dgate_s.row;
        dx += top * p.dx_s.row;
        auto backward = [&](const Raw& raw, int s) {
            const int left = at.left - s;
            dgate -= kGatedSub * p.dgate_s.row;
            dx -= kGatedSub * p.dx_s.row;
            float2 a[kGatedSub][kGatedPairs], g[kGatedSub][kGatedPairs], before[kGatedSub][kGatedPairs];
            const float4 hk = kept[s / kGatedSub * 32];
            h[0] = make_float2(hk.x, hk.y);
            h[1] = make_float2(hk.z, hk.w);
#pragma unroll
            for (int i = 0; i < kGatedSub; ++i)
#pragma unroll
                for (int k = 0; k < kGatedPairs; ++k) {
                    gated_gains2<kLog>(raw.f[i].get(k), bias2[k], g[i][k], a[i][k]);
                    before[i][k] = h[k];
                    h[k] = __ffma2_rn(a[i][k], h[k], kLog ? raw.x[i].get(k) : __fmul2_rn(g[i][k], raw.x[i].get(k)));
                }
#pragma unroll
            for (int i = kGatedSub - 1; i >= 0; --i)
                if (i < left) {
                    float2 df[kGatedPairs], dv[kGatedPairs];
#pragma unroll
                    for (int k = 0; k < kGatedPairs; ++k) {
                        const float2 l = __fadd2_rn(raw.d[i].get(k), r[k]);
                        r[k] = __fmul2_rn(a[i][k], l);
                        if constexpr (kLog) {
                            dv[k] = l;
                            df[k] = __fmul2_rn(r[k], before[i][k]);
                        } else {
                            const float2 diff = __ffma2_rn(before[i][k], make_float2(-1.0f, -1.0f), raw.x[i].get(k));
                            dv[k] = __fmul2_rn(g[i][k], l);
                            df[k] = __fmul2_rn(__fmul2_rn(g[i][k], r[k]), diff);
                        }
                        db[k] = __fadd2_rn(db[k], df[k]);
                    }
                    store_quad<IoT, kVec>(dgate + i * p.dgate_s.row, live, df[0], df[1]);
                    store_quad<IoT, kVec>(dx + i * p.dx_s.row, live, dv[0], dv[1]);
                }
        };
        if constexpr (kAhead) {
            for (int s = top - kGatedSub; s >= 0; s -= 2 * kGatedSub) {
                if (s > 0) {
                    move(-kGatedSub);
                    load(rb, s - kGatedSub);
                }
                backward(ra, s);
                if (s == 0) break;
                if (s > kGatedSub) {
                    move(-kGatedSub);
                    load(ra, s - 2 * kGatedSub);
                }
                backward(rb, s - kGatedSub);
            }
        } else {
            for (int s = top - kGatedSub; s >= 0; s -= kGatedSub) {
                Raw raw;
                move(-kGatedSub);
                load(raw, s);
                backward(raw, s);
            }
        }
        if (p.dh0 != nullptr && at.block == 0)
            store_quad<float, kVec>(p.dh0 + at.b * p.dim + at.c.d, live, r[0], r[1]);
        if (p.bias_partial != nullptr) {
            // the warps' sums, in order; kept is free again (each lane's own entries)
            kept[0] = make_float4(db[0].x, db[0].y, db[1].x, db[1].y);
            __syncthreads();
            if (warp == 0) {
                float2 sum[kGatedPairs] = {zero, zero};
                for (int v = 0; v < warps; ++v) {
                    const float4 q = kept[v * kGatedKept * 32];
                    sum[0] = __fadd2_rn(sum[0], make_float2(q.x, q.y));
                    sum[1] = __fadd2_rn(sum[1], make_float2(q.z, q.w));
                }
                store_quad<float, kVec>(p.bias_partial + (at.b * p.segments + at.segment) * p.dim + at.c.d, live,
                                        sum[0], sum[1]);
            }
            __syncthreads();
        }
        item = following;
    }
}

// ------------------------------------------------ (batch, dim, seqlen) layout
// Two neighbouring chains side by side, one per half of the packed arithmetic.

// Compositions over a team of `width` lanes in scan order (kReverse: from the
// team's last lane down): (A, H) becomes the map of the lanes up to this one.
template <bool kReverse>
__device__ __forceinline__ void team_scan(float2& A, float2& H, int rank, int width) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        if (o >= width) break;
        const float2 Ao = kReverse ? shfl_down2(A, o, width) : shfl_up2(A, o, width);
        const float2 Ho = kReverse ? shfl_down2(H, o, width) : shfl_up2(H, o, width);
        if (kReverse ? rank + o < width : rank >= o) {
            H = __ffma2_rn(A, Ho, H);
            A = __fmul2_rn(A, Ao);
        }
    }
}

// The state entering this warp's part of a tile: folds the maps of the `warps`
// warps that share a pair of chains, `maps` being the first one's.  carry, the
// state entering the tile, becomes the one that leaves it.
template <bool kReverse>
__device__ __forceinline__ float2 fold_warps(float2& carry, const float4* maps, int rank, int warps) {
    float2 h = carry;
#pragma unroll
    for (int k = 0; k < kRowWarps; ++k) {
        if (k == warps) break;
        const int v = kReverse ? warps - 1 - k : k;
        if (v == rank) h = carry;
        const float4 m = maps[v];
        carry = __ffma2_rn(make_float2(m.x, m.y), carry, make_float2(m.z, m.w));
    }
    return h;
}

// The state entering a lane, from its inclusive map and the state h entering its
// warp (team); `leaving`, if asked for, becomes the state behind the team.
template <bool kReverse, bool kLeaving>
__device__ __forceinline__ float2 enter_lane(float2 A, float2 H, float2 h, float2* leaving, int rank, int width) {
    const float2 mine = __ffma2_rn(A, h, H);
    if constexpr (kLeaving) *leaving = shfl2(mine, kReverse ? 0 : width - 1, width);
    const float2 before = kReverse ? shfl_down2(mine, 1, width) : shfl_up2(mine, 1, width);
    return rank == (kReverse ? width - 1 : 0) ? h : before;
}

// Pairs of neighbouring channels of a batch row (an odd one's last has one chain),
// in the order in which a team takes them.  Fewer than 2^31 chains.
struct PairWalk {
    int64_t pair, pairs;
    int b, half;                            // batch row, pair within it
    int halves, step_b, step_half;
    __device__ __forceinline__ PairWalk(const GatedParams& p, int64_t first, int64_t stride) {
        halves = (int)((p.dim + 1) / 2);
        pairs = p.batch * halves;
        pair = first;
        b = (int)(first / halves);
        half = (int)(first - (int64_t)b * halves);
        step_b = (int)(stride / halves);
        step_half = (int)(stride - (int64_t)step_b * halves);
        stride_ = stride;
    }
    __device__ __forceinline__ void advance() {
        pair += stride_;
        b += step_b;
        half += step_half;
        if (half >= halves) {
            half -= halves;
            ++b;
        }
    }
    int64_t stride_;
};

// A lane's pair of chains.
template <typename IoT>
struct GatedRows {
    int b, d;                               // of the first; the second is channel d + 1
    bool live0, live1;
    int shift0, shift1;                     // first step of this lane in tile 0
    __device__ __forceinline__ GatedRows(const GatedParams& p, const PairWalk& at, int offset) {
        live0 = at.pair < at.pairs;
        b = live0 ? at.b : 0;
        d = live0 ? 2 * at.half : 0;
        live1 = live0 && d + 1 < (int)p.dim;
        shift0 = offset - row_phase(row0(p.gate, p.gate_s));
        shift1 = offset - row_phase(row1(p.gate, p.gate_s));
    }
    __device__ __forceinline__ IoT* row0(const void* base, const GatedStrides& s) const {
        return const_cast<IoT*>(static_cast<const IoT*>(base)) + b * s.batch + d * s.row;
    }
    __device__ __forceinline__ IoT* row1(const void* base, const GatedStrides& s) const {
        return row0(base, s) + (live1 ? s.row : 0);
    }
    // one value per channel, per chain
    __device__ __forceinline__ float2 pick(const float* v, int64_t i) const {
        return v != nullptr ? make_float2(v[i], v[i + (live1 ? 1 : 0)]) : make_float2(0.0f, 0.0f);
    }
    __device__ __forceinline__ void put(float* v, int64_t i, float2 x) const {
        if (v == nullptr) return;
        if (live0) v[i] = x.x;
        if (live1) v[i + 1] = x.y;
    }
};

// The bytes between a tensor's first and last element, (batch, dim) rows of seqlen.
template <typename IoT>
__device__ __forceinline__ Span gated_span(const GatedParams& p, const void* base, const GatedStrides& s) {
    const unsigned char* b = static_cast<const unsigned char*>(base);
    return {b, b + ((p.batch - 1) * s.batch + (p.dim - 1) * s.row + p.seqlen) * (int64_t)sizeof(IoT)};
}

// Gains of a lane's eight steps; steps outside a sequence pass the state on.
template <bool kLog>
__device__ __forceinline__ void row_gains(float2 (&a)[8], float2 (&g)[8], float2 bias2, bool inside, int t0, int n0,
                                          int t1, int n1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) gated_gains2<kLog>(a[i], bias2, g[i], a[i]);
    if (!inside)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (t0 + i < 0 || t0 + i >= n0) {
                a[i].x = 1.0f;
                g[i].x = 0.0f;
            }
            if (t1 + i < 0 || t1 + i >= n1) {
                a[i].y = 1.0f;
                g[i].y = 0.0f;
            }
        }
}

// A lane's eight steps of two rows, for kTensors tensors, come through its own slots
// in shared memory (16 bytes per thread side by side): the next tile is on its way
// while this one is worked on.  What cannot be copied as aligned vectors inside the
// tensor is read element by element when its turn comes; a bit of `ok` per vector
// says which was copied.
template <typename IoT, int kTensors>
struct RowStages {
    static constexpr int kVecs = (int)sizeof(IoT) / 2;
    static constexpr int kStages = 2;
    static constexpr int kBytesPerThread = kStages * kTensors * 2 * kVecs * 16;
    uint4* own;
    __device__ __forceinline__ explicit RowStages(unsigned char* smem) : own(reinterpret_cast<uint4*>(smem) + threadIdx.x) {}
    __device__ __forceinline__ uint4* slot(int stage, int tensor, int row) const {
        return own + ((stage * kTensors + tensor) * 2 + row) * kVecs * blockDim.x;
    }
    // Both rows' vectors of a tensor; in0, in1: is the vector inside its row?
    __device__ __forceinline__ uint32_t copy(int stage, int tensor, const IoT* q0, bool in0, const IoT* q1, bool in1,
                                             const Span& span) const {
        return copy_row(stage, tensor, 0, q0, in0, span) | copy_row(stage, tensor, 1, q1, in1, span);
    }
    __device__ __forceinline__ uint32_t copy_row(int stage, int tensor, int row, const IoT* q, bool inside,
                                                 const Span& span) const {
        if (!inside) inside = span.holds(q, 8 * (int)sizeof(IoT));
        if ((reinterpret_cast<uintptr_t>(q) & 15) != 0 || !inside) return 0u;
        uint4* dst = slot(stage, tensor, row);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) copy_async16(smem_u32(dst + i * blockDim.x), reinterpret_cast<const uint4*>(q) + i);
        return 1u << (2 * tensor + row);
    }
    __device__ __forceinline__ void get(int stage, int tensor, float2 (&v)[8]) const {
        uint4 raw0[kVecs], raw1[kVecs];
        float a[8], b[8];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            raw0[i] = slot(stage, tensor, 0)[i * blockDim.x];
            raw1[i] = slot(stage, tensor, 1)[i * blockDim.x];
        }
        unpack_steps<IoT>(raw0, a);
        unpack_steps<IoT>(raw1, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = make_float2(a[i], b[i]);
    }
    // Steps outside [0, n) become 0; those that no vector brought are read.
    __device__ __forceinline__ static void fill(float2 (&v)[8], uint32_t ok, int tensor, const IoT* p0, int t0, int n0,
                                                const IoT* p1, int t1, int n1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (t0 + i < 0 || t0 + i >= n0) v[i].x = 0.0f;
            if (t1 + i < 0 || t1 + i >= n1) v[i].y = 0.0f;
        }
        if (!(ok >> (2 * tensor) & 1u))
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t0 + i >= 0 && t0 + i < n0) v[i].x = DType<IoT>::load(p0 + i);
        if (!(ok >> (2 * tensor + 1) & 1u))
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t1 + i >= 0 && t1 + i < n1) v[i].y = DType<IoT>::load(p1 + i);
    }
};

__device__ __forceinline__ bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename IoT>
__device__ __forceinline__ void store_pair_rows(IoT* p0, IoT* p1, const float2 (&v)[8]) {
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = v[i].x;
        b[i] = v[i].y;
    }
    store_eight(p0, a);
    store_eight(p1, b);
}

template <typename IoT, bool kLog, bool kMulti>
__global__ void __launch_bounds__(kRowThreads, 3)
    gated_scan_rows_fwd_kernel(const __grid_constant__ GatedParams p, int warps, int width_, int64_t blocks) {
    extern __shared__ __align__(128) unsigned char raw[];
    __shared__ float4 buf[2][kRowWarps];
    const RowStages<IoT, 2> ring(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int width = kMulti ? 32 : width_;              // lanes of a pair in a warp
    const int teams = (kMulti ? (int)(blockDim.x >> 5) / warps : (int)blockDim.x / width);
    const int team = kMulti ? warp / warps : (int)threadIdx.x / width;
    const int rank = kMulti ? warp - team * warps : 0, at_lane = lane & (width - 1);
    const int offset = rank * kWarpSteps + at_lane * kLaneSteps;
    const int tiles = (int)p.tiles, step = (kMulti ? warps : 1) * width * kLaneSteps, L = (int)p.seqlen;
    const Span gspan = gated_span<IoT>(p, p.gate, p.gate_s), xspan = gated_span<IoT>(p, p.x, p.x_s);
    auto request = [&](const GatedRows<IoT>& at, int tile, int stage) {
        const int t0 = tile * step + at.shift0, t1 = tile * step + at.shift1;
        const bool in0 = t0 >= 0 && t0 + 8 <= L, in1 = t1 >= 0 && t1 + 8 <= L;
        return ring.copy(stage, 0, at.row0(p.gate, p.gate_s) + t0, in0, at.row1(p.gate, p.gate_s) + t1, in1, gspan) |
               ring.copy(stage, 1, at.row0(p.x, p.x_s) + t0, in0, at.row1(p.x, p.x_s) + t1, in1, xspan);
    };
    PairWalk walk(p, (int64_t)blockIdx.x * teams + team, (int64_t)gridDim.x * teams);
    uint32_t ok_next = request(GatedRows<IoT>(p, walk, offset), 0, 0);
    copy_async_commit();
    int stage = 0;
    for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const GatedRows<IoT> at(p, walk, offset);
        const int n = (int)gated_length(p, at.b), n0 = at.live0 ? n : 0, n1 = at.live1 ? n : 0;
        const int64_t chain = (int64_t)at.b * p.dim + at.d;
        const float2 bias2 = __fmul2_rn(at.pick(p.bias, at.d), make_float2(kLog2e, kLog2e));
        float2 carry = at.pick(p.h0, chain);
        for (int tile = 0; tile < tiles; ++tile, stage ^= 1) {
            const uint32_t ok = ok_next;
            if (tile + 1 < tiles) {
                ok_next = request(at, tile + 1, stage ^ 1);
            } else if (block + gridDim.x < blocks) {
                walk.advance();
                ok_next = request(GatedRows<IoT>(p, walk, offset), 0, stage ^ 1);
            }
            copy_async_commit();
            copy_async_wait<1>();
            const int t0 = tile * step + at.shift0, t1 = tile * step + at.shift1;
            IoT *out0 = at.row0(p.out, p.out_s), *out1 = at.row1(p.out, p.out_s);
            float2 a[8], u[8], g[8];
            // the whole warp inside both sequences, on vectors
            const bool whole = __all_sync(0xffffffffu, t0 >= 0 && t1 >= 0 && t0 + 8 <= n0 && t1 + 8 <= n1 &&
                                                           ok == 15u && on16(out0 + t0) && on16(out1 + t1));
            ring.get(stage, 0, a);
            ring.get(stage, 1, u);
            if (!whole) {
                ring.fill(a, ok, 0, at.row0(p.gate, p.gate_s) + t0, t0, n0, at.row1(p.gate, p.gate_s) + t1, t1, n1);
                ring.fill(u, ok, 1, at.row0(p.x, p.x_s) + t0, t0, n0, at.row1(p.x, p.x_s) + t1, t1, n1);
            }
            row_gains<kLog>(a, g, bias2, whole, t0, n0, t1, n1);
            float2 A = make_float2(1.0f, 1.0f), H = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (!kLog) u[i] = __fmul2_rn(g[i], u[i]);
                H = i == 0 ? u[0] : __ffma2_rn(a[i], H, u[i]);
                A = i == 0 ? a[0] : __fmul2_rn(A, a[i]);
            }
            team_scan<false>(A, H, at_lane, width);
            float2 h;
            if constexpr (kMulti) {
                if (lane == 31) buf[stage][warp] = make_float4(A.x, A.y, H.x, H.y);
                __syncthreads();
                h = fold_warps<false>(carry, buf[stage] + warp - rank, rank, warps);
                h = enter_lane<false, false>(A, H, h, nullptr, at_lane, width);
            } else {
                h = enter_lane<false, true>(A, H, carry, &carry, at_lane, width);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h = __ffma2_rn(a[i], h, u[i]);
                u[i] = h;
            }
            if (whole) {
                store_pair_rows(out0 + t0, out1 + t1, u);
                continue;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (t0 + i >= n0) u[i].x = 0.0f;
                if (t1 + i >= n1) u[i].y = 0.0f;
            }
            store_steps2(out0, t0, 0, at.live0 ? L : 0, out1, t1, 0, at.live1 ? L : 0, u);
        }
        if (offset == 0) at.put(p.last, chain, carry);
    }
}

// Backward: with more than one tile per chain, a first sweep keeps the states
// entering the tiles; the second runs from the last tile to the first and reads
// gate and x again (from L2 while the chains in flight fit there).
template <typename IoT, bool kLog, bool kMulti>
__global__ void __launch_bounds__(kRowThreads, 2)
    gated_scan_rows_bwd_kernel(const __grid_constant__ GatedParams p, int warps, int width_, int64_t blocks) {
    extern __shared__ __align__(128) unsigned char raw[];
    __shared__ float4 buf[2][kRowWarps], back[2][kRowWarps];
    __shared__ float2 sums[kRowWarps];
    const RowStages<IoT, 3> ring(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2 one = make_float2(1.0f, 1.0f), zero = make_float2(0.0f, 0.0f);
    const int width = kMulti ? 32 : width_;              // lanes of a pair in a warp
    const int teams = (kMulti ? (int)(blockDim.x >> 5) / warps : (int)blockDim.x / width);
    const int team = kMulti ? warp / warps : (int)threadIdx.x / width;
    const int rank = kMulti ? warp - team * warps : 0, at_lane = lane & (width - 1);
    const int offset = rank * kWarpSteps + at_lane * kLaneSteps;
    const int tiles = (int)p.tiles, step = (kMulti ? warps : 1) * width * kLaneSteps, L = (int)p.seqlen;
    const Span gspan = gated_span<IoT>(p, p.gate, p.gate_s), xspan = gated_span<IoT>(p, p.x, p.x_s),
               dspan = gated_span<IoT>(p, p.dout, p.out_s);
    // a pair's items: tiles 0 .. tiles - 2 of the first sweep, then all backwards
    const int64_t items = 2 * (int64_t)tiles - 1;
    auto request = [&](const GatedRows<IoT>& at, int64_t item, int stage) {
        const bool sweep = item < tiles - 1;
        const int tile = (int)(sweep ? item : items - 1 - item);
        const int t0 = tile * step + at.shift0, t1 = tile * step + at.shift1;
        const bool in0 = t0 >= 0 && t0 + 8 <= L, in1 = t1 >= 0 && t1 + 8 <= L;
        uint32_t ok =
            ring.copy(stage, 0, at.row0(p.gate, p.gate_s) + t0, in0, at.row1(p.gate, p.gate_s) + t1, in1, gspan) |
            ring.copy(stage, 1, at.row0(p.x, p.x_s) + t0, in0, at.row1(p.x, p.x_s) + t1, in1, xspan);
        if (!sweep)
            ok |= ring.copy(stage, 2, at.row0(p.dout, p.out_s) + t0, in0, at.row1(p.dout, p.out_s) + t1, in1, dspan);
        return ok;
    };
    PairWalk walk(p, (int64_t)blockIdx.x * teams + team, (int64_t)gridDim.x * teams);
    uint32_t ok_next = request(GatedRows<IoT>(p, walk, offset), 0, 0);
    copy_async_commit();
    int stage = 0;
    for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const GatedRows<IoT> at(p, walk, offset);
        const int n = (int)gated_length(p, at.b), n0 = at.live0 ? n : 0, n1 = at.live1 ? n : 0;
        const int64_t chain = (int64_t)at.b * p.dim + at.d;
        const float2 bias2 = __fmul2_rn(at.pick(p.bias, at.d), make_float2(kLog2e, kLog2e));
        float2 carry = at.pick(p.h0, chain), r_carry = at.pick(p.dlast, chain);
        float2 db = zero;
        float* states0 = p.chain_states + chain * p.tiles;
        float* states1 = states0 + (at.live1 ? p.tiles : 0);
        for (int64_t item = 0; item < items; ++item, stage ^= 1) {
            const bool sweep = item < tiles - 1;
            const int tile = (int)(sweep ? item : items - 1 - item);
            const uint32_t ok = ok_next;
            if (item + 1 < items) {
                ok_next = request(at, item + 1, stage ^ 1);
            } else if (block + gridDim.x < blocks) {
                walk.advance();
                ok_next = request(GatedRows<IoT>(p, walk, offset), 0, stage ^ 1);
            }
            copy_async_commit();
            copy_async_wait<1>();
            const int t0 = tile * step + at.shift0, t1 = tile * step + at.shift1;
            const bool inside = __all_sync(0xffffffffu, t0 >= 0 && t1 >= 0 && t0 + 8 <= n0 && t1 + 8 <= n1 &&
                                                            ok == (sweep ? 15u : 63u));
            float2 a[8], g[8], x[8];
            ring.get(stage, 0, a);
            ring.get(stage, 1, x);
            if (!inside) {
                ring.fill(a, ok, 0, at.row0(p.gate, p.gate_s) + t0, t0, n0, at.row1(p.gate, p.gate_s) + t1, t1, n1);
                ring.fill(x, ok, 1, at.row0(p.x, p.x_s) + t0, t0, n0, at.row1(p.x, p.x_s) + t1, t1, n1);
            }
            row_gains<kLog>(a, g, bias2, inside, t0, n0, t1, n1);
            float2 A = one, H = zero;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 u = kLog ? x[i] : __fmul2_rn(g[i], x[i]);
                H = i == 0 ? u : __ffma2_rn(a[i], H, u);
                A = i == 0 ? a[0] : __fmul2_rn(A, a[i]);
            }
            float2 B = A;
            team_scan<false>(A, H, at_lane, width);
            if (sweep) {
                const float2 entering = carry;
                if constexpr (kMulti) {
                    if (lane == 31) buf[stage][warp] = make_float4(A.x, A.y, H.x, H.y);
                    __syncthreads();
                    fold_warps<false>(carry, buf[stage] + warp - rank, rank, warps);
                } else {
                    enter_lane<false, true>(A, H, carry, &carry, at_lane, width);
                }
                if (offset == 0) {
                    if (at.live0) states0[tile] = entering.x;
                    if (at.live1) states1[tile] = entering.y;
                }
                continue;
            }
            float2 dd[8];
            ring.get(stage, 2, dd);
            if (!inside)
                ring.fill(dd, ok, 2, at.row0(p.dout, p.out_s) + t0, t0, n0, at.row1(p.dout, p.out_s) + t1, t1, n1);
            float2 R = zero;
#pragma unroll
            for (int i = 7; i >= 0; --i) R = __fmul2_rn(a[i], i == 7 ? dd[7] : __fadd2_rn(dd[i], R));
            team_scan<true>(B, R, at_lane, width);
            float2 h, r;
            if constexpr (kMulti) {
                if (lane == 31) buf[stage][warp] = make_float4(A.x, A.y, H.x, H.y);
                if (lane == 0) back[stage][warp] = make_float4(B.x, B.y, R.x, R.y);
                __syncthreads();                 // also orders the first sweep's states before the reads below
                if (tile + 1 < tiles) carry = make_float2(states0[tile], states1[tile]);
                h = fold_warps<false>(carry, buf[stage] + warp - rank, rank, warps);
                r = fold_warps<true>(r_carry, back[stage] + warp - rank, rank, warps);
                h = enter_lane<false, false>(A, H, h, nullptr, at_lane, width);
                r = enter_lane<true, false>(B, R, r, nullptr, at_lane, width);
            } else {
                __syncwarp();
                if (tile + 1 < tiles) carry = make_float2(states0[tile], states1[tile]);
                h = enter_lane<false, false>(A, H, carry, nullptr, at_lane, width);
                r = enter_lane<true, true>(B, R, r_carry, &r_carry, at_lane, width);
            }
            // x becomes what the decay's gradient multiplies: x_t - h_{t-1}, or h_{t-1}
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 u = kLog ? x[i] : __fmul2_rn(g[i], x[i]);
                x[i] = kLog ? h : __ffma2_rn(h, make_float2(-1.0f, -1.0f), x[i]);
                h = __ffma2_rn(a[i], h, u);
            }
#pragma unroll
            for (int i = 7; i >= 0; --i) {
                const float2 l = __fadd2_rn(dd[i], r);
                r = __fmul2_rn(a[i], l);
                dd[i] = __fmul2_rn(r, x[i]);
                x[i] = l;
                if constexpr (!kLog) {
                    dd[i] = __fmul2_rn(g[i], dd[i]);
                    x[i] = __fmul2_rn(g[i], l);
                }
            }
            if (!inside)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (t0 + i < 0 || t0 + i >= n0) dd[i].x = x[i].x = 0.0f;
                    if (t1 + i < 0 || t1 + i >= n1) dd[i].y = x[i].y = 0.0f;
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) db = __fadd2_rn(db, dd[i]);
            IoT *dgate0 = at.row0(p.dgate, p.dgate_s), *dgate1 = at.row1(p.dgate, p.dgate_s);
            IoT *dx0 = at.row0(p.dx, p.dx_s), *dx1 = at.row1(p.dx, p.dx_s);
            if (__all_sync(0xffffffffu, inside && on16(dgate0 + t0) && on16(dgate1 + t1) && on16(dx0 + t0) && on16(dx1 + t1))) {
                store_pair_rows(dgate0 + t0, dgate1 + t1, dd);
                store_pair_rows(dx0 + t0, dx1 + t1, x);
            } else {
                const int hi0 = at.live0 ? L : 0, hi1 = at.live1 ? L : 0;
                store_steps2(dgate0, t0, 0, hi0, dgate1, t1, 0, hi1, dd);
                store_steps2(dx0, t0, 0, hi0, dx1, t1, 0, hi1, x);
            }
        }
        if (offset == 0) at.put(p.dh0, chain, r_carry);
        if (p.bias_partial != nullptr) {
            for (int o = width / 2; o > 0; o >>= 1)
                db = __fadd2_rn(db, make_float2(__shfl_xor_sync(0xffffffffu, db.x, o, width),
                                                __shfl_xor_sync(0xffffffffu, db.y, o, width)));
            if constexpr (kMulti) {
                if (lane == 0) sums[warp] = db;
                __syncthreads();                 // the next writes follow another tile's barrier
                db = zero;
                for (int v = 0; v < warps; ++v) db = __fadd2_rn(db, sums[warp - rank + v]);
            }
            if (offset == 0) at.put(p.bias_partial, chain, db);
        }
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
// batches, launch latency below (1 x 4096 and 128 x 4096 bf16: 8 us in a replayed
// graph with cold caches, 9 us called from Python).
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
        load_eight(state, h);
        load_eight(gate, f);
        load_eight(x, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) bias[k] = 0.0f;
        if (p.bias != nullptr) load_eight(p.bias + d, bias);
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
