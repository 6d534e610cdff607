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
// Layout (batch, seqlen, dim): a tile is 64 steps x 64 channels; each of 8
// warps takes 8 steps, a lane two neighbouring channels (128- or 256-byte rows
// per warp access).  A warp folds its steps into one map, the CTA composes the
// maps through shared memory, and the tiles of a chain are joined by a
// look-back: a tile publishes its map, then takes the state entering it from
// the nearest earlier tile that knows its own (folding the published maps in
// between), publishes the state that leaves it, and replays its steps from
// registers.  Each input is read once.  Tiles are handed out by a counter, the
// earliest steps of all chains first, so that every tile's predecessors belong
// to CTAs that are running or done; the wait is bounded all the same.
//
// Layout (batch, dim, seqlen): a lane takes 8 consecutive steps of one chain,
// the warp composes its lanes' maps by shuffles, and 1 to 8 warps per chain
// share a tile through shared memory.  Chains are plentiful here (one per
// channel instead of one per 64), so a chain stays with its warps and nothing
// waits.
#pragma once

#include "row_vectors.cuh"

namespace mamba {

constexpr int kGatedSteps = 8;                              // steps per thread
constexpr int kGatedWarps = 8;
constexpr int kGatedTile = kGatedSteps * kGatedWarps;       // 64 steps
constexpr int kGatedChannels = 64;                          // per tile, two per lane
constexpr int kGatedThreads = kGatedWarps * 32;
static_assert(kGatedTile == MAMBA_GATED_CHECKPOINT_STEPS, "checkpoints are the states entering tiles");

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
    float* bias_partial;          // bwd: [batch * tiles][dim] (seqlen fastest: [batch][dim]) or null
    // (batch, seqlen, dim): states entering tiles, [batch][tiles][dim]
    float* enter;                 // fwd: written; bwd: read
    float* carry;                 // bwd: r entering tiles from the right, [batch][tiles][dim]
    float4* maps;                 // [groups][tiles][32]: a lane's two (A, H) pairs
    unsigned int* flags;          // [groups][tiles]: 0, 1 = map published, 2 = state published
    unsigned int* ticket;
    // (batch, dim, seqlen), bwd: states entering tiles, [chains][tiles]
    float* chain_states;
    GatedStrides gate_s, x_s, out_s, dgate_s, dx_s;          // out_s: out, or dout
    int64_t batch, dim, seqlen, chains;
    int64_t tiles;                // per chain
    int64_t groups_per_row;       // 64-channel groups per batch row
    int64_t groups;
    int64_t items;                // groups * tiles
    int withhold;                 // test only: publish nothing
};

constexpr unsigned int kGatedPollLimit = 1u << 19;

// g and a of the sigmoid gate; a = 1 - g to fp32 on both sides.  With
// e = exp(-|f|), small = e / (1 + e) is the smaller of the two and the other is
// 1 - small, rounded to nearest: a decay close to 1 is applied over about 1 / g
// steps, and a biased rounding would grow with that memory.
__device__ __forceinline__ void sigmoid_gate(float f, float& g, float& a) {
    const float e = ex2_approx(-fabsf(f) * kLog2e);
    const float small = __fdividef(e, 1.0f + e);
    const float big = 1.0f - small;
    g = f < 0.0f ? small : big;
    a = f < 0.0f ? big : small;
}

template <bool kLog>
__device__ __forceinline__ void gated_terms(float f, float x, float& a, float& u) {
    if constexpr (kLog) {
        a = exp2_near_one_exact(f * kLog2e);
        u = x;
    } else {
        float g;
        sigmoid_gate(f, g, a);
        u = g * x;
    }
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

// Where a tile lies: item = position * groups + group, positions in the order
// of the scan (kReverse: the last tile of a chain first).
struct GatedTileAt {
    int64_t b, group, tile, t0, d;      // d: this lane's first channel
    int64_t n;                          // the row's length
};

template <bool kReverse>
__device__ __forceinline__ GatedTileAt gated_tile(const GatedParams& p, int64_t item, int lane) {
    GatedTileAt at;
    const int64_t pos = item / p.groups;
    at.group = item - pos * p.groups;
    at.tile = kReverse ? p.tiles - 1 - pos : pos;
    at.b = at.group / p.groups_per_row;
    at.d = (at.group - at.b * p.groups_per_row) * kGatedChannels + 2 * lane;
    at.t0 = at.tile * kGatedTile;
    at.n = gated_length(p, at.b);
    return at;
}

// The state (or r) entering tile `at` of a chain that is scanned from `pos` 0
// on, for this lane's two channels: `own` is what chain position 0 starts from.
// Called by one warp.  Walks back from the tile before: published maps are
// folded until a tile with a published state is met.  state_row(k) is where
// the state that LEAVES position k is kept.
template <bool kVec, typename StateAt>
__device__ __forceinline__ float2 gated_look_back(const GatedParams& p, int64_t group, int64_t pos,
                                                  int lane, bool c0, bool c1, StateAt state_at) {
    const unsigned int* flags = p.flags + group * p.tiles;
    const float4* maps = p.maps + (group * p.tiles) * 32 + lane;
    float2 A = make_float2(1.0f, 1.0f), H = make_float2(0.0f, 0.0f);
    int64_t next = pos - 1;               // nearest position not folded yet
    for (unsigned int poll = 0; poll < kGatedPollLimit; ++poll) {
        const int64_t k = next - lane;
        const unsigned int f = k >= 0 ? load_acquire(flags + k) : 2u;
        const unsigned int known = __ballot_sync(0xffffffffu, f == 2u);
        const unsigned int missing = __ballot_sync(0xffffffffu, f == 0u);
        // fold the run of published maps before the first known state or gap
        const int stop = known ? __ffs(known) - 1 : 32;
        const int gap = missing ? __ffs(missing) - 1 : 32;
        const int run = stop < gap ? stop : gap;
        if (run > 0 && (stop < gap || run >= 8)) {
            for (int j = 0; j < run; ++j) {
                const float4 m = __ldcg(maps + (next - j) * 32);
                H.x = fmaf(A.x, m.y, H.x);
                H.y = fmaf(A.y, m.w, H.y);
                A.x *= m.x;
                A.y *= m.z;
            }
            next -= run;
        }
        if (stop < gap) {                 // position `next` has published its state
            const float2 h = load_f2<kVec>(state_at(next), c0, c1);
            return make_float2(fmaf(A.x, h.x, H.x), fmaf(A.y, h.y, H.y));
        }
    }
    if (lane == 0) record_device_error(MAMBA_ERR_TIMEOUT);
    return make_float2(0.0f, 0.0f);
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

// Forward.  Shared memory holds the warps' maps and the entering state.
template <typename IoT, bool kLog, bool kVec>
__global__ void __launch_bounds__(kGatedThreads, 2)
    gated_scan_fwd_kernel(const __grid_constant__ GatedParams p) {
    __shared__ float4 maps[kGatedWarps][32];
    __shared__ float2 entering[32];
    __shared__ int64_t first_item, next_item;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool dynamic = p.ticket != nullptr;
    if (threadIdx.x == 0) first_item = dynamic ? (int64_t)atomicAdd(p.ticket, 1u) : (int64_t)blockIdx.x;
    __syncthreads();
    int64_t item = first_item;
    Pair<IoT> rf[kGatedSteps], rx[kGatedSteps];

    auto request = [&](int64_t it) {
        const GatedTileAt at = gated_tile<false>(p, it, lane);
        const bool c0 = at.d < p.dim, c1 = at.d + 1 < p.dim;
        const int64_t t = at.t0 + warp * kGatedSteps;
        const IoT* gate = static_cast<const IoT*>(p.gate) + at.b * p.gate_s.batch + t * p.gate_s.row + at.d;
        const IoT* x = static_cast<const IoT*>(p.x) + at.b * p.x_s.batch + t * p.x_s.row + at.d;
#pragma unroll
        for (int i = 0; i < kGatedSteps; ++i) {
            const bool in = t + i < at.n;
            rf[i] = load_pair<IoT, kVec>(gate + i * p.gate_s.row, in && c0, in && c1);
            rx[i] = load_pair<IoT, kVec>(x + i * p.x_s.row, in && c0, in && c1);
        }
    };
    if (item < p.items) request(item);

    while (item < p.items) {
        const GatedTileAt at = gated_tile<false>(p, item, lane);
        const bool c0 = at.d < p.dim, c1 = at.d + 1 < p.dim;
        const int64_t t = at.t0 + warp * kGatedSteps;
        const float2 bias = p.bias != nullptr ? load_f2<kVec>(p.bias + at.d, c0, c1) : make_float2(0.0f, 0.0f);
        float2 a[kGatedSteps], u[kGatedSteps];
        float2 A = make_float2(1.0f, 1.0f), H = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kGatedSteps; ++i) {
            const float2 f = rf[i].get(), x = rx[i].get();
            gated_terms<kLog>(f.x + bias.x, x.x, a[i].x, u[i].x);
            gated_terms<kLog>(f.y + bias.y, x.y, a[i].y, u[i].y);
            if (t + i >= at.n) {
                a[i] = make_float2(1.0f, 1.0f);
                u[i] = make_float2(0.0f, 0.0f);
            }
            H.x = fmaf(a[i].x, H.x, u[i].x);
            H.y = fmaf(a[i].y, H.y, u[i].y);
            A.x *= a[i].x;
            A.y *= a[i].y;
        }
        maps[warp][lane] = make_float4(A.x, H.x, A.y, H.y);
        if (threadIdx.x == 0)
            next_item = dynamic ? (int64_t)atomicAdd(p.ticket, 1u) : item + gridDim.x;
        __syncthreads();
        const int64_t following = next_item;
        if (following < p.items) request(following);

        // the map of the warps before this one (warp 0: of the whole tile)
        float2 Ap = make_float2(1.0f, 1.0f), Hp = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < kGatedWarps; ++v)
            if (v < warp || warp == 0) {
                const float4 m = maps[v][lane];
                Hp.x = fmaf(m.x, Hp.x, m.y);
                Hp.y = fmaf(m.z, Hp.y, m.w);
                Ap.x *= m.x;
                Ap.y *= m.z;
            }
        float* enter = p.enter != nullptr ? p.enter + (at.b * p.tiles + at.tile) * p.dim + at.d : nullptr;
        if (warp == 0) {
            float2 h;
            unsigned int* flag = p.flags + at.group * p.tiles + at.tile;
            if (at.tile == 0) {
                h = p.h0 != nullptr ? load_f2<kVec>(p.h0 + at.b * p.dim + at.d, c0, c1) : make_float2(0.0f, 0.0f);
                if (enter != nullptr) store_f2<kVec>(enter, c0, c1, h);
            } else {
                __stcg(p.maps + (at.group * p.tiles + at.tile) * 32 + lane,
                       make_float4(Ap.x, Hp.x, Ap.y, Hp.y));
                gated_publish(p, flag, lane, 1u);
                // the state leaving tile k is the one entering tile k + 1
                const float* base = p.enter + (at.b * p.tiles + 1) * p.dim + at.d;
                const int64_t dim = p.dim;
                h = gated_look_back<kVec>(p, at.group, at.tile, lane, c0, c1,
                                          [base, dim](int64_t k) { return base + k * dim; });
            }
            const float2 leave = make_float2(fmaf(Ap.x, h.x, Hp.x), fmaf(Ap.y, h.y, Hp.y));
            if (at.tile + 1 < p.tiles) {
                store_f2<kVec>(enter + p.dim, c0, c1, leave);
                gated_publish(p, flag, lane, 2u);
            } else if (p.last != nullptr) {
                store_f2<kVec>(p.last + at.b * p.dim + at.d, c0, c1, leave);
            }
            entering[lane] = h;
            Ap = make_float2(1.0f, 1.0f);
            Hp = make_float2(0.0f, 0.0f);
        }
        __syncthreads();
        const float2 h_in = entering[lane];
        if (p.out != nullptr) {
            float2 h = make_float2(fmaf(Ap.x, h_in.x, Hp.x), fmaf(Ap.y, h_in.y, Hp.y));
            IoT* out = static_cast<IoT*>(p.out) + at.b * p.out_s.batch + t * p.out_s.row + at.d;
#pragma unroll
            for (int i = 0; i < kGatedSteps; ++i) {
                h.x = fmaf(a[i].x, h.x, u[i].x);
                h.y = fmaf(a[i].y, h.y, u[i].y);
                if (t + i < p.seqlen)
                    store_pair<IoT, kVec>(out + i * p.out_s.row, c0, c1,
                                          t + i < at.n ? h : make_float2(0.0f, 0.0f));
            }
        }
        item = following;
    }
}

// Backward.  r runs from the last tile to the first; the states of a tile are
// replayed from the state entering it.
template <typename IoT, bool kLog, bool kVec>
__global__ void __launch_bounds__(kGatedThreads, 2)
    gated_scan_bwd_kernel(const __grid_constant__ GatedParams p) {
    __shared__ float4 maps[kGatedWarps][32];            // (A, H) of the warps' steps
    __shared__ float2 rights[kGatedWarps][32];          // R: r leaving a warp's steps when 0 enters
    __shared__ float2 entering[32];
    __shared__ float2 bias_sums[kGatedWarps][32];
    __shared__ int64_t first_item, next_item;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool dynamic = p.ticket != nullptr;
    if (threadIdx.x == 0) first_item = dynamic ? (int64_t)atomicAdd(p.ticket, 1u) : (int64_t)blockIdx.x;
    __syncthreads();
    int64_t item = first_item;
    Pair<IoT> rf[kGatedSteps], rx[kGatedSteps], rd[kGatedSteps];
    float2 enter = make_float2(0.0f, 0.0f);

    auto request = [&](int64_t it) {
        const GatedTileAt at = gated_tile<true>(p, it, lane);
        const bool c0 = at.d < p.dim, c1 = at.d + 1 < p.dim;
        const int64_t t = at.t0 + warp * kGatedSteps;
        const IoT* gate = static_cast<const IoT*>(p.gate) + at.b * p.gate_s.batch + t * p.gate_s.row + at.d;
        const IoT* x = static_cast<const IoT*>(p.x) + at.b * p.x_s.batch + t * p.x_s.row + at.d;
        const IoT* dout = static_cast<const IoT*>(p.dout) + at.b * p.out_s.batch + t * p.out_s.row + at.d;
#pragma unroll
        for (int i = 0; i < kGatedSteps; ++i) {
            const bool in = t + i < at.n;
            rf[i] = load_pair<IoT, kVec>(gate + i * p.gate_s.row, in && c0, in && c1);
            rx[i] = load_pair<IoT, kVec>(x + i * p.x_s.row, in && c0, in && c1);
            rd[i] = load_pair<IoT, kVec>(dout + i * p.out_s.row, in && c0, in && c1);
        }
        enter = load_f2<kVec>(p.enter + (at.b * p.tiles + at.tile) * p.dim + at.d, c0, c1);
    };
    if (item < p.items) request(item);

    while (item < p.items) {
        const GatedTileAt at = gated_tile<true>(p, item, lane);
        const bool c0 = at.d < p.dim, c1 = at.d + 1 < p.dim;
        const int64_t t = at.t0 + warp * kGatedSteps;
        const float2 bias = p.bias != nullptr ? load_f2<kVec>(p.bias + at.d, c0, c1) : make_float2(0.0f, 0.0f);
        float2 a[kGatedSteps], g[kGatedSteps], x[kGatedSteps], dd[kGatedSteps];
        float2 A = make_float2(1.0f, 1.0f), H = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kGatedSteps; ++i) {
            const float2 f = rf[i].get();
            x[i] = rx[i].get();
            dd[i] = rd[i].get();
            if constexpr (kLog) {
                a[i].x = exp2_near_one_exact((f.x + bias.x) * kLog2e);
                a[i].y = exp2_near_one_exact((f.y + bias.y) * kLog2e);
                g[i] = make_float2(1.0f, 1.0f);
            } else {
                sigmoid_gate(f.x + bias.x, g[i].x, a[i].x);
                sigmoid_gate(f.y + bias.y, g[i].y, a[i].y);
            }
            if (t + i >= at.n) {          // outside: x and dout were not read and are 0
                a[i] = make_float2(1.0f, 1.0f);
                g[i] = make_float2(0.0f, 0.0f);
            }
            H.x = fmaf(a[i].x, H.x, g[i].x * x[i].x);
            H.y = fmaf(a[i].y, H.y, g[i].y * x[i].y);
            A.x *= a[i].x;
            A.y *= a[i].y;
        }
        float2 R = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = kGatedSteps - 1; i >= 0; --i) {
            R.x = a[i].x * (dd[i].x + R.x);
            R.y = a[i].y * (dd[i].y + R.y);
        }
        maps[warp][lane] = make_float4(A.x, H.x, A.y, H.y);
        rights[warp][lane] = R;
        if (threadIdx.x == 0)
            next_item = dynamic ? (int64_t)atomicAdd(p.ticket, 1u) : item + gridDim.x;
        __syncthreads();
        const int64_t following = next_item;
        // states: from the tile's entry through the warps before this one
        float2 h = enter;
#pragma unroll
        for (int v = 0; v < kGatedWarps - 1; ++v)
            if (v < warp) {
                const float4 m = maps[v][lane];
                h.x = fmaf(m.x, h.x, m.y);
                h.y = fmaf(m.z, h.y, m.w);
            }
        // r: the map of the warps after this one (last warp: of the whole tile)
        constexpr int kLast = kGatedWarps - 1;
        float2 Ap = make_float2(1.0f, 1.0f), Rp = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = kLast; v >= 0; --v)
            if (v > warp || warp == kLast) {
                const float4 m = maps[v][lane];
                const float2 r = rights[v][lane];
                Rp.x = fmaf(m.x, Rp.x, r.x);
                Rp.y = fmaf(m.z, Rp.y, r.y);
                Ap.x *= m.x;
                Ap.y *= m.z;
            }
        if (following < p.items) request(following);
        if (warp == kLast) {
            float2 r;
            const int64_t pos = p.tiles - 1 - at.tile;
            unsigned int* flag = p.flags + at.group * p.tiles + pos;
            float* carry = p.carry + (at.b * p.tiles + at.tile) * p.dim + at.d;   // r leaving this tile
            if (pos == 0) {
                r = p.dlast != nullptr ? load_f2<kVec>(p.dlast + at.b * p.dim + at.d, c0, c1)
                                       : make_float2(0.0f, 0.0f);
            } else {
                __stcg(p.maps + (at.group * p.tiles + pos) * 32 + lane,
                       make_float4(Ap.x, Rp.x, Ap.y, Rp.y));
                gated_publish(p, flag, lane, 1u);
                const float* base = p.carry + (at.b * p.tiles + p.tiles - 1) * p.dim + at.d;
                const int64_t dim = p.dim;
                r = gated_look_back<kVec>(p, at.group, pos, lane, c0, c1,
                                          [base, dim](int64_t k) { return base - k * dim; });
            }
            const float2 leave = make_float2(fmaf(Ap.x, r.x, Rp.x), fmaf(Ap.y, r.y, Rp.y));
            if (at.tile > 0) {
                store_f2<kVec>(carry, c0, c1, leave);
                gated_publish(p, flag, lane, 2u);
            } else if (p.dh0 != nullptr) {
                store_f2<kVec>(p.dh0 + at.b * p.dim + at.d, c0, c1, leave);
            }
            entering[lane] = r;
            Ap = make_float2(1.0f, 1.0f);
            Rp = make_float2(0.0f, 0.0f);
        }
        // replay the states while the last warp looks back
        float2 before[kGatedSteps];
#pragma unroll
        for (int i = 0; i < kGatedSteps; ++i) {
            before[i] = h;
            h.x = fmaf(a[i].x, h.x, g[i].x * x[i].x);
            h.y = fmaf(a[i].y, h.y, g[i].y * x[i].y);
        }
        __syncthreads();
        const float2 r_in = entering[lane];
        float2 r = make_float2(fmaf(Ap.x, r_in.x, Rp.x), fmaf(Ap.y, r_in.y, Rp.y));
        float2 db = make_float2(0.0f, 0.0f);
        IoT* dgate = static_cast<IoT*>(p.dgate) + at.b * p.dgate_s.batch + t * p.dgate_s.row + at.d;
        IoT* dx = static_cast<IoT*>(p.dx) + at.b * p.dx_s.batch + t * p.dx_s.row + at.d;
#pragma unroll
        for (int i = kGatedSteps - 1; i >= 0; --i) {
            const float2 l = make_float2(dd[i].x + r.x, dd[i].y + r.y);
            r.x = a[i].x * l.x;
            r.y = a[i].y * l.y;
            float2 df, dv;
            if constexpr (kLog) {
                df = make_float2(r.x * before[i].x, r.y * before[i].y);
                dv = l;
            } else {
                dv = make_float2(g[i].x * l.x, g[i].y * l.y);
                df.x = g[i].x * r.x * (x[i].x - before[i].x);
                df.y = g[i].y * r.y * (x[i].y - before[i].y);
            }
            if (t + i >= at.n) df = dv = make_float2(0.0f, 0.0f);
            db.x += df.x;
            db.y += df.y;
            if (t + i < p.seqlen) {
                store_pair<IoT, kVec>(dgate + i * p.dgate_s.row, c0, c1, df);
                store_pair<IoT, kVec>(dx + i * p.dx_s.row, c0, c1, dv);
            }
        }
        if (p.bias_partial != nullptr) {
            bias_sums[warp][lane] = db;
            __syncthreads();
            if (warp == 0) {
                float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int v = 0; v < kGatedWarps; ++v) {
                    sum.x += bias_sums[v][lane].x;
                    sum.y += bias_sums[v][lane].y;
                }
                store_f2<kVec>(p.bias_partial + (at.b * p.tiles + at.tile) * p.dim + at.d, c0, c1, sum);
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
            gated_terms<kLog>(a[i] + bias, x8[i], a[i], u[i]);
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
            gated_terms<kLog>(f[i] + bias, x8[i], a, u);
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
            if constexpr (kLog) {
                a[i] = exp2_near_one_exact((a[i] + bias) * kLog2e);
                g[i] = 1.0f;
            } else {
                sigmoid_gate(a[i] + bias, g[i], a[i]);
            }
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
            gated_terms<kLog>(f[k] + bias[k], v[k], a, u);
            h[k] = fmaf(a, h[k], u);
        }
        store_steps(state, 0, 0, 8, h);
        store_steps(out, 0, 0, 8, h);
    } else {
        float a, u;
        gated_terms<kLog>(DType<IoT>::load(gate) + (p.bias != nullptr ? p.bias[d] : 0.0f),
                          DType<IoT>::load(x), a, u);
        const float h = fmaf(a, *state, u);
        *state = h;
        DType<IoT>::store(out, h);
    }
}

}  // namespace mamba
