// Gated linear recurrence, (batch, seqlen, dim), for many chains (sm_100a).
//
// The definitions are those of gated_scan.cuh.  With enough groups of 64
// channels to occupy the GPU, a CTA walks a stretch of one group tile by tile
// and carries the state along, so every step's arithmetic is done once.  A tile
// is 64 steps x 64 channels; a producer warp brings tiles into a ring in shared
// memory by TMA (gate and x; dout as well in the backward), eight warps take 8
// steps each, two channels per lane.  A warp folds its steps into one affine
// map, the maps are exchanged through shared memory (one barrier per tile),
// and the warp replays its steps from registers, writes its results over its
// inputs in the ring, and sends its 8 rows out by TMA.
//
// A chain is cut into stretches, handed out by a counter (the earliest of all
// chains first, in the order of the scan), so that the last wave of CTAs is
// short; a stretch starts from the state that its predecessor published, which
// belongs to a CTA that is running or done.  Every wait is bounded; one that
// runs out is recorded and the call ends with undefined outputs.
//
// Measured, sigmoid gate (copy rate 6529 GB/s): bf16 8 x 2048 x 4096 (batch, seqlen,
// dim) forward 94 us, 4.28 TB/s, 66 %, backward from checkpoints 168 us, 4.02 TB/s,
// 62 %; 16 x 2048 x 5120 forward 188 us, 82 %; fp32 4 x 2048 x 4096 82 and 154 us,
// 75 and 67 %.  Neither memory nor the issue slots are full (8 x 1024 x 4096: DRAM 42
// and 43 % of its peak, 58 % of the issue slots forward at 25 instructions per
// element, 53 % backward at 45).  The warps stall on long-latency results first (2.7
// cycles per instruction forward; the polls of a hand-off count there) and on fixed
// latencies; all eight meet at a barrier in every tile, between its maps and its
// results.  Rounds of CTAs count too: 8 x 2048 x 4096 gives 1536 stretches to 444
// places for CTAs forward, 3.5 rounds; 16 x 2048 x 5120 gives 2.9, better filled.
#pragma once

#include "gated_scan.cuh"

namespace mamba {

constexpr int kChainSteps = 8;                              // per warp and tile
constexpr int kChainWarps = 8;                              // besides the producer
constexpr int kChainTile = kChainSteps * kChainWarps;
constexpr int kChainChannels = 64;
constexpr int kChainThreads = (kChainWarps + 1) * 32;
static_assert(kChainTile == MAMBA_GATED_CHECKPOINT_STEPS, "checkpoints are the states entering tiles");

struct ChainParams {
    CUtensorMap gate, x, dout;     // loads: boxes of 64 channels x 64 steps
    CUtensorMap states;            // bwd: the states entering tiles, 64 channels of one tile
    CUtensorMap out0, out1;        // stores: 64 channels x 8 steps; out, or dgate and dx
    const float* bias;             // (dim) or null
    const float* h0;               // (batch, dim) or null
    const float* dlast;            // bwd, (batch, dim) or null
    const int32_t* seqlens;        // (batch) or null
    float* last;                   // fwd: last state; bwd: gradient of the initial state; or null
    float* enter;                  // fwd, [batch][tiles][dim] or null
    float* bias_partial;           // bwd: [batch * stretches][dim] or null
    float* handoff;                // [groups][stretches][64]
    unsigned int* flags;           // [groups][stretches]
    unsigned int* ticket;
    unsigned int* failed;          // 0, or 1 once a wait of this call has run out
    int64_t dim, seqlen;
    int64_t tiles;                 // per chain
    int64_t groups_per_row, groups;
    int64_t stretch_tiles, stretches;
    int64_t items;                 // groups * stretches
    int withhold;
};

template <typename IoT, bool kBackward>
struct ChainSizes {
    static constexpr int kTensor = kChainTile * kChainChannels * (int)sizeof(IoT);     // bytes of a tile
    static constexpr int kStage = kBackward ? 3 * kTensor + kChainChannels * 4 : 2 * kTensor;   // + entering states
    // stages of the ring: two or three CTAs share an SM's shared memory
    static constexpr int kStages = sizeof(IoT) == 2 ? 3 : (kBackward ? 2 : 3);
};

// What the producer says about the tile in a stage.
struct alignas(16) ChainTile {
    int group, b, tile, position;          // position: stretch in scan order
    int d0;                                // first channel of the group
    int rows_left;                         // steps of the sequence in the tile
    int edge;                              // kChainFirst, kChainLast: of its stretch, in scan order
    int stop;                              // no tile: the CTA is done
};
constexpr int kChainFirst = 1, kChainLast = 2;

template <typename IoT, bool kBackward>
struct ChainShared {
    static constexpr int kStages = ChainSizes<IoT, kBackward>::kStages;
    alignas(128) unsigned char ring[kStages][ChainSizes<IoT, kBackward>::kStage];
    float4 maps[2][kChainWarps][32];               // (A, H) of a lane's two channels, by tile parity
    float2 rights[kBackward ? 2 : 1][kChainWarps][32];
    ChainTile tile[kStages];
    uint64_t full[kStages], empty[kStages];
    int failed;
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int c0, int c1, int c2, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
}

// Asks L2 for a box that a later load will fetch.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// Bounded wait on an mbarrier; false when it ran out, or at once after another did.
__device__ __forceinline__ bool chain_wait(uint64_t* bar, uint32_t parity, volatile int* failed) {
    const uint32_t b = smem_u32(bar);
    for (uint32_t i = 0; i < kMaxWaitPolls; ++i) {
        if (mbar_try_wait(b, parity)) return true;
        if (*failed) return false;
    }
    *failed = 1;
    record_device_error(MAMBA_ERR_TIMEOUT);
    return false;
}

template <typename IoT>
__device__ __forceinline__ float2 ring_get(const unsigned char* row, int lane) {
    if constexpr (sizeof(IoT) == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(row + 4 * lane);
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        return *reinterpret_cast<const float2*>(row + 8 * lane);
    }
}

template <typename IoT>
__device__ __forceinline__ void ring_put(unsigned char* row, int lane, float2 v) {
    if constexpr (sizeof(IoT) == 2) *reinterpret_cast<uint32_t*>(row + 4 * lane) = pack_bf16x2(v.x, v.y);
    else *reinterpret_cast<float2*>(row + 8 * lane) = v;
}

__device__ __forceinline__ float2 chain_load2(const float* p, int64_t d, int64_t dim) {
    return make_float2(d < dim ? load_ordered(p + d) : 0.0f, d + 1 < dim ? load_ordered(p + d + 1) : 0.0f);
}

__device__ __forceinline__ void chain_store2(float* p, int64_t d, int64_t dim, float2 v) {
    if (d < dim) p[d] = v.x;
    if (d + 1 < dim) p[d + 1] = v.y;
}

// The producer warp: takes stretches and requests their tiles in scan order.
template <typename IoT, bool kBackward>
__device__ __forceinline__ void chain_produce(const ChainParams& p, ChainShared<IoT, kBackward>& sh, int lane) {
    constexpr int kStages = ChainShared<IoT, kBackward>::kStages;
    constexpr int kBytes = ChainSizes<IoT, kBackward>::kTensor;
    if (lane != 0) return;
    int64_t n = 0;                                 // stages handed over
    auto next_stage = [&](int* s) -> bool {
        *s = (int)(n % kStages);
        return n < kStages || chain_wait(&sh.empty[*s], (uint32_t)((n / kStages - 1) & 1), &sh.failed);
    };
    bool ok = true;
    while (ok) {
        const int64_t item = p.ticket != nullptr ? (int64_t)atomicAdd(p.ticket, 1u)
                                                 : (n == 0 ? (int64_t)blockIdx.x : p.items);
        if (item >= p.items) break;
        ChainTile at;
        at.position = (int)(item / p.groups);
        at.group = (int)(item - at.position * p.groups);
        at.b = (int)(at.group / p.groups_per_row);
        at.d0 = (int)(at.group - at.b * p.groups_per_row) * kChainChannels;
        at.stop = 0;
        const int64_t len = p.seqlens != nullptr ? min(max((int64_t)p.seqlens[at.b], (int64_t)0), p.seqlen) : p.seqlen;
        const int64_t stretch = kBackward ? p.stretches - 1 - at.position : at.position;
        const int64_t begin = stretch * p.stretch_tiles, end = min(begin + p.stretch_tiles, p.tiles);
        for (int64_t k = 0; ok && k < end - begin; ++k) {
            const int64_t tile = kBackward ? end - 1 - k : begin + k;
            int s;
            ok = next_stage(&s);
            if (!ok) break;
            ++n;
            const int t = (int)(tile * kChainTile);
            at.tile = (int)tile;
            const int64_t left = len - t;
            at.rows_left = (int)(left > kChainTile ? kChainTile : (left < 0 ? 0 : left));
            at.edge = (k == 0 ? kChainFirst : 0) | (k == end - begin - 1 ? kChainLast : 0);
            sh.tile[s] = at;
            const uint32_t bar = smem_u32(&sh.full[s]), dst = smem_u32(sh.ring[s]);
            mbar_arrive_expect_tx(bar, (ChainSizes<IoT, kBackward>::kStage));
            tma_load_3d(dst, &p.gate, at.d0, t, at.b, bar);
            tma_load_3d(dst + kBytes, &p.x, at.d0, t, at.b, bar);
            if constexpr (kBackward) {
                tma_load_3d(dst + 2 * kBytes, &p.dout, at.d0, t, at.b, bar);
                tma_load_3d(dst + 3 * kBytes, &p.states, at.d0, at.tile, at.b, bar);
            }
        }
    }
    int s;
    if (ok && next_stage(&s)) {
        sh.tile[s].stop = 1;
        mbar_arrive(smem_u32(&sh.full[s]));
        return;
    }
    // Given up: the tiles under way still have to land before the CTA ends.
    for (int64_t k = n > kStages ? n - kStages : 0; k < n; ++k)
        mbar_wait_bounded(smem_u32(&sh.full[k % kStages]), (uint32_t)((k / kStages) & 1));
}

// The state that the stretch before this one left, for a lane's two channels.
__device__ __forceinline__ bool chain_receive(const ChainParams& p, const ChainTile& at, int lane,
                                              volatile int* failed, float2* h) {
    const int64_t k = (int64_t)at.group * p.stretches + at.position - 1;
    unsigned int poll = 0;
    while (load_acquire(p.flags + k) == 0u) {
        if (*failed) return false;
        if (gated_look(poll) && load_acquire(p.failed) != 0u) {
            *failed = 1;
            return false;
        }
        if (++poll == kGatedPollLimit) {
            *failed = 1;
            gated_give_up(p.failed);
            return false;
        }
    }
    *h = load_ordered(reinterpret_cast<const float2*>(p.handoff + k * kChainChannels) + lane);
    return true;
}

__device__ __forceinline__ void chain_send(const ChainParams& p, const ChainTile& at, int lane, float2 h) {
    const int64_t k = (int64_t)at.group * p.stretches + at.position;
    __stcg(reinterpret_cast<float2*>(p.handoff + k * kChainChannels) + lane, h);
    __syncwarp();
    if (lane == 0 && !p.withhold) {
        __threadfence();
        store_release(p.flags + k, 1u);
    }
}

template <typename IoT, bool kBackward>
__device__ __forceinline__ void chain_setup(ChainShared<IoT, kBackward>& sh) {
    constexpr int kStages = ChainShared<IoT, kBackward>::kStages;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), kChainWarps);
        }
        sh.failed = 0;
        fence_mbar_init();
    }
    __syncthreads();
}

// Barriers of the eight computing warps (the producer runs by itself).  The
// second also tells every warp whether any of them wants to leave.
__device__ __forceinline__ void chain_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kChainWarps * 32) : "memory");
}

__device__ __forceinline__ bool chain_sync_any(bool leave) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)leave), "n"(kChainWarps * 32)
        : "memory");
    return any != 0;
}

// After a warp has written its rows over the ring: send them, and give the
// stage used one tile earlier back once its rows have been read.
template <int kStores>
__device__ __forceinline__ void chain_send_rows(const CUtensorMap* map0, const CUtensorMap* map1, uint32_t src0,
                                                uint32_t src1, int d0, int t, int b, int lane, bool inside,
                                                uint64_t* previous_empty) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (inside) {
            tma_store_3d(map0, d0, t, b, src0);
            if constexpr (kStores == 2) tma_store_3d(map1, d0, t, b, src1);
        }
        bulk_commit();
        if (previous_empty != nullptr) {
            bulk_wait_read<1>();
            mbar_arrive(smem_u32(previous_empty));
        }
    }
}

template <typename IoT, bool kLog>
__global__ void __launch_bounds__(kChainThreads, sizeof(IoT) == 2 ? 3 : 2)
    gated_chain_fwd_kernel(const __grid_constant__ ChainParams p) {
    extern __shared__ __align__(128) unsigned char raw[];
    auto& sh = *reinterpret_cast<ChainShared<IoT, false>*>(raw);
    constexpr int kStages = ChainShared<IoT, false>::kStages;
    constexpr int kBytes = ChainSizes<IoT, false>::kTensor;
    constexpr int kRow = kChainChannels * (int)sizeof(IoT);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2 one = make_float2(1.0f, 1.0f), zero = make_float2(0.0f, 0.0f);
    chain_setup(sh);
    if (warp == kChainWarps) {
        chain_produce<IoT, false>(p, sh, lane);
        return;
    }
    float2 carry = zero, bias2 = zero;
    uint64_t* previous = nullptr;
    int s = kStages - 1;
    uint32_t turn = 1;                                  // parity of the ring's current round
    for (int n = 0;; n ^= 1) {                          // n: tile parity
        if (++s == kStages) {
            s = 0;
            turn ^= 1;
        }
        bool leave = !chain_wait(&sh.full[s], turn, &sh.failed);
        const ChainTile at = sh.tile[s];
        leave = leave || at.stop;
        const int64_t d = leave ? p.dim : (int64_t)(at.d0 + 2 * lane);
        if (!leave && (at.edge & kChainFirst)) {
            bias2 = p.bias != nullptr ? __fmul2_rn(chain_load2(p.bias, d, p.dim), make_float2(kLog2e, kLog2e)) : zero;
            if (at.position == 0) carry = p.h0 != nullptr ? chain_load2(p.h0 + at.b * p.dim, d, p.dim) : zero;
            else leave = !chain_receive(p, at, lane, &sh.failed, &carry);
        }
        const int left = at.rows_left - warp * kChainSteps;
        unsigned char* grow = sh.ring[s] + warp * kChainSteps * kRow;
        unsigned char* xrow = grow + kBytes;
        float2 a[kChainSteps], u[kChainSteps];
#pragma unroll
        for (int i = 0; i < kChainSteps; ++i)
            gated_terms2<kLog>(ring_get<IoT>(grow + i * kRow, lane), bias2, ring_get<IoT>(xrow + i * kRow, lane), a[i], u[i]);
        if (left < kChainSteps)
#pragma unroll
            for (int i = 0; i < kChainSteps; ++i)
                if (i >= left) {
                    a[i] = one;
                    u[i] = zero;
                }
        float2 A = a[0], H = u[0];
#pragma unroll
        for (int i = 1; i < kChainSteps; ++i) {
            H = __ffma2_rn(a[i], H, u[i]);
            A = __fmul2_rn(A, a[i]);
        }
        float4 (&maps)[kChainWarps][32] = sh.maps[n];
        maps[warp][lane] = make_float4(A.x, A.y, H.x, H.y);
        if (chain_sync_any(leave)) break;
        float2 h = carry;
        if (warp == 0 && p.enter != nullptr)
            chain_store2(p.enter + ((int64_t)at.b * p.tiles + at.tile) * p.dim, d, p.dim, carry);
#pragma unroll
        for (int v = 0; v < kChainWarps; ++v) {
            if (v == warp) h = carry;
            const float4 m = maps[v][lane];
            carry = __ffma2_rn(make_float2(m.x, m.y), carry, make_float2(m.z, m.w));
        }
        if (warp == 0 && (at.edge & kChainLast)) {
            if (at.position + 1 < p.stretches) chain_send(p, at, lane, carry);
            else if (p.last != nullptr) chain_store2(p.last + at.b * p.dim, d, p.dim, carry);
        }
#pragma unroll
        for (int i = 0; i < kChainSteps; ++i) {
            h = __ffma2_rn(a[i], h, u[i]);
            ring_put<IoT>(xrow + i * kRow, lane, h);
        }
        if (left < kChainSteps)
#pragma unroll
            for (int i = 0; i < kChainSteps; ++i)
                if (i >= left) ring_put<IoT>(xrow + i * kRow, lane, zero);
        const int t = at.tile * kChainTile + warp * kChainSteps;
        chain_send_rows<1>(&p.out0, nullptr, smem_u32(xrow), 0, at.d0, t, at.b, lane, t < p.seqlen, previous);
        previous = &sh.empty[s];
    }
    if (lane == 0) bulk_wait_read<0>();
}

template <typename IoT, bool kLog>
__global__ void __launch_bounds__(kChainThreads, 2)
    gated_chain_bwd_kernel(const __grid_constant__ ChainParams p) {
    extern __shared__ __align__(128) unsigned char raw[];
    auto& sh = *reinterpret_cast<ChainShared<IoT, true>*>(raw);
    constexpr int kStages = ChainShared<IoT, true>::kStages;
    constexpr int kBytes = ChainSizes<IoT, true>::kTensor;
    constexpr int kRow = kChainChannels * (int)sizeof(IoT);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2 one = make_float2(1.0f, 1.0f), zero = make_float2(0.0f, 0.0f);
    chain_setup(sh);
    if (warp == kChainWarps) {
        chain_produce<IoT, true>(p, sh, lane);
        return;
    }
    float2 carry = zero, bias2 = zero, db = zero;        // carry: r entering from the right
    uint64_t* previous = nullptr;
    int s = kStages - 1;
    uint32_t turn = 1;                                  // parity of the ring's current round
    for (int n = 0;; n ^= 1) {                          // n: tile parity
        if (++s == kStages) {
            s = 0;
            turn ^= 1;
        }
        bool leave = !chain_wait(&sh.full[s], turn, &sh.failed);
        const ChainTile at = sh.tile[s];
        leave = leave || at.stop;
        const int64_t d = leave ? p.dim : (int64_t)(at.d0 + 2 * lane);
        if (!leave && (at.edge & kChainFirst)) {
            bias2 = p.bias != nullptr ? __fmul2_rn(chain_load2(p.bias, d, p.dim), make_float2(kLog2e, kLog2e)) : zero;
            if (at.position == 0) carry = p.dlast != nullptr ? chain_load2(p.dlast + at.b * p.dim, d, p.dim) : zero;
            else leave = !chain_receive(p, at, lane, &sh.failed, &carry);
            db = zero;
        }
        const int left = at.rows_left - warp * kChainSteps;
        unsigned char* grow = sh.ring[s] + warp * kChainSteps * kRow;
        unsigned char* xrow = grow + kBytes;
        const unsigned char* drow = xrow + kBytes;
        float2 a[kChainSteps], g[kChainSteps];
#pragma unroll
        for (int i = 0; i < kChainSteps; ++i)
            gated_gains2<kLog>(ring_get<IoT>(grow + i * kRow, lane), bias2, g[i], a[i]);
        float2 x[kChainSteps];
#pragma unroll
        for (int i = 0; i < kChainSteps; ++i) x[i] = ring_get<IoT>(xrow + i * kRow, lane);
        if (left < kChainSteps)
#pragma unroll
            for (int i = 0; i < kChainSteps; ++i)
                if (i >= left) {
                    a[i] = one;
                    x[i] = zero;
                }
        // dout, read twice from the ring: registers are short
        auto dout_at = [&](int i) {
            const float2 v = ring_get<IoT>(drow + i * kRow, lane);
            return left < kChainSteps && i >= left ? zero : v;
        };
        float2 A = one, H = zero, R = zero;
#pragma unroll
        for (int i = 0; i < kChainSteps; ++i) {
            H = __ffma2_rn(a[i], H, kLog ? x[i] : __fmul2_rn(g[i], x[i]));
            A = __fmul2_rn(A, a[i]);
            R = __ffma2_rn(A, dout_at(i), R);
        }
        float4 (&maps)[kChainWarps][32] = sh.maps[n];
        float2 (&rights)[kChainWarps][32] = sh.rights[n];
        maps[warp][lane] = make_float4(A.x, A.y, H.x, H.y);
        rights[warp][lane] = R;
        if (chain_sync_any(leave)) break;
        float2 r = carry;
#pragma unroll
        for (int v = kChainWarps - 1; v >= 0; --v) {
            if (v == warp) r = carry;
            const float2 av = *reinterpret_cast<const float2*>(&maps[v][lane]);
            carry = __ffma2_rn(av, carry, rights[v][lane]);
        }
        float2 h = *reinterpret_cast<const float2*>(sh.ring[s] + 3 * kBytes + 8 * lane);
        for (int v = 0; v < warp; ++v) {
            const float4 m = maps[v][lane];
            h = __ffma2_rn(make_float2(m.x, m.y), h, make_float2(m.z, m.w));
        }
        if (warp == 0 && (at.edge & kChainLast)) {
            if (at.position + 1 < p.stretches) chain_send(p, at, lane, carry);
            else if (p.last != nullptr) chain_store2(p.last + at.b * p.dim, d, p.dim, carry);
        }
        // x becomes what the decay's gradient multiplies: x_t - h_{t-1}, or h_{t-1}
#pragma unroll
        for (int i = 0; i < kChainSteps; ++i) {
            const float2 u = kLog ? x[i] : __fmul2_rn(g[i], x[i]);
            x[i] = kLog ? h : __ffma2_rn(h, make_float2(-1.0f, -1.0f), x[i]);
            h = __ffma2_rn(a[i], h, u);
        }
#pragma unroll
        for (int i = kChainSteps - 1; i >= 0; --i) {
            const float2 l = __fadd2_rn(dout_at(i), r);
            r = __fmul2_rn(a[i], l);
            float2 df = __fmul2_rn(r, x[i]), dv = l;
            if constexpr (!kLog) {
                df = __fmul2_rn(g[i], df);
                dv = __fmul2_rn(g[i], l);
            }
            if (left < kChainSteps && i >= left) df = dv = zero;
            db = __fadd2_rn(db, df);
            ring_put<IoT>(grow + i * kRow, lane, df);
            ring_put<IoT>(xrow + i * kRow, lane, dv);
        }
        const int t = at.tile * kChainTile + warp * kChainSteps;
        chain_send_rows<2>(&p.out0, &p.out1, smem_u32(grow), smem_u32(xrow), at.d0, t, at.b, lane,
                           t < p.seqlen, previous);
        previous = &sh.empty[s];
        if ((at.edge & kChainLast) && p.bias_partial != nullptr) {
            // the warps' sums over the stretch, in order
            const int64_t row = (int64_t)at.b * p.stretches + at.position;
            chain_sync();                              // maps of this tile have been read
            rights[warp][lane] = db;
            chain_sync();
            if (warp == 0) {
                float2 sum = zero;
#pragma unroll
                for (int v = 0; v < kChainWarps; ++v) sum = __fadd2_rn(sum, rights[v][lane]);
                chain_store2(p.bias_partial + row * p.dim, d, p.dim, sum);
            }
        }
    }
    if (lane == 0) bulk_wait_read<0>();
}

// --------------------------------------------------------------- few chains
//
// With fewer groups of channels than fill the GPU, time has to be split as well.
// A segment is 8 blocks of kSteps steps x 64 channels, one per warp, brought by
// TMA and kept in shared memory while the segments of a chain are joined
// (gated_join): phase one reads a block for its map, phase two again for its
// outputs, which replace x there and leave by TMA.  HBM sees each input once; the
// steps' arithmetic is done twice.  Three CTAs per SM cover one another's loads
// and joins, and each asks L2 for its next segment before it joins.  bf16, 1 x 131072
// x 1536 (batch, seqlen, dim), log decay, last state: 324 us, 3.73 TB/s, 57 % (342 without
// the request to L2); 1 x 4096 x 4096 47 us (a CTA per chain: 115).  Bound by the waits
// for earlier segments' maps; 32 steps per warp measured best.
template <typename IoT>
struct SegmentSizes {
    static constexpr int kSteps = sizeof(IoT) == 2 ? 32 : 16;                      // per warp
    static constexpr int kBlock = kSteps * kChainChannels * (int)sizeof(IoT);      // bytes of one tensor's block
    static constexpr int kSegment = kSteps * kChainWarps;
};

template <typename IoT>
struct SegmentShared {
    alignas(128) unsigned char blocks[kChainWarps][2][SegmentSizes<IoT>::kBlock];  // gate, x (then out)
    float4 maps[kChainWarps][32];
    float2 entering[kChainWarps][32];
    uint64_t full[kChainWarps];
    int64_t first_slot, next_slot;
};

struct SegmentParams {
    CUtensorMap gate, x, out;      // boxes of 64 channels x kSteps steps
    const float* bias;             // (dim) or null
    const float* h0;               // (batch, dim) or null
    const int32_t* seqlens;        // (batch) or null
    float* last;                   // or null
    float* enter;                  // [batch][blocks of 64 steps][dim] or null
    GatedLinks links;
    unsigned int* ticket;          // null: one segment per chain
    int64_t dim, seqlen, blocks;
    int64_t groups_per_row, groups, items;
};

template <typename IoT, bool kLog>
__global__ void __launch_bounds__(kChainWarps * 32, 3)
    gated_segment_fwd_kernel(const __grid_constant__ SegmentParams p) {
    extern __shared__ __align__(128) unsigned char raw[];
    auto& sh = *reinterpret_cast<SegmentShared<IoT>*>(raw);
    using Sizes = SegmentSizes<IoT>;
    constexpr int kSteps = Sizes::kSteps, kAt = 8;       // steps worked on at a time
    constexpr int kRow = kChainChannels * (int)sizeof(IoT);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2 one = make_float2(1.0f, 1.0f), zero = make_float2(0.0f, 0.0f);
    if (lane == 0) {
        mbar_init(smem_u32(&sh.full[warp]), 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) sh.first_slot = p.ticket != nullptr ? (int64_t)atomicAdd(p.ticket, 1u) : (int64_t)blockIdx.x;
    __syncthreads();
    unsigned char* grow = sh.blocks[warp][0];
    unsigned char* xrow = sh.blocks[warp][1];
    const uint32_t bar = smem_u32(&sh.full[warp]);
    // This warp's block of an item: its first step may lie behind the tensor's end
    // (then nothing is asked for).
    auto place = [&](int64_t item, int* b, int* d0, int64_t* t, int64_t* pos, int64_t* group) {
        *pos = item / p.groups;
        *group = item - *pos * p.groups;
        *b = (int)(*group / p.groups_per_row);
        *d0 = (int)(*group - *b * p.groups_per_row) * kChainChannels;
        *t = *pos * Sizes::kSegment + warp * kSteps;
    };
    auto prefetch = [&](int64_t item) {
        if (item >= p.items || lane != 0) return;
        int b, d0;
        int64_t t, pos, group;
        place(item, &b, &d0, &t, &pos, &group);
        if (t >= p.seqlen) return;
        tma_prefetch_3d(&p.gate, d0, (int)t, b);
        tma_prefetch_3d(&p.x, d0, (int)t, b);
    };
    auto request = [&](int64_t item) {
        if (item >= p.items || lane != 0) return;
        int b, d0;
        int64_t t, pos, group;
        place(item, &b, &d0, &t, &pos, &group);
        if (t >= p.seqlen) return;
        mbar_arrive_expect_tx(bar, 2 * Sizes::kBlock);
        tma_load_3d(smem_u32(grow), &p.gate, d0, (int)t, b, bar);
        tma_load_3d(smem_u32(xrow), &p.x, d0, (int)t, b, bar);
    };
    int64_t item = sh.first_slot;
    request(item);
    uint32_t parity = 0;
    while (item < p.items) {
        int b, d0;
        int64_t t, pos, group;
        place(item, &b, &d0, &t, &pos, &group);
        int64_t coming = p.items;                // asked for now, needed at the barrier
        if (threadIdx.x == 0 && p.ticket != nullptr) coming = atomicAdd(p.ticket, 1u);
        const int64_t d = d0 + 2 * lane;
        const int64_t len = p.seqlens != nullptr ? min(max((int64_t)p.seqlens[b], (int64_t)0), p.seqlen) : p.seqlen;
        const int left = (int)min(max(len - t, (int64_t)0), (int64_t)kSteps);
        float2 start[1] = {p.h0 != nullptr ? chain_load2(p.h0 + (int64_t)b * p.dim, d, p.dim) : zero};
        const float2 bias2 = p.bias != nullptr ? __fmul2_rn(chain_load2(p.bias, d, p.dim), make_float2(kLog2e, kLog2e)) : zero;
        bool failed = false;
        if (t < p.seqlen) {
            failed = !mbar_wait_bounded(bar, parity);
            parity ^= 1;
            if (failed) {
                record_device_error(MAMBA_ERR_TIMEOUT);
                mbar_wait_bounded(bar, parity ^ 1);      // the copy may still be on its way
            }
        }
        auto terms = [&](int s, float2 (&a)[kAt], float2 (&u)[kAt]) {
#pragma unroll
            for (int i = 0; i < kAt; ++i)
                gated_terms2<kLog>(ring_get<IoT>(grow + (s + i) * kRow, lane), bias2,
                                   ring_get<IoT>(xrow + (s + i) * kRow, lane), a[i], u[i]);
            if (left - s < kAt)
#pragma unroll
                for (int i = 0; i < kAt; ++i)
                    if (s + i >= left) {
                        a[i] = one;
                        u[i] = zero;
                    }
        };
        float2 A = one, H = zero;
        for (int s = 0; s < left; s += kAt) {
            float2 a[kAt], u[kAt];
            terms(s, a, u);
#pragma unroll
            for (int i = 0; i < kAt; ++i) {
                H = __ffma2_rn(a[i], H, u[i]);
                A = __fmul2_rn(A, a[i]);
            }
        }
        sh.maps[warp][lane] = make_float4(A.x, A.y, H.x, H.y);
        if (threadIdx.x == 0) sh.next_slot = coming;
        // a CTA whose copy never came leaves as a whole
        if (__syncthreads_or(failed)) break;
        const int64_t following = sh.next_slot;
        prefetch(following);                     // HBM works while the CTA waits for the join
        bool lost = false;
        if (warp == 0) {
            if (p.ticket != nullptr) {
                float2 At[1] = {one}, Ht[1] = {zero};
#pragma unroll
                for (int v = 0; v < kChainWarps; ++v) {
                    const float4 m = sh.maps[v][lane];
                    Ht[0] = __ffma2_rn(make_float2(m.x, m.y), Ht[0], make_float2(m.z, m.w));
                    At[0] = __fmul2_rn(At[0], make_float2(m.x, m.y));
                }
                lost = !gated_join<1>(p.links, group, pos, lane, At, Ht, start);
            }
            float2 h = start[0];
#pragma unroll
            for (int v = 0; v < kChainWarps; ++v) {
                const float4 m = sh.maps[v][lane];
                sh.entering[v][lane] = h;
                h = __ffma2_rn(make_float2(m.x, m.y), h, make_float2(m.z, m.w));
            }
        }
        // a wait that ran out is recorded: the CTA takes no further item, the call's outputs are undefined
        if (__syncthreads_or(lost)) break;
        float2 h = sh.entering[warp][lane];
        if (t < p.seqlen) {
            if (p.enter != nullptr && t % kChainTile == 0)
                chain_store2(p.enter + ((int64_t)b * p.blocks + t / kChainTile) * p.dim, d, p.dim, h);
            for (int s = 0; s < kSteps; s += kAt) {
                if (s < left) {
                    float2 a[kAt], u[kAt];
                    terms(s, a, u);
#pragma unroll
                    for (int i = 0; i < kAt; ++i) {
                        h = __ffma2_rn(a[i], h, u[i]);
                        ring_put<IoT>(xrow + (s + i) * kRow, lane, s + i < left ? h : zero);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kAt; ++i) ring_put<IoT>(xrow + (s + i) * kRow, lane, zero);
                }
            }
            if (p.last != nullptr && t + kSteps >= p.seqlen) chain_store2(p.last + (int64_t)b * p.dim, d, p.dim, h);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(&p.out, d0, (int)t, b, smem_u32(xrow));
                bulk_commit();
                bulk_wait_read<0>();
            }
        }
        request(following);                      // the block's own shared memory is free again
        item = following;
    }
    if (lane == 0) bulk_wait_read<0>();
}

}  // namespace mamba
