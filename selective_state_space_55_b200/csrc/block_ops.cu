// C ABI of the operators around a recurrent block's projections: layer norm,
// gated linear recurrence and the convolution's backward.  Argument checks,
// planning and kernel dispatch.
#include <algorithm>
#include <mutex>

#include "mamba_ssm.h"
#include "host_util.cuh"
#include "layer_norm.cuh"
#include "conv1d_backward.cuh"
#include "gated_scan.cuh"
#include "gated_chain.cuh"


namespace mamba {

bool block_ops_take_status(int* code) { return take_device_status(code); }

namespace {

constexpr int64_t kLimit31 = (int64_t)1 << 31;

mamba_status_t status_of(cudaError_t e) { return e == cudaSuccess ? MAMBA_OK : MAMBA_ERR_CUDA; }

// CTAs of `kernel` that fit on an SM, cached per device by the caller's slot array.
template <typename Kernel>
int resident_ctas(Kernel kernel, int threads, size_t smem, int* cache, int dev) {
    int n = (dev >= 0 && dev < kMaxDevices) ? cache[dev] : 0;
    if (n > 0) return n;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess) return 0;
    if (dev >= 0 && dev < kMaxDevices) cache[dev] = n;
    return n;
}

cudaError_t launch_column_sum(const float* partial, int64_t rows, int64_t cols, int64_t split,
                              float* first, float* second, cudaStream_t stream) {
    // A dependent launch: the CTAs may take their places while the kernel before
    // finishes, and wait for it on the device.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((cols + 31) / 32));
    cfg.blockDim = dim3(kColSumThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, column_sum_kernel, partial, rows, cols, split, first, second);
}

// ------------------------------------------------------------------ layer norm

struct NormPlan {
    bool wide;          // rows beyond a team's registers
    int chunks;         // of 8 elements per lane
    int warps;          // of a team (one row)
    int teams;          // side by side in a CTA
    int64_t ctas;
    int64_t slices;     // wide backward: row slices of the column sums
};

// Rows with a team each.  bf16 with a residual, us:
//  - few rows forward (fewer than two per SM): one or two chunks of 8 elements per
//    lane on many warps, the shortest way through a row (200 x 2560: 8 against 27);
//  - many rows forward: as many chunks per lane as waste the fewest lanes, the larger
//    number first (32768 x 2560: 5 chunks on 2 warps 119, 2 on 5 warps 152; 768
//    columns, 65536 rows: 3 on 1 warp 74, 2 on 2 warps 92);
//  - backward: two chunks, whatever lanes that wastes, because fewer teams keep more
//    column sums (32768 x 2560: 127 against 221 with one), but one chunk where rows x
//    256-column units leave less than 176 per SM (1000 x 2560: 18 against 25, 2000: 25
//    against 29, 4000: 39 against 35).
NormPlan plan_norm(int64_t rows, int64_t dim, int sms, bool backward) {
    NormPlan n{};
    const int64_t units = (dim + 255) / 256;               // chunks of a whole warp
    const int most = backward || rows < 2 * (int64_t)sms ? kNormFewChunks : kNormFwdChunks;
    const bool few = backward ? rows < 176 * (int64_t)sms / units : rows < 2 * (int64_t)sms;
    int64_t best = 0;
    for (int v = most; v >= 1; --v) {
        if (v == 7) continue;                               // not built: 1537 to 1792 columns take 8
        const int64_t warps = (units + v - 1) / v;
        if (warps > (v <= kNormFewChunks ? kNormFewWarps : kNormCtaWarps)) continue;
        // few rows: the smallest number that fits
        if (n.chunks == 0 || few || (!backward && warps * v < best)) {
            n.chunks = v;
            best = warps * v;
        }
    }
    if (n.chunks == 0 && !backward && units <= kNormFwdChunks * kNormCtaWarps) {
        n.chunks = kNormFwdChunks;                          // few wide rows
    }
    if (n.chunks == 0) {
        n.wide = true;
        n.warps = kNormWideThreads / 32;
        n.teams = 1;
    } else {
        n.warps = (int)((units + n.chunks - 1) / n.chunks);
        n.teams = std::max(1, kNormCtaWarps / n.warps);
        if (rows < (int64_t)sms * n.teams) n.teams = 1;
    }
    // CTAs that walk rows, at most: 1024 threads per SM.  The launch takes as many
    // of them as are resident at once.
    const int per_sm = std::max(1, 1024 / (n.warps * 32 * n.teams));
    n.ctas = std::max<int64_t>(1, std::min<int64_t>((rows + n.teams - 1) / n.teams, (int64_t)sms * per_sm));
    const int64_t col_blocks = (dim + kNormColThreads - 1) / kNormColThreads;
    n.slices = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(rows, 1024), (int64_t)sms * 8 / col_blocks));
    return n;
}

mamba_status_t check_norm(const mamba_norm_dims_t* d) {
    if (d == nullptr) return MAMBA_ERR_INVALID_ARG;
    if (d->rows < 0 || d->dim < 0 || d->rows >= ((int64_t)1 << 40)) return MAMBA_ERR_INVALID_ARG;
    if (d->dim > ((int64_t)1 << 28)) return MAMBA_ERR_UNSUPPORTED;
    if (!dtype_ok(d->io_dtype)) return MAMBA_ERR_UNSUPPORTED;
    if (d->residual_dtype != d->io_dtype && d->residual_dtype != MAMBA_F32) return MAMBA_ERR_UNSUPPORTED;
    const int64_t strides[5] = {d->x_stride, d->out_stride, d->residual_stride, d->residual_out_stride, d->dx_stride};
    for (const int64_t s : strides)
        if (s != 0 && (s < d->dim || s >= ((int64_t)1 << 40) || (d->rows > 0 && s > INT64_MAX / 8 / d->rows)))
            return MAMBA_ERR_INVALID_ARG;
    return MAMBA_OK;
}

int64_t norm_stride(int64_t s, int64_t dim) { return s != 0 ? s : dim; }

// Vectors of 8 elements: pointer and stride on 16-byte boundaries.
bool norm_vec(const void* p, int64_t stride, int es) {
    return p == nullptr || (aligned(p, 16) && (stride * es) % 16 == 0);
}

struct NormResident { size_t smem; int ctas; };

// Launches one instance.  Shared memory: first `fixed` bytes (the weights beyond
// a lane's registers, where the backward's sums of several teams come later),
// then every team's ring of rows of `stage` bytes.
template <typename Kernel>
cudaError_t launch_norm_kernel(Kernel kernel, const NormParams& prm, NormPlan& n, size_t fixed, size_t stage,
                               NormResident* resident, bool* attr_done, int dev, int sms, cudaStream_t stream) {
    // as many stages, two to four, as leave room for the CTAs that the registers
    // allow (512 threads of 128); with two, 32768 x 2560 bf16 backward takes 166 us
    // instead of 127
    constexpr int most = 226 * 1024;             // beside the kernels' static part
    const size_t share = most / std::max(1, 512 / (n.warps * n.teams * 32));
    int stages = stage == 0 ? 0 : kNormStages;
    while (stages > 2 && fixed + stages * stage * n.teams + 3 * 1024 > share) --stages;
    const size_t smem = fixed + stages * stage * n.teams;
    if (smem > most) return cudaErrorInvalidConfiguration;
    if (smem > 40 * 1024) {
        const cudaError_t e = ensure_smem_attr(kernel, most, attr_done, dev);
        if (e != cudaSuccess) return e;
    }
    // resident CTAs per SM; kept for the last shared memory size of each team size
    // (the number fixes the order of the backward's sums: it has to be this call's own)
    static std::mutex lock;
    int per_sm = 0;
    {
        std::lock_guard<std::mutex> guard(lock);
        NormResident& slot = resident[n.warps * (kNormCtaWarps + 1) + n.teams];
        if (slot.ctas <= 0 || slot.smem != smem) {
            int found = 0;
            const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&found, kernel, n.warps * n.teams * 32, smem);
            if (e != cudaSuccess) return e;
            if (found <= 0) return cudaErrorInvalidConfiguration;
            slot.smem = smem;
            slot.ctas = found;
        }
        per_sm = slot.ctas;
    }
    n.ctas = std::min<int64_t>(n.ctas, (int64_t)per_sm * sms);
    kernel<<<(unsigned)n.ctas, dim3(n.warps * 32, n.teams), smem, stream>>>(prm, (int)(fixed / 16), (int)stage, stages);
    return cudaGetLastError();
}

constexpr int kNormPlans = (kNormFewWarps + 1) * (kNormCtaWarps + 1);

template <typename IoT, typename ResT, int kV, bool kVec, bool kBackward>
cudaError_t launch_norm_chunks(const NormParams& prm, NormPlan& n, int dev, int sms, cudaStream_t stream) {
    static bool attr_done[kMaxDevices] = {false};
    static NormResident resident[kNormPlans] = {};
    const size_t width = (size_t)kV * 8 * 32 * n.warps * sizeof(float);
    // a stage: a row of x (dout) and of the residual stream's tensors
    size_t stage = 0;
    if (kVec && kV <= kNormFewChunks)
        stage = (size_t)prm.dim * (sizeof(IoT) + (kBackward ? 1 + (prm.dresidual_out != nullptr)
                                                            : prm.residual != nullptr) * sizeof(ResT));
    if constexpr (kBackward)
        return launch_norm_kernel(layer_norm_bwd_kernel<IoT, ResT, kV, kVec>, prm, n,
                                  n.teams > 1 ? 2 * width : (kV > 1 ? width : 0),
                                  stage, resident, attr_done, dev, sms, stream);
    else
        return launch_norm_kernel(layer_norm_fwd_kernel<IoT, ResT, kV, kVec>, prm, n, kV > 1 ? 2 * width : 0,
                                  stage, resident, attr_done, dev, sms, stream);
}

template <typename IoT, typename ResT, bool kVec>
cudaError_t dispatch_norm_fwd(const NormParams& prm, NormPlan& n, int dev, int sms, cudaStream_t stream) {
    switch (n.chunks) {
        case 1: return launch_norm_chunks<IoT, ResT, 1, kVec, false>(prm, n, dev, sms, stream);
        case 2: return launch_norm_chunks<IoT, ResT, 2, kVec, false>(prm, n, dev, sms, stream);
        case 3: return launch_norm_chunks<IoT, ResT, 3, kVec, false>(prm, n, dev, sms, stream);
        case 4: return launch_norm_chunks<IoT, ResT, 4, kVec, false>(prm, n, dev, sms, stream);
        case 5: return launch_norm_chunks<IoT, ResT, 5, kVec, false>(prm, n, dev, sms, stream);
        case 6: return launch_norm_chunks<IoT, ResT, 6, kVec, false>(prm, n, dev, sms, stream);
        default: return launch_norm_chunks<IoT, ResT, 8, kVec, false>(prm, n, dev, sms, stream);
    }
}

template <typename IoT, bool kVec>
cudaError_t launch_norm_fwd(const NormParams& prm, NormPlan& n, int dev, int sms, cudaStream_t stream) {
    if (n.wide) {
        layer_norm_fwd_wide_kernel<IoT, kVec><<<(unsigned)n.ctas, kNormWideThreads, 0, stream>>>(prm);
        return cudaGetLastError();
    }
    if (sizeof(IoT) == 2 && prm.res_f32 && (prm.residual != nullptr || prm.residual_out != nullptr))
        return dispatch_norm_fwd<IoT, float, kVec>(prm, n, dev, sms, stream);
    return dispatch_norm_fwd<IoT, IoT, kVec>(prm, n, dev, sms, stream);
}

// n.ctas becomes the number of partial rows.
template <typename IoT, bool kVec>
cudaError_t launch_norm_bwd(const NormParams& prm, NormPlan& n, int dev, int sms, cudaStream_t stream) {
    if (n.wide) {                       // sums first: dx may replace dout
        if (prm.partial != nullptr) {
            const dim3 cols((unsigned)((prm.dim + kNormColThreads - 1) / kNormColThreads), (unsigned)n.slices);
            layer_norm_bwd_cols_kernel<IoT><<<cols, kNormColThreads, 0, stream>>>(prm);
        }
        layer_norm_bwd_wide_kernel<IoT, kVec><<<(unsigned)n.ctas, kNormWideThreads, 0, stream>>>(prm);
        return cudaGetLastError();
    }
    if (sizeof(IoT) == 2 && prm.res_f32)
        return n.chunks == 1 ? launch_norm_chunks<IoT, float, 1, kVec, true>(prm, n, dev, sms, stream)
                             : launch_norm_chunks<IoT, float, 2, kVec, true>(prm, n, dev, sms, stream);
    return n.chunks == 1 ? launch_norm_chunks<IoT, IoT, 1, kVec, true>(prm, n, dev, sms, stream)
                         : launch_norm_chunks<IoT, IoT, 2, kVec, true>(prm, n, dev, sms, stream);
}

// ------------------------------------------------------------------ gated recurrence

// Distances of one tensor: packed when both are 0.
bool resolve_strides(const mamba_strides_t& s, int64_t batch, int64_t rows, int64_t inner, bool output,
                     GatedStrides* out) {
    out->batch = s.batch;
    out->row = s.row;
    if (s.batch == 0 && s.row == 0) {
        out->batch = rows * inner;
        out->row = inner;
        return true;
    }
    const int64_t lim = (int64_t)1 << 50;
    if (s.batch < 0 || s.row < 0 || s.batch >= lim || s.row >= lim) return false;
    if ((rows > 1 && s.row < inner) || (batch > 1 && s.batch < inner)) return false;
    if ((rows > 1 && s.row > lim / rows) || (batch > 1 && s.batch > lim / batch)) return false;
    if (output && rows > 1 && batch > 1) {
        const bool row_first = s.row <= s.batch;
        const int64_t near = row_first ? s.row : s.batch, far = row_first ? s.batch : s.row;
        if (far < near * ((row_first ? rows : batch) - 1) + inner) return false;
    }
    if (rows <= 1) out->row = inner;            // distances of extent one are never stepped
    if (batch <= 1) out->batch = out->row * std::max<int64_t>(rows, 1);
    return true;
}

mamba_status_t check_gated(const mamba_gated_dims_t* d) {
    if (d == nullptr) return MAMBA_ERR_INVALID_ARG;
    if (d->batch < 0 || d->dim < 0 || d->seqlen < 0) return MAMBA_ERR_INVALID_ARG;
    if (d->batch >= kLimit31 || d->dim >= kLimit31 || d->seqlen >= kLimit31) return MAMBA_ERR_INVALID_ARG;
    if (!dtype_ok(d->io_dtype)) return MAMBA_ERR_UNSUPPORTED;
    if ((d->flags & ~(MAMBA_FLAG_LAYOUT_BLD | MAMBA_FLAG_TEST_WITHHOLD_HANDOFF)) != 0) return MAMBA_ERR_UNSUPPORTED;
    if (d->seqlen > kMaxRowSteps) return MAMBA_ERR_UNSUPPORTED;
    // element counts stay far inside 64 bits
    if (d->batch > 0 && d->dim > 0 && d->seqlen > 0 &&
        (d->batch > ((int64_t)1 << 50) / d->dim || d->batch * d->dim > ((int64_t)1 << 50) / d->seqlen))
        return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

bool gated_bld(const mamba_gated_dims_t* d) { return (d->flags & MAMBA_FLAG_LAYOUT_BLD) != 0; }

struct GatedLayout {           // offsets in the workspace, bytes
    size_t counters, flags, flags2, zeroed, maps, joins, enter, bias, states, total;
    int64_t blocks, segments, groups_per_row, groups, items;
    int64_t tiles;
    int warps, width;          // (batch, seqlen, dim): blocks per segment; else warps and lanes per chain
    // chained stretches
    size_t chain_zeroed, chain_zeroed_bytes, chain_handoff, chain_bias;
    bool chained;
    int64_t chain_groups, chain_stretches, chain_stretch_tiles;
    // segments of few chains, forward
    size_t seg_zeroed, seg_zeroed_bytes, seg_maps, seg_states;
    int64_t seg_segments;
};

// Chains of 64 channels from which a CTA per chain beats splitting time, both timed
// with dim 4096 (us, chained / split).  bf16 forward, L 4096: 128 groups 117 / 68, 192
// 123 / 92, 256 129 / 115, 512 183 / 226; L 1024, 256: 45 / 41.  bf16 backward, L 4096:
// 128 164 / 131, 192 178 / 186, 256 180 / 238.  fp32, L 4096: forward 128 115 / 96, 192
// 125 / 135; backward 192 264 / 266.
constexpr int64_t kChainMinGroups = 192, kChainMinGroupsBf16Forward = 320;
// What the plans take a B200 to hold (the workspace query must not depend on more than the
// sizes): 20 warps per SM along time, and two CTAs of the chained kernels per SM, which is
// the backward's and the fp32 forward's number (bf16 forward: three).
constexpr int64_t kRowResident = 20 * 148;
constexpr int64_t kChainResident = 2 * 148;

// One segment per chain needs no look-back: no tickets, flags or maps.
mamba_status_t gated_layout(const mamba_gated_dims_t* d, bool backward, bool recompute, int phase_max,
                            GatedLayout* w) {
    *w = GatedLayout{};
    const int64_t L = d->seqlen, chains = d->batch * d->dim;
    size_t off = 0;
    auto take = [&off](size_t bytes) { const size_t at = off; off += align256(bytes); return at; };
    if (gated_bld(d)) {
        w->blocks = (L + kGatedBlock - 1) / kGatedBlock;
        w->warps = (int)std::min<int64_t>(kGatedWarps, w->blocks);
        w->segments = (w->blocks + w->warps - 1) / w->warps;
        w->groups_per_row = (d->dim + kGatedChannels - 1) / kGatedChannels;
        w->groups = d->batch * w->groups_per_row;
        w->items = w->groups * w->segments;
        if (w->items >= kLimit31 / 2) return MAMBA_ERR_UNSUPPORTED;
        if (w->segments > 1) {
            w->counters = take(3 * sizeof(unsigned int));      // two tickets, the mark of a wait that ran out
            w->flags = take((size_t)w->items * sizeof(unsigned int));
            if (backward && recompute) w->flags2 = take((size_t)w->items * sizeof(unsigned int));
            w->zeroed = off;
            w->maps = take((size_t)w->items * 64 * sizeof(float4));
            w->joins = take((size_t)w->groups * ((w->segments + kGatedJoin - 1) / kGatedJoin) * 32 * sizeof(float4));
        }
        if (backward && recompute) w->enter = take((size_t)d->batch * w->blocks * d->dim * sizeof(float));
        if (backward) w->bias = take((size_t)d->batch * w->segments * d->dim * sizeof(float));
        // Chained stretches: some 4 items per resident CTA, 8 tiles or more each (bf16 8 x
        // 2048 x 4096, us with 1 / 4 / 8: forward 104 / 94 / 96, backward 174 / 168 / 164;
        // backward 8 x 4096 x 2048 178 / 180 / 184).
        w->chain_groups = d->batch * ((d->dim + kChainChannels - 1) / kChainChannels);
        const int64_t want = (4 * kChainResident + w->chain_groups - 1) / w->chain_groups;
        w->chain_stretches = std::max<int64_t>(1, std::min<int64_t>(want, w->blocks / 8));
        w->chain_stretch_tiles = (w->blocks + w->chain_stretches - 1) / w->chain_stretches;
        w->chain_stretches = (w->blocks + w->chain_stretch_tiles - 1) / w->chain_stretch_tiles;
        const size_t items = (size_t)w->chain_groups * w->chain_stretches;
        const bool bf16 = d->io_dtype == MAMBA_BF16;
        w->chained = w->chain_groups >= (bf16 && !backward ? kChainMinGroupsBf16Forward : kChainMinGroups) &&
                     items < (size_t)kLimit31 / 2;
        if (!backward && !w->chained) {
            const int64_t steps = bf16 ? SegmentSizes<__nv_bfloat16>::kSegment : SegmentSizes<float>::kSegment;
            w->seg_segments = (L + steps - 1) / steps;
            if (w->seg_segments > 1) {
                const size_t n = (size_t)w->chain_groups * w->seg_segments;
                w->seg_zeroed_bytes = 256 + n * sizeof(unsigned int);
                w->seg_zeroed = take(w->seg_zeroed_bytes);
                w->seg_maps = take(n * 32 * sizeof(float4));
                w->seg_states = take((size_t)w->chain_groups * ((w->seg_segments + kGatedJoin - 1) / kGatedJoin) * 32 * sizeof(float2));
            }
        }
        if (w->chained) {
            if (w->chain_stretches > 1) {
                w->chain_zeroed = take(256 + items * sizeof(unsigned int));
                w->chain_zeroed_bytes = 256 + items * sizeof(unsigned int);
                w->chain_handoff = take(items * kChainChannels * sizeof(float));
            }
            if (backward) w->chain_bias = take((size_t)d->batch * w->chain_stretches * d->dim * sizeof(float));
        }
    } else {
        // Lanes take 8 steps each; the row's start may lie up to phase_max steps into its tile.
        const int64_t span = L + phase_max, units = (span + kWarpSteps - 1) / kWarpSteps;
        if (chains >= kLimit31 - 1) return MAMBA_ERR_UNSUPPORTED;
        // Backward: as few tiles as possible, a second one costs a sweep.  Forward: one
        // warp per pair of chains where pairs are plentiful (tiles hand a state on for
        // less than warps do), more where they would not fill the GPU.  bf16, us with
        // at most 1 / 2 / 4 / 8 warps: 16384 pairs of 2048 steps 98 / 96 / 104 / 121, of
        // 2047 steps 127 / 147 / 139 / 166, 768 pairs of 32768 steps 143 / 107 / 82 / 86.
        int64_t most = kRowWarps;
        if (!backward) {
            const int64_t pairs = d->batch * ((d->dim + 1) / 2);
            for (most = 1; most < kRowWarps && pairs * most < kRowResident;) most *= 2;
        }
        w->tiles = (units + most - 1) / most;
        w->warps = (int)((units + w->tiles - 1) / w->tiles);
        w->width = 32;
        if (units == 1)
            while (w->width > 1 && (w->width / 2) * (int64_t)kLaneSteps >= span) w->width /= 2;
        if (backward) {
            w->bias = take((size_t)chains * sizeof(float));
            if (w->tiles > 1) w->states = take((size_t)chains * w->tiles * sizeof(float));
        }
    }
    w->total = off;
    return MAMBA_OK;
}

template <typename IoT, bool kLog, bool kVec, bool kBackward>
cudaError_t launch_gated_tiles(const GatedParams& prm, int warps, int dev, int sms, cudaStream_t stream) {
    static int resident[kMaxDevices] = {0};
    auto kernel = gated_scan_fwd_kernel<IoT, kLog, kVec>;
    size_t smem = 0;
    if constexpr (kBackward) {
        static bool attr_done[kMaxDevices] = {false};
        kernel = gated_scan_bwd_kernel<IoT, kLog, kVec>;
        const cudaError_t e = ensure_smem_attr(kernel, kGatedBwdSmem, attr_done, dev);
        if (e != cudaSuccess) return e;
        smem = (size_t)kGatedBwdSmem / kGatedWarps * warps;
    }
    int64_t grid = prm.items;
    if (prm.ticket != nullptr) {        // several segments: CTAs that stay and take one after another
        const int per_sm = resident_ctas(kernel, kGatedThreads, smem, resident, dev);
        if (per_sm <= 0) return cudaErrorInvalidConfiguration;
        grid = std::min<int64_t>(grid, (int64_t)per_sm * sms);
    }
    kernel<<<(unsigned)grid, warps * 32, smem, stream>>>(prm);
    return cudaGetLastError();
}

template <bool kBackward>
cudaError_t dispatch_gated_tiles(const GatedParams& prm, int warps, bool bf16, bool log_decay, bool vec,
                                 int dev, int sms, cudaStream_t stream) {
    using B = __nv_bfloat16;
    if (bf16) {
        if (log_decay)
            return vec ? launch_gated_tiles<B, true, true, kBackward>(prm, warps, dev, sms, stream)
                       : launch_gated_tiles<B, true, false, kBackward>(prm, warps, dev, sms, stream);
        return vec ? launch_gated_tiles<B, false, true, kBackward>(prm, warps, dev, sms, stream)
                   : launch_gated_tiles<B, false, false, kBackward>(prm, warps, dev, sms, stream);
    }
    if (log_decay)
        return vec ? launch_gated_tiles<float, true, true, kBackward>(prm, warps, dev, sms, stream)
                   : launch_gated_tiles<float, true, false, kBackward>(prm, warps, dev, sms, stream);
    return vec ? launch_gated_tiles<float, false, true, kBackward>(prm, warps, dev, sms, stream)
               : launch_gated_tiles<float, false, false, kBackward>(prm, warps, dev, sms, stream);
}

// Can TMA move boxes of this tensor?  16-byte base and distances.
bool chain_tensor_ok(const void* p, const GatedStrides& s, int es, int64_t batch) {
    return aligned(p, 16) && (s.row * es) % 16 == 0 && s.row * es < ((int64_t)1 << 40) &&
           (batch == 1 || ((s.batch * es) % 16 == 0 && s.batch * es < ((int64_t)1 << 40)));
}

bool encode_chain_map(CUtensorMap* map, const void* base, const GatedStrides& s, const mamba_gated_dims_t* d,
                      int es, uint32_t steps) {
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d->dim, (cuuint64_t)d->seqlen, (cuuint64_t)d->batch};
    const cuuint64_t row = (cuuint64_t)s.row * es;
    const cuuint64_t strides[2] = {row, d->batch > 1 ? (cuuint64_t)s.batch * es : row};
    const cuuint32_t box[3] = {(cuuint32_t)kChainChannels, steps, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(map, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The states entering tiles, (batch, tiles, dim) fp32, one tile's 64 channels per box.
bool encode_chain_states(CUtensorMap* map, const float* base, int64_t dim, int64_t tiles, int64_t batch) {
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)tiles, (cuuint64_t)batch};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 4, (cuuint64_t)(dim * tiles) * 4};
    const cuuint32_t box[3] = {(cuuint32_t)kChainChannels, 1, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename IoT, bool kLog, bool kBackward>
cudaError_t launch_gated_chain(const ChainParams& prm, int dev, int sms, cudaStream_t stream) {
    static int resident[kMaxDevices] = {0};
    static bool attr_done[kMaxDevices] = {false};
    auto kernel = gated_chain_fwd_kernel<IoT, kLog>;
    if constexpr (kBackward) kernel = gated_chain_bwd_kernel<IoT, kLog>;
    constexpr int smem = (int)sizeof(ChainShared<IoT, kBackward>);
    const cudaError_t e = ensure_smem_attr(kernel, smem, attr_done, dev);
    if (e != cudaSuccess) return e;
    int64_t grid = prm.items;
    if (prm.ticket != nullptr) {
        const int per_sm = resident_ctas(kernel, kChainThreads, smem, resident, dev);
        if (per_sm <= 0) return cudaErrorInvalidConfiguration;
        grid = std::min<int64_t>(grid, (int64_t)per_sm * sms);
    }
    kernel<<<(unsigned)grid, kChainThreads, smem, stream>>>(prm);
    return cudaGetLastError();
}

// The chained kernels: what the tile kernels' parameters say, with TMA maps.
template <bool kBackward>
mamba_status_t run_gated_chain(const GatedParams& g, const GatedLayout& w, const mamba_gated_dims_t* d, uint8_t* ws,
                               int dev, int sms, cudaStream_t stream) {
    const int es = dtype_bytes(d->io_dtype);
    ChainParams prm{};
    bool ok = encode_chain_map(&prm.gate, g.gate, g.gate_s, d, es, kChainTile) &&
              encode_chain_map(&prm.x, g.x, g.x_s, d, es, kChainTile);
    if (kBackward)
        ok = ok && encode_chain_map(&prm.dout, g.dout, g.out_s, d, es, kChainTile) &&
             encode_chain_map(&prm.out0, g.dgate, g.dgate_s, d, es, kChainSteps) &&
             encode_chain_map(&prm.out1, g.dx, g.dx_s, d, es, kChainSteps) &&
             encode_chain_states(&prm.states, g.enter, d->dim, w.blocks, d->batch);
    else
        ok = ok && encode_chain_map(&prm.out0, g.out, g.out_s, d, es, kChainSteps);
    if (!ok) return MAMBA_ERR_CUDA;
    prm.bias = g.bias;
    prm.h0 = g.h0;
    prm.dlast = g.dlast;
    prm.seqlens = g.seqlens;
    prm.last = kBackward ? g.dh0 : g.last;
    prm.enter = g.enter;
    prm.bias_partial = kBackward && g.bias_partial != nullptr ? reinterpret_cast<float*>(ws + w.chain_bias) : nullptr;
    prm.dim = d->dim;
    prm.seqlen = d->seqlen;
    prm.tiles = w.blocks;
    prm.groups_per_row = (d->dim + kChainChannels - 1) / kChainChannels;
    prm.groups = w.chain_groups;
    prm.stretch_tiles = w.chain_stretch_tiles;
    prm.stretches = w.chain_stretches;
    prm.items = prm.groups * prm.stretches;
    prm.withhold = g.links.withhold;
    if (prm.stretches > 1) {
        prm.ticket = reinterpret_cast<unsigned int*>(ws + w.chain_zeroed);
        prm.failed = prm.ticket + 1;
        prm.flags = reinterpret_cast<unsigned int*>(ws + w.chain_zeroed + 256);
        prm.handoff = reinterpret_cast<float*>(ws + w.chain_handoff);
        if (cudaMemsetAsync(ws + w.chain_zeroed, 0, w.chain_zeroed_bytes, stream) != cudaSuccess) return MAMBA_ERR_CUDA;
    }
    const bool log_decay = d->log_decay != 0;
    if (d->io_dtype == MAMBA_BF16)
        return status_of(log_decay ? launch_gated_chain<__nv_bfloat16, true, kBackward>(prm, dev, sms, stream)
                                   : launch_gated_chain<__nv_bfloat16, false, kBackward>(prm, dev, sms, stream));
    return status_of(log_decay ? launch_gated_chain<float, true, kBackward>(prm, dev, sms, stream)
                               : launch_gated_chain<float, false, kBackward>(prm, dev, sms, stream));
}

template <typename IoT, bool kLog>
cudaError_t launch_gated_segments(const SegmentParams& prm, int dev, int sms, cudaStream_t stream) {
    static int resident[kMaxDevices] = {0};
    static bool attr_done[kMaxDevices] = {false};
    auto kernel = gated_segment_fwd_kernel<IoT, kLog>;
    constexpr int smem = (int)sizeof(SegmentShared<IoT>);
    const cudaError_t e = ensure_smem_attr(kernel, smem, attr_done, dev);
    if (e != cudaSuccess) return e;
    int64_t grid = prm.items;
    if (prm.ticket != nullptr) {
        const int per_sm = resident_ctas(kernel, kChainWarps * 32, smem, resident, dev);
        if (per_sm <= 0) return cudaErrorInvalidConfiguration;
        grid = std::min<int64_t>(grid, (int64_t)per_sm * sms);
    }
    kernel<<<(unsigned)grid, kChainWarps * 32, smem, stream>>>(prm);
    return cudaGetLastError();
}

// Few chains, forward.
mamba_status_t run_gated_segments(const GatedParams& g, const GatedLayout& w, const mamba_gated_dims_t* d, uint8_t* ws,
                                  int dev, int sms, cudaStream_t stream) {
    const int es = dtype_bytes(d->io_dtype);
    const bool bf16 = d->io_dtype == MAMBA_BF16, log_decay = d->log_decay != 0;
    const uint32_t steps = bf16 ? SegmentSizes<__nv_bfloat16>::kSteps : SegmentSizes<float>::kSteps;
    SegmentParams prm{};
    if (!encode_chain_map(&prm.gate, g.gate, g.gate_s, d, es, steps) || !encode_chain_map(&prm.x, g.x, g.x_s, d, es, steps) ||
        !encode_chain_map(&prm.out, g.out, g.out_s, d, es, steps))
        return MAMBA_ERR_CUDA;
    prm.bias = g.bias;
    prm.h0 = g.h0;
    prm.seqlens = g.seqlens;
    prm.last = g.last;
    prm.enter = g.enter;
    prm.dim = d->dim;
    prm.seqlen = d->seqlen;
    prm.blocks = w.blocks;
    prm.groups_per_row = (d->dim + kChainChannels - 1) / kChainChannels;
    prm.groups = w.chain_groups;
    prm.items = prm.groups * w.seg_segments;
    prm.links.segments = w.seg_segments;
    prm.links.withhold = g.links.withhold;
    if (w.seg_segments > 1) {
        prm.ticket = reinterpret_cast<unsigned int*>(ws + w.seg_zeroed);
        prm.links.failed = prm.ticket + 1;
        prm.links.flags = reinterpret_cast<unsigned int*>(ws + w.seg_zeroed + 256);
        prm.links.maps = reinterpret_cast<float4*>(ws + w.seg_maps);
        prm.links.states = reinterpret_cast<float2*>(ws + w.seg_states);
        if (cudaMemsetAsync(ws + w.seg_zeroed, 0, w.seg_zeroed_bytes, stream) != cudaSuccess) return MAMBA_ERR_CUDA;
    }
    if (bf16)
        return status_of(log_decay ? launch_gated_segments<__nv_bfloat16, true>(prm, dev, sms, stream)
                                   : launch_gated_segments<__nv_bfloat16, false>(prm, dev, sms, stream));
    return status_of(log_decay ? launch_gated_segments<float, true>(prm, dev, sms, stream)
                               : launch_gated_segments<float, false>(prm, dev, sms, stream));
}

template <typename IoT, bool kLog, bool kMulti, bool kBackward>
cudaError_t launch_gated_rows(const GatedParams& prm, const GatedLayout& w, int dev, int sms, cudaStream_t stream) {
    static int resident[kRowWarps + 1][kMaxDevices] = {};
    static bool attr_done[kMaxDevices] = {false};
    auto kernel = gated_scan_rows_fwd_kernel<IoT, kLog, kMulti>;
    if constexpr (kBackward) kernel = gated_scan_rows_bwd_kernel<IoT, kLog, kMulti>;
    constexpr int per_thread = RowStages<IoT, kBackward ? 3 : 2>::kBytesPerThread;
    const cudaError_t e = ensure_smem_attr(kernel, per_thread * kRowThreads, attr_done, dev);
    if (e != cudaSuccess) return e;
    const int teams = std::max(1, kGatedWarps / w.warps), threads = teams * w.warps * 32;
    const int64_t per_cta = (int64_t)teams * (32 / w.width);                  // pairs of chains
    const int64_t blocks = (prm.batch * ((prm.dim + 1) / 2) + per_cta - 1) / per_cta;
    const int per_sm = resident_ctas(kernel, threads, (size_t)per_thread * threads, resident[w.warps], dev);
    if (per_sm <= 0) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)per_sm * sms);
    kernel<<<grid, threads, per_thread * threads, stream>>>(prm, w.warps, w.width, blocks);
    return cudaGetLastError();
}

template <typename IoT, bool kLog, bool kBackward>
cudaError_t dispatch_gated_teams(const GatedParams& prm, const GatedLayout& w, int dev, int sms, cudaStream_t stream) {
    return w.warps > 1 ? launch_gated_rows<IoT, kLog, true, kBackward>(prm, w, dev, sms, stream)
                       : launch_gated_rows<IoT, kLog, false, kBackward>(prm, w, dev, sms, stream);
}

template <bool kBackward>
cudaError_t dispatch_gated_rows(const GatedParams& prm, const GatedLayout& w, bool bf16, bool log_decay,
                                int dev, int sms, cudaStream_t stream) {
    using B = __nv_bfloat16;
    if (bf16)
        return log_decay ? dispatch_gated_teams<B, true, kBackward>(prm, w, dev, sms, stream)
                         : dispatch_gated_teams<B, false, kBackward>(prm, w, dev, sms, stream);
    return log_decay ? dispatch_gated_teams<float, true, kBackward>(prm, w, dev, sms, stream)
                     : dispatch_gated_teams<float, false, kBackward>(prm, w, dev, sms, stream);
}

// Can every row of this tensor start a vector of `bytes`?
bool rows_aligned(const void* p, const GatedStrides& s, int es, int bytes) {
    return p == nullptr || (aligned(p, bytes) && (s.batch * es) % bytes == 0 && (s.row * es) % bytes == 0);
}

// Steps by which a row of gate may start past a 16-byte boundary, at most.
int gated_phase_max(const void* gate, const GatedStrides& s, int es) {
    return rows_aligned(gate, s, es, 16) ? 0 : 16 / es - 1;
}

// What both directions share: sizes, inputs, distances of gate and x.
mamba_status_t gated_common(const void* gate, const void* x, const float* bias, const float* h0,
                            const mamba_gated_dims_t* d, GatedParams* prm) {
    const int64_t rows = gated_bld(d) ? d->seqlen : d->dim, inner = gated_bld(d) ? d->dim : d->seqlen;
    const int es = dtype_bytes(d->io_dtype);
    if (d->seqlen > 0 && (gate == nullptr || x == nullptr)) return MAMBA_ERR_INVALID_ARG;
    if ((gate && !aligned(gate, es)) || (x && !aligned(x, es)) || (bias && !aligned(bias, 4)) ||
        (h0 && !aligned(h0, 4)) || (d->seqlens && !aligned(d->seqlens, 4)))
        return MAMBA_ERR_ALIGN;
    if (!resolve_strides(d->gate, d->batch, rows, inner, false, &prm->gate_s) ||
        !resolve_strides(d->x, d->batch, rows, inner, false, &prm->x_s))
        return MAMBA_ERR_INVALID_ARG;
    prm->gate = gate;
    prm->x = x;
    prm->bias = bias;
    prm->h0 = h0;
    prm->seqlens = d->seqlens;
    prm->batch = d->batch;
    prm->dim = d->dim;
    prm->seqlen = d->seqlen;
    prm->chains = d->batch * d->dim;
    prm->links.withhold = (d->flags & MAMBA_FLAG_TEST_WITHHOLD_HANDOFF) != 0;
    return MAMBA_OK;
}

void gated_apply_layout(const GatedLayout& w, uint8_t* ws, GatedParams* prm) {
    prm->tiles = w.tiles;
    prm->blocks = w.blocks;
    prm->segments = w.segments;
    prm->groups_per_row = w.groups_per_row;
    prm->groups = w.groups;
    prm->items = w.items;
    prm->ticket = w.zeroed ? reinterpret_cast<unsigned int*>(ws + w.counters) : nullptr;
    prm->links.failed = reinterpret_cast<unsigned int*>(ws + w.counters) + 2;
    prm->links.segments = w.segments;
    prm->links.flags = reinterpret_cast<unsigned int*>(ws + w.flags);
    prm->links.maps = reinterpret_cast<float4*>(ws + w.maps);
    prm->links.states = reinterpret_cast<float2*>(ws + w.joins);
}

mamba_status_t check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return MAMBA_OK;
    if (ws == nullptr || have < need) return MAMBA_ERR_WORKSPACE;
    return aligned(ws, 256) ? MAMBA_OK : MAMBA_ERR_ALIGN;
}

cudaError_t copy_or_zero(float* dst, const float* src, size_t bytes, cudaStream_t stream) {
    if (dst == nullptr || dst == src) return cudaSuccess;
    return src != nullptr ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, stream)
                          : cudaMemsetAsync(dst, 0, bytes, stream);
}

// ------------------------------------------------------------------ convolution backward

struct ConvBwdPlan { int64_t stretch_tiles, stretches; size_t bytes; };

// A warp per pair of rows, or several, each with a stretch of whole tiles: enough of
// them to occupy the 16 warps that an SM holds.  A stretch costs about 4 tiles beside
// its own (its sums, its ring's first fill), and a started last wave about half a wave.
// bf16, us: 1 x 5120 x 2048 in 1 / 2 / 3 stretches 35 / 43 / 49; 1 x 1536 x 65536 in 2 /
// 3 / 4 / 10 stretches 186 / 158 / 184 / 168.
mamba_status_t plan_conv_bwd(const mamba_dims_t* d, int width, int sms, ConvBwdPlan* n) {
    const int64_t chains = d->batch * d->dim;
    const int es = dtype_bytes(d->io_dtype);
    const int64_t tiles = std::max<int64_t>(1, (d->seqlen + 16 / es - 1 + kWarpSteps - 1) / kWarpSteps);
    const int64_t pairs = (chains + 1) / 2;
    const double resident = 16.0 * sms;
    const int64_t most = std::min<int64_t>(tiles, (int64_t)(4 * resident) / std::max<int64_t>(pairs, 1) + 1);
    double best = 0;
    n->stretches = 1;
    for (int64_t s = 1; s <= std::min<int64_t>(most, 1024); ++s) {
        const double waves = (double)s * pairs / resident;
        const double cost = (waves <= 1 ? 1.0 : waves + 0.5) * (double)((tiles + s - 1) / s + 4);
        if (s == 1 || cost < best) {
            best = cost;
            n->stretches = s;
        }
    }
    n->stretch_tiles = (tiles + n->stretches - 1) / n->stretches;
    n->stretches = (tiles + n->stretch_tiles - 1) / n->stretch_tiles;
    if (pairs * n->stretches / kConvBwdWarps >= kLimit31 - 1) return MAMBA_ERR_UNSUPPORTED;
    n->bytes = align256((size_t)d->batch * n->stretches * (width + 1) * d->dim * sizeof(float));
    return MAMBA_OK;
}

mamba_status_t check_conv_bwd(const mamba_dims_t* d, int width) {
    if (d == nullptr) return MAMBA_ERR_INVALID_ARG;
    if (d->batch < 0 || d->dim < 0 || d->seqlen < 0) return MAMBA_ERR_INVALID_ARG;
    if (width < 1 || width > MAMBA_MAX_CONV_WIDTH) return MAMBA_ERR_UNSUPPORTED;
    if (!dtype_ok(d->io_dtype)) return MAMBA_ERR_UNSUPPORTED;
    if (d->batch >= kLimit31 || d->dim >= kLimit31 || d->seqlen >= kLimit31) return MAMBA_ERR_INVALID_ARG;
    if (d->batch * d->dim >= ((int64_t)1 << 40) || d->seqlen > kMaxRowSteps) return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

template <typename IoT, int kW>
cudaError_t launch_conv_bwd_width(const ConvBwdParams& prm, int dev, cudaStream_t stream) {
    static bool attr_done[kMaxDevices] = {false};
    constexpr int smem = ConvRing<IoT>::kBytes;
    const cudaError_t e = ensure_smem_attr(causal_conv1d_bwd_kernel<IoT, kW>, smem, attr_done, dev);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((prm.pairs * prm.stretches + kConvBwdWarps - 1) / kConvBwdWarps);
    causal_conv1d_bwd_kernel<IoT, kW><<<grid, kConvBwdWarps * 32, smem, stream>>>(prm);
    return cudaGetLastError();
}

template <typename IoT>
cudaError_t launch_conv_bwd(const ConvBwdParams& prm, int width, int dev, cudaStream_t stream) {
    switch (width) {
        case 1: return launch_conv_bwd_width<IoT, 1>(prm, dev, stream);
        case 2: return launch_conv_bwd_width<IoT, 2>(prm, dev, stream);
        case 3: return launch_conv_bwd_width<IoT, 3>(prm, dev, stream);
        default: return launch_conv_bwd_width<IoT, 4>(prm, dev, stream);
    }
}

}  // namespace
}  // namespace mamba

using namespace mamba;

extern "C" {

MAMBA_API mamba_status_t mamba_layer_norm_fwd(const void* x, const void* residual, const float* weight,
                                              const float* bias, void* out, void* residual_out,
                                              float* mean, float* rstd, const mamba_norm_dims_t* dims,
                                              cudaStream_t stream) {
    const mamba_status_t st = check_norm(dims);
    if (st != MAMBA_OK) return st;
    if (!(dims->eps >= 0.0f)) return MAMBA_ERR_INVALID_ARG;
    if (dims->rows == 0) return MAMBA_OK;
    if (dims->dim == 0) {               // moments of nothing: 0 / 0 (all bits set is a NaN)
        if ((mean && !aligned(mean, 4)) || (rstd && !aligned(rstd, 4))) return MAMBA_ERR_ALIGN;
        const size_t bytes = (size_t)dims->rows * sizeof(float);
        cudaError_t e = mean != nullptr ? cudaMemsetAsync(mean, dims->rms ? 0 : 0xff, bytes, stream) : cudaSuccess;
        if (e == cudaSuccess && rstd != nullptr) e = cudaMemsetAsync(rstd, 0xff, bytes, stream);
        return status_of(e);
    }
    if (x == nullptr || out == nullptr) return MAMBA_ERR_INVALID_ARG;
    const int es = dtype_bytes(dims->io_dtype), rs = dtype_bytes(dims->residual_dtype);
    if (!aligned(x, es) || !aligned(out, es) || (residual && !aligned(residual, rs)) ||
        (residual_out && !aligned(residual_out, rs)) || (weight && !aligned(weight, 4)) ||
        (bias && !aligned(bias, 4)) || (mean && !aligned(mean, 4)) || (rstd && !aligned(rstd, 4)))
        return MAMBA_ERR_ALIGN;
    NormParams prm{};
    prm.x = x;
    prm.residual = residual;
    prm.weight = weight;
    prm.bias = bias;
    prm.out = out;
    prm.residual_out = residual_out;
    prm.mean = mean;
    prm.rstd = rstd;
    prm.rows = dims->rows;
    prm.dim = (int)dims->dim;
    prm.x_stride = norm_stride(dims->x_stride, dims->dim);
    prm.out_stride = norm_stride(dims->out_stride, dims->dim);
    prm.residual_stride = norm_stride(dims->residual_stride, dims->dim);
    prm.residual_out_stride = norm_stride(dims->residual_out_stride, dims->dim);
    prm.eps = dims->eps;
    prm.rms = dims->rms != 0;
    prm.res_f32 = dims->residual_dtype == MAMBA_F32;
    // buffers may coincide only element for element
    if ((out == x && prm.out_stride != prm.x_stride) || (residual != nullptr && residual == out) ||
        (residual_out != nullptr &&
         (residual_out == x || residual_out == out ||
          (residual_out == residual && prm.residual_out_stride != prm.residual_stride))))
        return MAMBA_ERR_INVALID_ARG;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return MAMBA_ERR_CUDA;
    NormPlan n = plan_norm(dims->rows, dims->dim, sms, false);
    const bool vec = dims->dim % kNormElems == 0 && norm_vec(x, prm.x_stride, es) &&
                     norm_vec(out, prm.out_stride, es) && norm_vec(residual, prm.residual_stride, rs) &&
                     norm_vec(residual_out, prm.residual_out_stride, rs) && norm_vec(weight, 0, 4) &&
                     norm_vec(bias, 0, 4);
    if (dims->io_dtype == MAMBA_BF16)
        return status_of(vec ? launch_norm_fwd<__nv_bfloat16, true>(prm, n, dev, sms, stream)
                             : launch_norm_fwd<__nv_bfloat16, false>(prm, n, dev, sms, stream));
    return status_of(vec ? launch_norm_fwd<float, true>(prm, n, dev, sms, stream)
                         : launch_norm_fwd<float, false>(prm, n, dev, sms, stream));
}

MAMBA_API size_t mamba_layer_norm_bwd_workspace_bytes(const mamba_norm_dims_t* dims) {
    if (check_norm(dims) != MAMBA_OK) return static_cast<size_t>(-1);
    if (dims->rows == 0 || dims->dim == 0) return 0;
    const int sms = current_sm_count(nullptr);
    if (sms <= 0) return static_cast<size_t>(-1);
    const NormPlan n = plan_norm(dims->rows, dims->dim, sms, true);
    return align256((size_t)(n.wide ? n.slices : n.ctas) * 2 * dims->dim * sizeof(float));
}

MAMBA_API mamba_status_t mamba_layer_norm_bwd(const void* s, const float* weight, const float* mean,
                                              const float* rstd, const void* dout,
                                              const void* dresidual_out, void* dx, void* dresidual,
                                              float* dweight, float* dbias,
                                              const mamba_norm_dims_t* dims, cudaStream_t stream) {
    mamba_status_t st = check_norm(dims);
    if (st != MAMBA_OK) return st;
    if (dims->dim == 0) return MAMBA_OK;
    if ((dweight && !aligned(dweight, 4)) || (dbias && !aligned(dbias, 4))) return MAMBA_ERR_ALIGN;
    if (dims->rows == 0) {              // sums over no rows
        cudaError_t e = copy_or_zero(dweight, nullptr, (size_t)dims->dim * sizeof(float), stream);
        if (e == cudaSuccess) e = copy_or_zero(dbias, nullptr, (size_t)dims->dim * sizeof(float), stream);
        return status_of(e);
    }
    if (s == nullptr || dout == nullptr || dx == nullptr || rstd == nullptr ||
        (!dims->rms && mean == nullptr))
        return MAMBA_ERR_INVALID_ARG;
    const int es = dtype_bytes(dims->io_dtype), rs = dtype_bytes(dims->residual_dtype);
    if (!aligned(s, rs) || !aligned(dout, es) || !aligned(dx, es) ||
        (dresidual_out && !aligned(dresidual_out, rs)) || (dresidual && !aligned(dresidual, rs)) ||
        (weight && !aligned(weight, 4)) || (mean && !aligned(mean, 4)) || !aligned(rstd, 4))
        return MAMBA_ERR_ALIGN;
    NormParams prm{};
    prm.x = s;
    prm.weight = weight;
    prm.mean_in = mean;
    prm.rstd_in = rstd;
    prm.dout = dout;
    prm.dresidual_out = dresidual_out;
    prm.dx = dx;
    prm.dresidual = dresidual;
    prm.rows = dims->rows;
    prm.dim = (int)dims->dim;
    prm.x_stride = norm_stride(dims->x_stride, dims->dim);
    prm.out_stride = norm_stride(dims->out_stride, dims->dim);
    prm.residual_out_stride = norm_stride(dims->residual_out_stride, dims->dim);
    prm.dx_stride = norm_stride(dims->dx_stride, dims->dim);
    prm.dresidual_stride = norm_stride(dims->residual_stride, dims->dim);
    prm.rms = dims->rms != 0;
    prm.res_f32 = dims->residual_dtype == MAMBA_F32;
    prm.has_dw = dweight != nullptr;
    prm.has_db = dbias != nullptr;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return MAMBA_ERR_CUDA;
    NormPlan n = plan_norm(dims->rows, dims->dim, sms, true);
    // buffers may coincide only element for element
    if (dx == s || (dresidual != nullptr && (dresidual == s || dresidual == dx || dresidual == dout)) ||
        (dx == dout && prm.dx_stride != prm.out_stride) ||
        (dx == dresidual_out && (prm.dx_stride != prm.residual_out_stride || es != rs)) ||
        (dresidual != nullptr && dresidual == dresidual_out && prm.dresidual_stride != prm.residual_out_stride))
        return MAMBA_ERR_INVALID_ARG;
    const int sums = prm.has_dw + prm.has_db;
    if (sums > 0) {
        const size_t need = align256((size_t)(n.wide ? n.slices : n.ctas) * 2 * dims->dim * sizeof(float));
        st = check_workspace(dims->workspace, dims->workspace_bytes, need);
        if (st != MAMBA_OK) return st;
        prm.partial = static_cast<float*>(dims->workspace);
    }
    const bool vec = dims->dim % kNormElems == 0 && norm_vec(s, prm.x_stride, rs) &&
                     norm_vec(dout, prm.out_stride, es) && norm_vec(dresidual_out, prm.residual_out_stride, rs) &&
                     norm_vec(dx, prm.dx_stride, es) && norm_vec(dresidual, prm.dresidual_stride, rs) &&
                     norm_vec(weight, 0, 4);
    cudaError_t e;
    if (dims->io_dtype == MAMBA_BF16)
        e = vec ? launch_norm_bwd<__nv_bfloat16, true>(prm, n, dev, sms, stream)
                : launch_norm_bwd<__nv_bfloat16, false>(prm, n, dev, sms, stream);
    else
        e = vec ? launch_norm_bwd<float, true>(prm, n, dev, sms, stream) : launch_norm_bwd<float, false>(prm, n, dev, sms, stream);
    if (e == cudaSuccess && sums > 0)
        e = launch_column_sum(prm.partial, n.wide ? n.slices : n.ctas, (int64_t)sums * dims->dim,
                              prm.has_dw ? dims->dim : 0, dweight, dbias, stream);
    return status_of(e);
}

MAMBA_API size_t mamba_causal_conv1d_bwd_workspace_bytes(const mamba_dims_t* dims, int width) {
    if (check_conv_bwd(dims, width) != MAMBA_OK) return static_cast<size_t>(-1);
    if (dims->batch * dims->dim == 0) return 0;
    const int sms = current_sm_count(nullptr);
    ConvBwdPlan n;
    if (sms <= 0 || plan_conv_bwd(dims, width, sms, &n) != MAMBA_OK) return static_cast<size_t>(-1);
    return n.bytes;
}

MAMBA_API mamba_status_t mamba_causal_conv1d_bwd(
    const void* x, const float* weight, const float* bias, const void* initial_conv_state, int width,
    int silu, const void* dout, const void* dfinal_conv_state, void* dx, float* dweight, float* dbias,
    void* dinitial_conv_state, const mamba_dims_t* dims, cudaStream_t stream) {
    mamba_status_t st = check_conv_bwd(dims, width);
    if (st != MAMBA_OK) return st;
    if (dims->dim == 0) return MAMBA_OK;
    if (weight == nullptr || dweight == nullptr) return MAMBA_ERR_INVALID_ARG;
    if (!aligned(weight, 4) || !aligned(dweight, 4) || (bias && !aligned(bias, 4)) || (dbias && !aligned(dbias, 4)))
        return MAMBA_ERR_ALIGN;
    const int64_t chains = dims->batch * dims->dim;
    if (chains == 0) {                  // sums over no rows
        cudaError_t e = copy_or_zero(dweight, nullptr, (size_t)dims->dim * width * sizeof(float), stream);
        if (e == cudaSuccess) e = copy_or_zero(dbias, nullptr, (size_t)dims->dim * sizeof(float), stream);
        return status_of(e);
    }
    if (dims->seqlen > 0 && (x == nullptr || dout == nullptr || dx == nullptr)) return MAMBA_ERR_INVALID_ARG;
    const int es = dtype_bytes(dims->io_dtype);
    const void* io_ptrs[6] = {x, dout, dx, initial_conv_state, dfinal_conv_state, dinitial_conv_state};
    for (const void* q : io_ptrs)
        if (q && !aligned(q, es)) return MAMBA_ERR_ALIGN;
    if ((dx != nullptr && (dx == x || dx == dout)) ||
        (dinitial_conv_state != nullptr &&
         (dinitial_conv_state == initial_conv_state || dinitial_conv_state == dfinal_conv_state)))
        return MAMBA_ERR_INVALID_ARG;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return MAMBA_ERR_CUDA;
    ConvBwdPlan n;
    st = plan_conv_bwd(dims, width, sms, &n);
    if (st != MAMBA_OK) return st;
    st = check_workspace(dims->workspace, dims->workspace_bytes, n.bytes);
    if (st != MAMBA_OK) return st;
    ConvBwdParams prm{};
    prm.x = x;
    prm.dout = dout;
    prm.weight = weight;
    prm.bias = bias;
    prm.init = initial_conv_state;
    prm.dfinal = dfinal_conv_state;
    prm.dx = dx;
    prm.dinit = dinitial_conv_state;
    prm.partial = static_cast<float*>(dims->workspace);
    prm.dim = dims->dim;
    prm.seqlen = dims->seqlen;
    prm.chains = chains;
    prm.pairs = (chains + 1) / 2;
    prm.stretch_tiles = n.stretch_tiles;
    prm.stretches = n.stretches;
    prm.silu = silu != 0;
    cudaError_t e = dims->io_dtype == MAMBA_BF16 ? launch_conv_bwd<__nv_bfloat16>(prm, width, dev, stream)
                                                 : launch_conv_bwd<float>(prm, width, dev, stream);
    if (e == cudaSuccess)
        e = launch_column_sum(prm.partial, dims->batch * n.stretches, (int64_t)(width + 1) * dims->dim,
                              (int64_t)width * dims->dim, dweight, dbias, stream);
    return status_of(e);
}

MAMBA_API size_t mamba_gated_scan_workspace_bytes(const mamba_gated_dims_t* dims) {
    GatedLayout w;
    if (check_gated(dims) != MAMBA_OK) return static_cast<size_t>(-1);
    if (dims->batch * dims->dim == 0 || dims->seqlen == 0) return 0;
    return gated_layout(dims, false, false, 0, &w) == MAMBA_OK ? w.total : static_cast<size_t>(-1);
}

MAMBA_API mamba_status_t mamba_gated_scan_fwd(const void* gate, const void* x, const float* gate_bias,
                                              const float* initial_state, void* out, float* last_state,
                                              float* checkpoints, const mamba_gated_dims_t* dims,
                                              cudaStream_t stream) {
    mamba_status_t st = check_gated(dims);
    if (st != MAMBA_OK) return st;
    if (dims->batch * dims->dim == 0) return MAMBA_OK;
    const bool bld = gated_bld(dims);
    const int64_t rows = bld ? dims->seqlen : dims->dim, inner = bld ? dims->dim : dims->seqlen;
    const int es = dtype_bytes(dims->io_dtype);
    GatedParams prm{};
    st = gated_common(gate, x, gate_bias, initial_state, dims, &prm);
    if (st != MAMBA_OK) return st;
    if (dims->seqlen > 0 && out == nullptr) return MAMBA_ERR_INVALID_ARG;
    if (checkpoints != nullptr && !bld) return MAMBA_ERR_UNSUPPORTED;
    if ((out && !aligned(out, es)) || (last_state && !aligned(last_state, 4)) || (checkpoints && !aligned(checkpoints, 4)))
        return MAMBA_ERR_ALIGN;
    if (!resolve_strides(dims->out, dims->batch, rows, inner, true, &prm.out_s)) return MAMBA_ERR_INVALID_ARG;
    if (out != nullptr && (out == gate || out == x)) return MAMBA_ERR_INVALID_ARG;
    if (partly_overlap(initial_state, last_state, (size_t)prm.chains * sizeof(float))) return MAMBA_ERR_INVALID_ARG;
    if (dims->seqlen == 0)
        return status_of(copy_or_zero(last_state, initial_state, (size_t)prm.chains * sizeof(float), stream));
    GatedLayout w;
    st = gated_layout(dims, false, false, bld ? 0 : gated_phase_max(gate, prm.gate_s, es), &w);
    if (st != MAMBA_OK) return st;
    st = check_workspace(dims->workspace, dims->workspace_bytes, w.total);
    if (st != MAMBA_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(dims->workspace);
    gated_apply_layout(w, ws, &prm);
    prm.out = out;
    prm.last = last_state;
    const bool bf16 = dims->io_dtype == MAMBA_BF16, log_decay = dims->log_decay != 0;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return MAMBA_ERR_CUDA;
    if (!bld) return status_of(dispatch_gated_rows<false>(prm, w, bf16, log_decay, dev, sms, stream));
    prm.enter = checkpoints;
    if (chain_tensor_ok(gate, prm.gate_s, es, dims->batch) && chain_tensor_ok(x, prm.x_s, es, dims->batch) &&
        chain_tensor_ok(out, prm.out_s, es, dims->batch))
        return w.chained ? run_gated_chain<false>(prm, w, dims, ws, dev, sms, stream)
                                                 : run_gated_segments(prm, w, dims, ws, dev, sms, stream);
    if (w.zeroed && cudaMemsetAsync(ws, 0, w.zeroed, stream) != cudaSuccess) return MAMBA_ERR_CUDA;
    const bool vec = dims->dim % 4 == 0 && rows_aligned(gate, prm.gate_s, es, 4 * es) &&
                     rows_aligned(x, prm.x_s, es, 4 * es) && rows_aligned(out, prm.out_s, es, 4 * es) &&
                     (!gate_bias || aligned(gate_bias, 16)) && (!initial_state || aligned(initial_state, 16)) &&
                     (!last_state || aligned(last_state, 16)) && (!checkpoints || aligned(checkpoints, 16));
    return status_of(dispatch_gated_tiles<false>(prm, w.warps, bf16, log_decay, vec, dev, sms, stream));
}

MAMBA_API size_t mamba_gated_scan_bwd_workspace_bytes(const mamba_gated_dims_t* dims, int have_checkpoints) {
    GatedLayout w;
    if (check_gated(dims) != MAMBA_OK) return static_cast<size_t>(-1);
    if (dims->batch * dims->dim == 0 || dims->seqlen == 0) return 0;
    // the largest phase: alignment is only known at the call
    return gated_layout(dims, true, have_checkpoints == 0, 16 / dtype_bytes(dims->io_dtype) - 1, &w) == MAMBA_OK
               ? w.total : static_cast<size_t>(-1);
}

MAMBA_API mamba_status_t mamba_gated_scan_bwd(
    const void* gate, const void* x, const float* gate_bias, const float* initial_state,
    const float* checkpoints, const void* dout, const float* dlast_state, void* dgate, void* dx,
    float* dgate_bias, float* dinitial_state, const mamba_gated_dims_t* dims, cudaStream_t stream) {
    mamba_status_t st = check_gated(dims);
    if (st != MAMBA_OK) return st;
    if (dims->dim == 0) return MAMBA_OK;
    if (dgate_bias && !aligned(dgate_bias, 4)) return MAMBA_ERR_ALIGN;
    const size_t bias_bytes = (size_t)dims->dim * sizeof(float);
    if (dims->batch == 0) return status_of(copy_or_zero(dgate_bias, nullptr, bias_bytes, stream));
    const bool bld = gated_bld(dims);
    const int64_t rows = bld ? dims->seqlen : dims->dim, inner = bld ? dims->dim : dims->seqlen;
    const int es = dtype_bytes(dims->io_dtype);
    GatedParams prm{};
    st = gated_common(gate, x, gate_bias, initial_state, dims, &prm);
    if (st != MAMBA_OK) return st;
    if (dims->seqlen > 0 && (dout == nullptr || dgate == nullptr || dx == nullptr)) return MAMBA_ERR_INVALID_ARG;
    if (checkpoints != nullptr && !bld) return MAMBA_ERR_UNSUPPORTED;
    if ((dout && !aligned(dout, es)) || (dgate && !aligned(dgate, es)) || (dx && !aligned(dx, es)) ||
        (dlast_state && !aligned(dlast_state, 4)) || (dinitial_state && !aligned(dinitial_state, 4)) ||
        (checkpoints && !aligned(checkpoints, 4)))
        return MAMBA_ERR_ALIGN;
    if (!resolve_strides(dims->out, dims->batch, rows, inner, false, &prm.out_s) ||
        !resolve_strides(dims->dgate, dims->batch, rows, inner, true, &prm.dgate_s) ||
        !resolve_strides(dims->dx, dims->batch, rows, inner, true, &prm.dx_s))
        return MAMBA_ERR_INVALID_ARG;
    if (partly_overlap(dlast_state, dinitial_state, (size_t)prm.chains * sizeof(float))) return MAMBA_ERR_INVALID_ARG;
    if (dims->seqlen > 0 && (dgate == dx || dgate == gate || dgate == x || dgate == dout || dx == gate || dx == x || dx == dout))
        return MAMBA_ERR_INVALID_ARG;
    if (dims->seqlen == 0) {
        cudaError_t e = copy_or_zero(dgate_bias, nullptr, bias_bytes, stream);
        if (e == cudaSuccess) e = copy_or_zero(dinitial_state, dlast_state, (size_t)prm.chains * sizeof(float), stream);
        return status_of(e);
    }
    const bool recompute = checkpoints == nullptr;
    GatedLayout w;
    st = gated_layout(dims, true, recompute, bld ? 0 : gated_phase_max(gate, prm.gate_s, es), &w);
    if (st != MAMBA_OK) return st;
    st = check_workspace(dims->workspace, dims->workspace_bytes, w.total);
    if (st != MAMBA_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(dims->workspace);
    gated_apply_layout(w, ws, &prm);
    prm.dout = dout;
    prm.dlast = dlast_state;
    prm.dgate = dgate;
    prm.dx = dx;
    prm.dh0 = dinitial_state;
    prm.bias_partial = dgate_bias != nullptr ? reinterpret_cast<float*>(ws + w.bias) : nullptr;
    const bool bf16 = dims->io_dtype == MAMBA_BF16, log_decay = dims->log_decay != 0;
    cudaError_t e;
    int dev = 0;
    const int sms = current_sm_count(&dev);
    if (sms <= 0) return MAMBA_ERR_CUDA;
    if (!bld) {
        prm.chain_states = w.tiles > 1 ? reinterpret_cast<float*>(ws + w.states) : nullptr;
        e = dispatch_gated_rows<true>(prm, w, bf16, log_decay, dev, sms, stream);
        if (e == cudaSuccess && dgate_bias != nullptr)
            e = launch_column_sum(prm.bias_partial, dims->batch, dims->dim, dims->dim, dgate_bias, nullptr, stream);
        return status_of(e);
    }
    if (w.zeroed && cudaMemsetAsync(ws, 0, w.zeroed, stream) != cudaSuccess) return MAMBA_ERR_CUDA;
    const bool vec_in = dims->dim % 4 == 0 && rows_aligned(gate, prm.gate_s, es, 4 * es) &&
                        rows_aligned(x, prm.x_s, es, 4 * es) && (!gate_bias || aligned(gate_bias, 16)) &&
                        (!initial_state || aligned(initial_state, 16));
    if (recompute) {                    // the forward's states, no outputs
        GatedParams fwd = prm;
        fwd.out = nullptr;
        fwd.last = nullptr;
        fwd.enter = reinterpret_cast<float*>(ws + w.enter);
        if (w.zeroed) {
            fwd.ticket = prm.ticket + 1;
            fwd.links.flags = reinterpret_cast<unsigned int*>(ws + w.flags2);
        }
        e = dispatch_gated_tiles<false>(fwd, w.warps, bf16, log_decay, vec_in, dev, sms, stream);
        if (e != cudaSuccess) return MAMBA_ERR_CUDA;
        prm.enter = fwd.enter;
    } else {
        prm.enter = const_cast<float*>(checkpoints);
    }
    if (w.chained && chain_tensor_ok(gate, prm.gate_s, es, dims->batch) &&
        chain_tensor_ok(x, prm.x_s, es, dims->batch) && chain_tensor_ok(dout, prm.out_s, es, dims->batch) &&
        chain_tensor_ok(dgate, prm.dgate_s, es, dims->batch) && chain_tensor_ok(dx, prm.dx_s, es, dims->batch) &&
        dims->dim % 4 == 0 && aligned(prm.enter, 16)) {
        st = run_gated_chain<true>(prm, w, dims, ws, dev, sms, stream);
        if (st != MAMBA_OK || dgate_bias == nullptr) return st;
        return status_of(launch_column_sum(reinterpret_cast<float*>(ws + w.chain_bias), dims->batch * w.chain_stretches,
                                           dims->dim, dims->dim, dgate_bias, nullptr, stream));
    }
    const bool vec = vec_in && rows_aligned(dout, prm.out_s, es, 4 * es) &&
                     rows_aligned(dgate, prm.dgate_s, es, 4 * es) && rows_aligned(dx, prm.dx_s, es, 4 * es) &&
                     (!dlast_state || aligned(dlast_state, 16)) && (!dinitial_state || aligned(dinitial_state, 16)) &&
                     (!checkpoints || aligned(checkpoints, 16));
    e = dispatch_gated_tiles<true>(prm, w.warps, bf16, log_decay, vec, dev, sms, stream);
    if (e == cudaSuccess && dgate_bias != nullptr)
        e = launch_column_sum(prm.bias_partial, dims->batch * w.segments, dims->dim, dims->dim, dgate_bias, nullptr, stream);
    return status_of(e);
}

MAMBA_API mamba_status_t mamba_gated_state_update(float* state, const void* gate, const void* x,
                                                  const float* gate_bias, void* out,
                                                  const mamba_gated_dims_t* dims, cudaStream_t stream) {
    if (dims == nullptr || dims->batch < 0 || dims->dim < 0 || dims->batch >= kLimit31 || dims->dim >= kLimit31)
        return MAMBA_ERR_INVALID_ARG;
    if (!dtype_ok(dims->io_dtype)) return MAMBA_ERR_UNSUPPORTED;
    if (dims->batch * dims->dim == 0) return MAMBA_OK;
    if (state == nullptr || gate == nullptr || x == nullptr || out == nullptr) return MAMBA_ERR_INVALID_ARG;
    const int es = dtype_bytes(dims->io_dtype);
    if (!aligned(state, 4) || !aligned(gate, es) || !aligned(x, es) || !aligned(out, es) || (gate_bias && !aligned(gate_bias, 4)))
        return MAMBA_ERR_ALIGN;
    GatedUpdateParams prm{};
    const int64_t strides[3] = {dims->gate.batch, dims->x.batch, dims->out.batch};
    for (const int64_t s : strides)
        if (s < 0 || (s != 0 && (s < dims->dim || s > ((int64_t)1 << 50) / dims->batch))) return MAMBA_ERR_INVALID_ARG;
    prm.gate_stride = strides[0] ? strides[0] : dims->dim;
    prm.x_stride = strides[1] ? strides[1] : dims->dim;
    prm.out_stride = strides[2] ? strides[2] : dims->dim;
    if ((out == x && prm.out_stride != prm.x_stride) || (out == gate && prm.out_stride != prm.gate_stride) || out == state)
        return MAMBA_ERR_INVALID_ARG;
    prm.state = state;
    prm.gate = gate;
    prm.x = x;
    prm.bias = gate_bias;
    prm.out = out;
    prm.batch = dims->batch;
    prm.dim = dims->dim;
    auto on16 = [es](const void* p, int64_t stride) { return aligned(p, 16) && (stride * es) % 16 == 0; };
    const bool vec = dims->dim % 8 == 0 && aligned(state, 16) && on16(gate, prm.gate_stride) &&
                     on16(x, prm.x_stride) && on16(out, prm.out_stride) && (!gate_bias || aligned(gate_bias, 16));
    prm.per_row = vec ? dims->dim / 8 : dims->dim;
    const int64_t ctas = (prm.per_row * dims->batch + kGatedUpdateThreads - 1) / kGatedUpdateThreads;
    if (ctas >= kLimit31) return MAMBA_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)ctas;
#define MAMBA_GATED_UPDATE(T, LOG)                                                                   \
    if (vec) gated_update_kernel<T, LOG, 8><<<grid, kGatedUpdateThreads, 0, stream>>>(prm);          \
    else gated_update_kernel<T, LOG, 1><<<grid, kGatedUpdateThreads, 0, stream>>>(prm)
    if (dims->io_dtype == MAMBA_BF16) {
        if (dims->log_decay) { MAMBA_GATED_UPDATE(__nv_bfloat16, true); }
        else { MAMBA_GATED_UPDATE(__nv_bfloat16, false); }
    } else {
        if (dims->log_decay) { MAMBA_GATED_UPDATE(float, true); }
        else { MAMBA_GATED_UPDATE(float, false); }
    }
#undef MAMBA_GATED_UPDATE
    return status_of(cudaGetLastError());
}

}  // extern "C"
