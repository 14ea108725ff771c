// routing_api.cuh -- the C ABI of the expert-routing calls (declared in
// include/mxfp4.h): argument checks and launches.  Included by mxfp4_api.cu,
// whose error and launch helpers it uses.
#pragma once

#include "clip.cuh"
#include "plan.cuh"
#include "route.cuh"
#include "rows.cuh"

namespace {

// Launch a routing kernel.  It may be put in place while the stream's previous
// kernel ends, so every CTA waits for that one (cudaGridDependencySynchronize)
// before it touches what others write (plan_place_kernel behind its counting
// kernel leaves the wait for the ids to that one): 1.7 us less between two kernels
// (route, 8191 x 256 in groups: 14.3 -> 12.5 us a call).  cluster: CTAs of a
// cluster, 0 for the kernel's own.
template <typename... P>
mxfp4_status launch(const char* what, void (*kern)(P...), int64_t grid, int threads, size_t smem, cudaStream_t st,
                    unsigned cluster, const P&... args) {
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid), 1, 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(MXFP4_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
    }
    return ok();
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool known_dtype(int d) { return d == MXFP4_DTYPE_BF16 || d == MXFP4_DTYPE_F32; }

int dtype_bytes(int d) { return d == MXFP4_DTYPE_BF16 ? 2 : 4; }

// rows [rows, cols] of `esz`-byte elements, `ld` apart, start on 16 bytes and divide into vectors of 8 elements
bool wide_rows(const void* p, int64_t cols, int64_t ld, int esz) {
    return aligned16(p) && cols % 8 == 0 && (ld * esz) % 16 == 0;
}

// Raise a kernel's dynamic shared-memory limit, once per device.
template <auto Kern>
bool raise_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load() & bit) return true;
    if (cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit);
    return true;
}

constexpr int64_t kIndexEnd = int64_t(1) << 31;   // rows and slots are 32-bit indices

mxfp4_status check_route(const char* what, const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t ld,
                         const mxfp4_route_params* p) {
    if (!p) return fail(MXFP4_ERR_INVALID_ARG, "%s: null params", what);
    if (!known_dtype(dtype)) return fail(MXFP4_ERR_INVALID_ARG, "%s: bad dtype %d", what, dtype);
    if (p->score != MXFP4_SCORE_SOFTMAX && p->score != MXFP4_SCORE_SIGMOID)
        return fail(MXFP4_ERR_INVALID_ARG, "%s: bad score %d", what, p->score);
    if (tokens < 0 || experts < 1 || ld < experts) return fail(MXFP4_ERR_INVALID_ARG, "%s: bad geometry", what);
    if (experts > mxfp4::route::kMaxExperts)
        return fail(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: at most %d experts", what, mxfp4::route::kMaxExperts);
    if (p->top_k < 1 || p->top_k > experts) return fail(MXFP4_ERR_INVALID_ARG, "%s: top_k must lie in [1, experts]", what);
    if (p->top_k > mxfp4::route::kMaxTopK)
        return fail(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: top_k at most %d", what, mxfp4::route::kMaxTopK);
    if (tokens >= kIndexEnd || tokens * p->top_k >= kIndexEnd)
        return fail(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: tokens * top_k must be < 2^31", what);
    if (!(p->scale > -INFINITY && p->scale < INFINITY))
        return fail(MXFP4_ERR_INVALID_ARG, "%s: scale must be finite", what);
    if (tokens && !logits) return fail(MXFP4_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!aligned_to(logits, uintptr_t(dtype_bytes(dtype)))) return fail(MXFP4_ERR_MISALIGNED, "%s: logits misaligned", what);
    return ok();
}

template <bool BWD, typename T, bool SIGMOID>
mxfp4_status launch_route(const mxfp4::route::Args& a, cudaStream_t st) {
    using namespace mxfp4::route;
    const unsigned grid = unsigned((a.tokens + kWarps - 1) / kWarps);
    // the logits' own order where nothing is added to the scores
    const bool by_logit = !a.bias && (a.groups == 1 || a.group_best == 1);
    // a warp's keys: 64 bits of the scores', 32 of the groups'
    const size_t smem = BWD ? 0 : size_t(kWarps) * a.experts * (by_logit ? (a.groups > 1 ? 4 : 0) : 8);
    auto go = [&](auto kern) -> mxfp4_status {
        return launch(BWD ? "mxfp4_route_bwd" : "mxfp4_route", kern, grid, kWarps * 32, smem, st, 0, a);
    };
    if constexpr (BWD) {
        if (a.experts <= 32) return go(route_bwd_kernel<T, SIGMOID, 1>);
        if (a.experts <= 64) return go(route_bwd_kernel<T, SIGMOID, 2>);
        if (a.experts <= 128) return go(route_bwd_kernel<T, SIGMOID, 4>);
        if (a.experts <= 256) return go(route_bwd_kernel<T, SIGMOID, 8>);
        if (a.experts <= 512) return go(route_bwd_kernel<T, SIGMOID, 16>);
        return go(route_bwd_kernel<T, SIGMOID, 32>);
    } else {
        auto of = [&](auto v) -> mxfp4_status {
            return by_logit ? go(route_kernel<T, SIGMOID, decltype(v)::value, true>)
                            : go(route_kernel<T, SIGMOID, decltype(v)::value, false>);
        };
        if (a.experts <= 32) return of(std::integral_constant<int, 1>{});
        if (a.experts <= 64) return of(std::integral_constant<int, 2>{});
        if (a.experts <= 128) return of(std::integral_constant<int, 4>{});
        if (a.experts <= 256) return of(std::integral_constant<int, 8>{});
        if (a.experts <= 512) return of(std::integral_constant<int, 16>{});
        return of(std::integral_constant<int, 32>{});
    }
}

template <bool BWD>
mxfp4_status dispatch_route(const mxfp4::route::Args& a, int dtype, int score, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == MXFP4_DTYPE_BF16)
        return score == MXFP4_SCORE_SIGMOID ? launch_route<BWD, uint16_t, true>(a, st)
                                            : launch_route<BWD, uint16_t, false>(a, st);
    return score == MXFP4_SCORE_SIGMOID ? launch_route<BWD, float, true>(a, st) : launch_route<BWD, float, false>(a, st);
}

// The counting sort's cut of the slots: one CTA, one cluster, or as many CTAs
// as there may be, with as few slots a thread as that takes, up to kMaxRounds.
void plan_runs(int64_t slots, int64_t* run, int* runs, int* rounds) {
    using namespace mxfp4::plan;
    const int64_t most = slots <= kOneCta ? 1 : slots <= kOneCluster ? kPlaceCluster : kMaxRuns;
    const int64_t per = (slots + most * kThreads - 1) / (most * kThreads);   // slots a thread
    *rounds = int(per < 1 ? 1 : (per < kMaxRounds ? per : kMaxRounds));
    const int64_t pass = int64_t(*rounds) * kThreads;
    const int64_t passes = (slots + pass - 1) / pass;
    *run = (passes <= most ? 1 : (passes + most - 1) / most) * pass;
    // a cluster is always whole: its last CTAs may have no slots
    *runs = most == kPlaceCluster ? kPlaceCluster : int(slots < 1 ? 1 : (slots + *run - 1) / *run);
}

mxfp4_status check_rows(const char* what, int64_t tokens, int64_t top_k, int64_t rows, int64_t cols) {
    if (tokens < 0 || rows < 0 || cols < 0) return fail(MXFP4_ERR_INVALID_ARG, "%s: bad geometry", what);
    if (top_k < 1) return fail(MXFP4_ERR_INVALID_ARG, "%s: top_k must be at least 1", what);
    if (top_k > mxfp4::rows::kMaxTopK)
        return fail(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: top_k at most %d", what, mxfp4::rows::kMaxTopK);
    if (tokens >= kIndexEnd || tokens * top_k >= kIndexEnd || rows >= kIndexEnd)
        return fail(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: tokens * top_k and rows must be < 2^31", what);
    return ok();
}

// Warps of one token (log2): more while the tokens alone leave warps of the
// device idle (16 per SM asked for) and every warp still has a piece of
// `piece` columns.
mxfp4::rows::Share share_of(int64_t tokens, int64_t cols, int64_t piece) {
    mxfp4::rows::Share s{0};
    while (s.split < 3 && (tokens << s.split) < int64_t(num_sms()) * 16 && (cols >> s.split) > piece) ++s.split;
    return s;
}

unsigned token_blocks(int64_t tokens, mxfp4::rows::Share s) {
    const int64_t per = (mxfp4::rows::kThreads / 32) >> s.split;
    return unsigned((tokens + per - 1) / per);
}

unsigned padding_blocks(int64_t rows) {
    const int64_t per = mxfp4::rows::kThreads / 32 * mxfp4::rows::kPadRows;
    return unsigned((rows + per - 1) / per);
}

// CTAs of a kernel that walks `items` and looks over `rows` for padding, and
// the rows it looks over at a time: few tokens leave mostly padding, which is
// dealt out evenly, eight rows a CTA or more.
int64_t bulk_grid(int64_t items, int64_t rows, int64_t most, int* pad_rows) {
    int64_t grid = items > (rows + 7) / 8 ? items : (rows + 7) / 8;
    if (grid > most) grid = most;
    const int64_t each = (rows + grid - 1) / grid;
    *pad_rows = int(each < 1 ? 1 : (each < 32 ? each : 32));
    return grid;
}

template <typename TY, typename TO>
mxfp4_status launch_combine(mxfp4::rows::CombineArgs a, cudaStream_t st) {
    using namespace mxfp4::rows;
    if (wide_rows(a.y, a.cols, a.ldy, sizeof(TY)) && wide_rows(a.out, a.cols, a.ldo, sizeof(TO))) {
        // more than a token a CTA and at least 8 KB a token, the ring; 1000 tokens x 2880 f32, top 4, 8.9 us with it and
        // 13.7 without, 300 tokens 4.3 and 3.3, 8000 x 1024 bf16, top 1, 10.6 both, 12000 x 256 bf16, top 2, 16.3 and 4.3
        if (a.tokens > 4 * num_sms() && a.cols * int64_t(a.top_k * sizeof(TY) + sizeof(TO)) >= 8192) {
            CombineBulkArgs k{};
            k.y = static_cast<const uint8_t*>(a.y);
            k.out = a.out;
            k.weights = a.weights;
            k.row_of_slot = a.row_of_slot;
            k.tokens = a.tokens;
            k.rows = a.rows;
            k.ldy = a.ldy * int64_t(sizeof(TY));
            k.ldo = a.ldo;
            k.top_k = a.top_k;
            k.groups = uint32_t((a.top_k + kGroup - 1) / kGroup);
            const int64_t pieces = (a.cols + kSumCols - 1) / kSumCols;
            k.piece_cols = uint32_t(((a.cols + pieces - 1) / pieces + 7) / 8 * 8);
            k.pieces = uint32_t((a.cols + k.piece_cols - 1) / k.piece_cols);
            k.last_cols = uint32_t(a.cols - int64_t(k.pieces - 1) * k.piece_cols);
            k.row_bytes = (k.piece_cols * uint32_t(sizeof(TY)) + 127) & ~127u;
            const uint32_t fit = kSumRingBytes / (kGroup * k.row_bytes);
            k.ring = fit < kSumRingMost ? fit : kSumRingMost;
            k.status = status_word();
            if (!k.status) return fail(MXFP4_ERR_CUDA, "mxfp4_combine: cannot resolve the device status word");
            if (!raise_smem<combine_bulk_kernel<TY, TO>>(kSumRingBytes))
                return fail(MXFP4_ERR_CUDA, "mxfp4_combine: cannot raise the shared-memory limit");
            const size_t smem = size_t(k.ring) * kGroup * k.row_bytes;
            const int64_t most = resident_ctas(combine_bulk_kernel<TY, TO>, kSumThreads, smem);
            return launch("mxfp4_combine", combine_bulk_kernel<TY, TO>, a.tokens < most ? a.tokens : most, kSumThreads, smem, st, 0, k);
        }
        a.share = share_of(a.tokens, a.cols, 256);
        return launch("mxfp4_combine", combine_kernel<TY, TO, 8>, token_blocks(a.tokens, a.share), kThreads, 0, st, 0, a);
    }
    a.share = share_of(a.tokens, a.cols, 32);
    return launch("mxfp4_combine", combine_kernel<TY, TO, 1>, token_blocks(a.tokens, a.share), kThreads, 0, st, 0, a);
}

template <typename TY, typename TD>
mxfp4_status launch_combine_bwd(mxfp4::rows::CombineBwdArgs a, cudaStream_t st) {
    using namespace mxfp4::rows;
    const bool wide = aligned16(a.d) && aligned16(a.y) && aligned16(a.dy) && a.ldd % 16 == 0 && a.ldy % 16 == 0 &&
                      a.lddy % 16 == 0 && a.cols % 8 == 0 && a.cols > 0;
    // rows of more than one step of a warp go through the ring: 8000 tokens x 512 bf16, top 4, 15.9 us with it and 19.5
    // without, 12000 x 256, top 2, 13.5 and 9.8
    if (wide && a.cols > 256) {
        // equal pieces of the rows whose stage fits, whole 8 columns each
        const int64_t bytes = a.cols * int64_t(sizeof(TD) + kGroup * sizeof(TY));
        int64_t pieces = bytes > int64_t(kBwdStage) ? bytes / kBwdStage : 1;
        while (a.piece_cols = uint32_t(((a.cols + pieces - 1) / pieces + 7) / 8 * 8),
               bwd_stage<TY, TD>(a.piece_cols).total > kBwdStage)
            ++pieces;
        a.pieces = uint32_t((a.cols + a.piece_cols - 1) / a.piece_cols);
        a.last_cols = uint32_t(a.cols - int64_t(a.pieces - 1) * a.piece_cols);
        a.groups = uint32_t((a.top_k + kGroup - 1) / kGroup);
        a.status = status_word();
        if (!a.status) return fail(MXFP4_ERR_CUDA, "mxfp4_combine_bwd: cannot resolve the device status word");
        const BwdStage stage = bwd_stage<TY, TD>(a.piece_cols);
        const size_t smem = size_t(kBwdRing) * stage.total + stage.y;
        if (!raise_smem<combine_bwd_bulk_kernel<TY, TD>>((kBwdRing + 1) * kBwdStage))
            return fail(MXFP4_ERR_CUDA, "mxfp4_combine_bwd: cannot raise the shared-memory limit");
        const int64_t grid = bulk_grid(a.tokens * a.groups, a.rows,
                                       resident_ctas(combine_bwd_bulk_kernel<TY, TD>, kBwdThreads, smem), &a.pad_rows);
        return launch("mxfp4_combine_bwd", combine_bwd_bulk_kernel<TY, TD>, grid, kBwdThreads, smem, st, 0, a);
    }
    a.share = share_of(a.tokens * a.top_k, a.cols, wide ? 256 : 32);
    a.slot_blocks = token_blocks(a.tokens * a.top_k, a.share);
    const int64_t grid = a.slot_blocks + padding_blocks(a.rows);
    if (wide) return launch("mxfp4_combine_bwd", combine_bwd_kernel<TY, TD, 8>, grid, kThreads, 0, st, 0, a);
    return launch("mxfp4_combine_bwd", combine_bwd_kernel<TY, TD, 1>, grid, kThreads, 0, st, 0, a);
}

// one cluster's work: few pieces and one launch's tensors
bool clip_is_small(const mxfp4_grad_tensor* tensors, int count) {
    using namespace mxfp4::clip;
    if (count > kBatch) return false;
    int64_t pieces = 0;
    for (int i = 0; i < count; ++i) {
        if (tensors[i].numel > int64_t(kSmallPieces) * kPieceBytes) return false;
        pieces += (tensors[i].numel * dtype_bytes(tensors[i].dtype) + kPieceBytes - 1) / kPieceBytes;
    }
    return pieces <= kSmallPieces;
}

int clip_batches(int count) { return count <= 0 ? 1 : (count + mxfp4::clip::kBatch - 1) / mxfp4::clip::kBatch; }

}  // namespace

extern "C" {

mxfp4_status mxfp4_route(const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t ld, const float* bias,
                         const uint8_t* mask, const mxfp4_route_params* p, int32_t* ids, float* weights, void* stream) {
    const mxfp4_status s = check_route("mxfp4_route", logits, dtype, tokens, experts, ld, p);
    if (s != MXFP4_OK) return s;
    if (p->groups < 1 || experts % p->groups)
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_route: groups must divide experts");
    if (p->groups > mxfp4::route::kMaxGroups)
        return fail(MXFP4_ERR_UNSUPPORTED_SHAPE, "mxfp4_route: at most %d groups", mxfp4::route::kMaxGroups);
    if (p->top_groups < 1 || p->top_groups > p->groups)
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_route: top_groups must lie in [1, groups]");
    if (p->group_best != 1 && p->group_best != 2)
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_route: group_best must be 1 or 2");
    if (p->top_k > experts / p->groups * p->top_groups)
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_route: the kept groups have fewer than top_k experts");
    if (tokens == 0) return ok();
    if (!ids || !weights) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_route: null pointer");
    if (!aligned_to(bias, 4) || !aligned_to(ids, 4) || !aligned_to(weights, 4))
        return fail(MXFP4_ERR_MISALIGNED, "mxfp4_route: bias, ids or weights misaligned");
    mxfp4::route::Args a{};
    a.logits = logits;
    a.tokens = tokens;
    a.ld = ld;
    a.experts = int(experts);
    a.top_k = p->top_k;
    a.bias = bias;
    a.mask = mask;
    // keeping every group is the same as having none
    a.groups = p->top_groups == p->groups ? 1 : p->groups;
    a.group_size = int(experts) / a.groups;
    a.group_magic = uint32_t(((1u << 22) + a.group_size - 1) / a.group_size);
    for (a.group_shift = 5; (a.groups << a.group_shift) > 32;) --a.group_shift;
    a.group_lanes = 1 << a.group_shift;
    a.top_groups = p->top_groups == p->groups ? 1 : p->top_groups;
    a.group_best = p->group_best;
    a.renormalise = p->renormalise ? 1 : 0;
    a.scale = p->scale;
    a.ids = ids;
    a.weights = weights;
    return dispatch_route<false>(a, dtype, p->score, stream);
}

mxfp4_status mxfp4_route_bwd(const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t ld,
                             const int32_t* ids, const float* d_weights, const mxfp4_route_params* p, void* d_logits,
                             int64_t ldd, void* stream) {
    const mxfp4_status s = check_route("mxfp4_route_bwd", logits, dtype, tokens, experts, ld, p);
    if (s != MXFP4_OK) return s;
    if (ldd < experts) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_route_bwd: bad geometry");
    if (tokens == 0) return ok();
    if (!ids || !d_weights || !d_logits) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_route_bwd: null pointer");
    if (!aligned_to(ids, 4) || !aligned_to(d_weights, 4) || !aligned_to(d_logits, uintptr_t(dtype_bytes(dtype))))
        return fail(MXFP4_ERR_MISALIGNED, "mxfp4_route_bwd: ids, d_weights or d_logits misaligned");
    mxfp4::route::Args a{};
    a.logits = logits;
    a.tokens = tokens;
    a.ld = ld;
    a.experts = int(experts);
    a.top_k = p->top_k;
    a.renormalise = p->renormalise ? 1 : 0;
    a.scale = p->scale;
    a.ids_in = ids;
    a.d_weights = d_weights;
    a.d_logits = d_logits;
    a.ldd = ldd;
    return dispatch_route<true>(a, dtype, p->score, stream);
}

int64_t mxfp4_expert_plan_rows(int64_t tokens, int64_t top_k, int64_t experts, int64_t align) {
    if (tokens <= 0 || top_k <= 0 || experts <= 0 || align <= 0 || tokens >= kIndexEnd || top_k >= kIndexEnd ||
        align >= kIndexEnd)
        return 0;
    const int64_t slots = tokens * top_k;
    const int64_t used = experts < slots ? experts : slots;
    if (used > (INT64_MAX - slots) / align) return 0;
    return (slots + used * (align - 1)) / align * align;
}

size_t mxfp4_expert_plan_workspace(int64_t tokens, int64_t top_k, int64_t experts) {
    if (tokens <= 0 || top_k <= 0 || experts <= 0 || experts > mxfp4::plan::kMaxExperts || tokens >= kIndexEnd ||
        top_k >= kIndexEnd)
        return 0;
    int64_t run;
    int runs, rounds;
    plan_runs(tokens * top_k, &run, &runs, &rounds);
    return tokens * top_k <= mxfp4::plan::kOneCluster ? 0 : mxfp4::plan::hist_bytes(runs, int(experts));
}

mxfp4_status mxfp4_expert_plan(const int32_t* ids, int64_t tokens, int64_t top_k, int64_t experts, int64_t align,
                               int64_t rows, int fill, int32_t* counts, int32_t* offsets, int32_t* row_of_slot,
                               int32_t* slot_of_row, void* workspace, size_t workspace_bytes, void* stream) {
    mxfp4_status s = check_rows("mxfp4_expert_plan", tokens, top_k, rows, 0);
    if (s != MXFP4_OK) return s;
    if (experts < 1) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_expert_plan: experts must be at least 1");
    if (experts > mxfp4::plan::kMaxExperts)
        return fail(MXFP4_ERR_UNSUPPORTED_SHAPE, "mxfp4_expert_plan: at most %d experts", mxfp4::plan::kMaxExperts);
    if (align < 1 || align > 65536 || (align & (align - 1)))
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_expert_plan: align must be a power of two up to 65536");
    if (rows < mxfp4_expert_plan_rows(tokens, top_k, experts, align))
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_expert_plan: rows below mxfp4_expert_plan_rows");
    if (fill && rows % align)
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_expert_plan: fill needs rows to be a multiple of align");
    if (!counts || !offsets || (tokens && (!ids || !row_of_slot)) || (rows && !slot_of_row))
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_expert_plan: null pointer");
    if (!aligned_to(ids, 4) || !aligned_to(counts, 4) || !aligned_to(offsets, 4) || !aligned_to(row_of_slot, 4) ||
        !aligned_to(slot_of_row, 4) || !aligned16(workspace))
        return fail(MXFP4_ERR_MISALIGNED, "mxfp4_expert_plan: pointer misaligned");
    const size_t need = mxfp4_expert_plan_workspace(tokens, top_k, experts);
    if (need && (!workspace || workspace_bytes < need))
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_expert_plan: workspace below mxfp4_expert_plan_workspace");
    mxfp4::plan::Args a{};
    a.ids = ids;
    a.slots = tokens * top_k;
    plan_runs(a.slots, &a.run, &a.runs, &a.rounds);
    a.experts = int(experts);
    for (a.align_log2 = 0; (int64_t(1) << a.align_log2) < align;) ++a.align_log2;
    for (a.bits = 0; (1 << a.bits) < a.experts;) ++a.bits;
    a.rows = rows;
    a.fill = fill ? 1 : 0;
    a.counts = counts;
    a.offsets = offsets;
    a.row_of_slot = row_of_slot;
    a.slot_of_row = slot_of_row;
    a.hist = static_cast<int32_t*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (need) {
        s = launch("mxfp4_expert_plan", mxfp4::plan::plan_count_kernel,
                   mxfp4::plan::clusters(a.runs) * mxfp4::plan::kCluster, mxfp4::plan::kThreads,
                   size_t(mxfp4::plan::hist_row(a.experts)) * 4, st, 0, a);
        if (s != MXFP4_OK) return s;
    }
    using namespace mxfp4::plan;
    if (need) {
        if (!raise_smem<plan_place_kernel<false>>(int(kOnePerSm)))
            return fail(MXFP4_ERR_CUDA, "mxfp4_expert_plan: cannot raise the shared-memory limit");
        return launch("mxfp4_expert_plan", plan_place_kernel<false>, a.runs, kThreads, kOnePerSm, st, 0, a);
    }
    if (a.runs > 1) {
        static std::atomic<uint64_t> allowed{0};   // devices on which clusters of 16 were asked for
        int dev = 0;
        const uint64_t bit = cudaGetDevice(&dev) == cudaSuccess && dev < 64 ? uint64_t(1) << dev : 0;
        if (!(allowed.load() & bit)) {
            if (cudaFuncSetAttribute(plan_place_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
                return fail(MXFP4_ERR_CUDA, "mxfp4_expert_plan: clusters of 16 CTAs are not available");
            allowed.fetch_or(bit);
        }
        return launch("mxfp4_expert_plan", plan_place_kernel<true>, a.runs, kThreads, smem_bytes(a.experts), st,
                      unsigned(a.runs), a);
    }
    return launch("mxfp4_expert_plan", plan_place_kernel<false>, 1, kThreads, smem_bytes(a.experts), st, 0, a);
}

mxfp4_status mxfp4_dispatch(const void* x, int dtype, int64_t tokens, int64_t top_k, int64_t cols, int64_t ldx,
                            const int32_t* row_of_slot, const int32_t* slot_of_row, int64_t rows, void* out,
                            int64_t ldo, void* stream) {
    const mxfp4_status s = check_rows("mxfp4_dispatch", tokens, top_k, rows, cols);
    if (s != MXFP4_OK) return s;
    if (!known_dtype(dtype)) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_dispatch: bad dtype %d", dtype);
    if (ldx < cols || ldo < cols) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_dispatch: bad geometry");
    if (rows == 0 || cols == 0) return ok();
    if ((tokens && (!x || !row_of_slot)) || !slot_of_row || !out)
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_dispatch: null pointer");
    const int esz = dtype_bytes(dtype);
    if (!aligned_to(x, uintptr_t(esz)) || !aligned_to(out, uintptr_t(esz)) || !aligned_to(slot_of_row, 4) ||
        !aligned_to(row_of_slot, 4))
        return fail(MXFP4_ERR_MISALIGNED, "mxfp4_dispatch: pointer misaligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (aligned16(x) && aligned16(out) && (cols * esz) % 16 == 0 && (ldx * esz) % 16 == 0 && (ldo * esz) % 16 == 0) {
        using namespace mxfp4::rows;
        BulkArgs a{};
        a.x = static_cast<const uint8_t*>(x);
        a.out = static_cast<uint8_t*>(out);
        a.ldx = ldx * esz;
        a.ldo = ldo * esz;
        // equal pieces of at most kPiece bytes, whole 16 bytes each
        const int64_t bytes = cols * esz, pieces = (bytes + kPiece - 1) / kPiece;
        a.piece_bytes = uint32_t(((bytes + pieces - 1) / pieces + 15) / 16 * 16);
        a.pieces = uint32_t((bytes + a.piece_bytes - 1) / a.piece_bytes);
        a.last_bytes = uint32_t(bytes - int64_t(a.pieces - 1) * a.piece_bytes);
        a.items = tokens * a.pieces;
        a.tokens = tokens;
        a.rows = rows;
        a.top_k = int(top_k);
        a.row_of_slot = row_of_slot;
        a.slot_of_row = slot_of_row;
        a.status = status_word();
        if (!a.status) return fail(MXFP4_ERR_CUDA, "mxfp4_dispatch: cannot resolve the device status word");
        const size_t smem = size_t(kRing + 1) * ((a.piece_bytes + 127) & ~127u);
        if (!raise_smem<dispatch_bulk_kernel>((kRing + 1) * kPiece))
            return fail(MXFP4_ERR_CUDA, "mxfp4_dispatch: cannot raise the shared-memory limit");
        const int64_t grid = bulk_grid(a.items, rows, resident_ctas(dispatch_bulk_kernel, 32, smem), &a.pad_rows);
        return launch("mxfp4_dispatch", dispatch_bulk_kernel, grid, 32, smem, st, 0, a);
    }
    mxfp4::rows::DispatchArgs a{};
    a.x = static_cast<const uint8_t*>(x);
    a.out = static_cast<uint8_t*>(out);
    a.tokens = tokens;
    a.rows = rows;
    a.top_k = int(top_k);
    a.row_of_slot = row_of_slot;
    a.slot_of_row = slot_of_row;
    a.units = cols;
    a.ldx = ldx;
    a.ldo = ldo;
    a.share = share_of(tokens, a.units, 128);
    a.token_blocks = token_blocks(tokens, a.share);
    const int64_t grid = a.token_blocks + padding_blocks(rows);
    if (esz == 2)
        return launch("mxfp4_dispatch", mxfp4::rows::dispatch_kernel<uint16_t>, grid, mxfp4::rows::kThreads, 0, st, 0, a);
    return launch("mxfp4_dispatch", mxfp4::rows::dispatch_kernel<uint32_t>, grid, mxfp4::rows::kThreads, 0, st, 0, a);
}

mxfp4_status mxfp4_combine(const void* y, int y_dtype, int64_t rows, int64_t cols, int64_t ldy,
                           const int32_t* row_of_slot, const float* weights, int64_t tokens, int64_t top_k, void* out,
                           int out_dtype, int64_t ldo, void* stream) {
    const mxfp4_status s = check_rows("mxfp4_combine", tokens, top_k, rows, cols);
    if (s != MXFP4_OK) return s;
    if (!known_dtype(y_dtype) || !known_dtype(out_dtype)) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_combine: bad dtype");
    if (ldy < cols || ldo < cols) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_combine: bad geometry");
    if (tokens == 0 || cols == 0) return ok();
    if ((rows && !y) || !row_of_slot || !out) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_combine: null pointer");
    if (!aligned_to(y, uintptr_t(dtype_bytes(y_dtype))) || !aligned_to(out, uintptr_t(dtype_bytes(out_dtype))) ||
        !aligned_to(row_of_slot, 4) || !aligned_to(weights, 4))
        return fail(MXFP4_ERR_MISALIGNED, "mxfp4_combine: pointer misaligned");
    mxfp4::rows::CombineArgs a{};
    a.y = y;
    a.out = out;
    a.weights = weights;
    a.row_of_slot = row_of_slot;
    a.tokens = tokens;
    a.rows = rows;
    a.cols = cols;
    a.ldy = ldy;
    a.ldo = ldo;
    a.top_k = int(top_k);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool yb = y_dtype == MXFP4_DTYPE_BF16, ob = out_dtype == MXFP4_DTYPE_BF16;
    if (yb) return ob ? launch_combine<uint16_t, uint16_t>(a, st) : launch_combine<uint16_t, float>(a, st);
    return ob ? launch_combine<float, uint16_t>(a, st) : launch_combine<float, float>(a, st);
}

mxfp4_status mxfp4_combine_bwd(const void* d_out, int d_dtype, int64_t ldd, const void* y, int y_dtype, int64_t rows,
                               int64_t cols, int64_t ldy, const int32_t* row_of_slot, const int32_t* slot_of_row,
                               const float* weights, int64_t tokens, int64_t top_k, void* dy, int64_t lddy,
                               float* d_weights, void* stream) {
    const mxfp4_status s = check_rows("mxfp4_combine_bwd", tokens, top_k, rows, cols);
    if (s != MXFP4_OK) return s;
    if (!known_dtype(d_dtype) || !known_dtype(y_dtype))
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_combine_bwd: bad dtype");
    if (ldd < cols || ldy < cols || lddy < cols) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_combine_bwd: bad geometry");
    if (tokens == 0 && rows == 0) return ok();
    if ((tokens && (!row_of_slot || !weights || !d_weights)) || (rows && !slot_of_row) ||
        (cols && ((tokens && !d_out) || (rows && (!y || !dy)))))
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_combine_bwd: null pointer");
    const uintptr_t de = uintptr_t(dtype_bytes(d_dtype));
    if (!aligned_to(d_out, de) || !aligned_to(dy, de) || !aligned_to(y, uintptr_t(dtype_bytes(y_dtype))) ||
        !aligned_to(row_of_slot, 4) || !aligned_to(slot_of_row, 4) || !aligned_to(weights, 4) || !aligned_to(d_weights, 4))
        return fail(MXFP4_ERR_MISALIGNED, "mxfp4_combine_bwd: pointer misaligned");
    mxfp4::rows::CombineBwdArgs a{};
    a.d = static_cast<const uint8_t*>(d_out);
    a.y = static_cast<const uint8_t*>(y);
    a.dy = static_cast<uint8_t*>(dy);
    a.ldd = ldd * dtype_bytes(d_dtype);
    a.ldy = ldy * dtype_bytes(y_dtype);
    a.lddy = lddy * dtype_bytes(d_dtype);
    a.weights = weights;
    a.d_weights = d_weights;
    a.row_of_slot = row_of_slot;
    a.slot_of_row = slot_of_row;
    a.tokens = tokens;
    a.rows = rows;
    a.cols = cols;
    a.top_k = int(top_k);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool yb = y_dtype == MXFP4_DTYPE_BF16, db = d_dtype == MXFP4_DTYPE_BF16;
    if (yb) return db ? launch_combine_bwd<uint16_t, uint16_t>(a, st) : launch_combine_bwd<uint16_t, float>(a, st);
    return db ? launch_combine_bwd<float, uint16_t>(a, st) : launch_combine_bwd<float, float>(a, st);
}

size_t mxfp4_grad_clip_workspace(const mxfp4_grad_tensor* tensors, int count) {
    return !tensors || count <= 0 || clip_is_small(tensors, count)
               ? 0
               : size_t(clip_batches(count)) * mxfp4::clip::kMaxCtas * sizeof(double);
}

mxfp4_status mxfp4_grad_clip(const mxfp4_grad_tensor* tensors, int count, float max_norm, float* norm, void* workspace,
                             size_t workspace_bytes, void* stream) {
    using namespace mxfp4::clip;
    if (count < 0 || (count && !tensors)) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_grad_clip: null pointer or count < 0");
    if (!(max_norm > 0.0f)) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_grad_clip: max_norm must be positive");
    if (!norm) return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_grad_clip: null norm");
    if (!aligned_to(norm, 4) || !aligned_to(workspace, 8))
        return fail(MXFP4_ERR_MISALIGNED, "mxfp4_grad_clip: norm or workspace misaligned");
    int outputs = -1;   // of the tensors with elements: 1 with outputs, 0 without
    for (int i = 0; i < count; ++i) {
        const mxfp4_grad_tensor& t = tensors[i];
        if (!known_dtype(t.dtype) || t.numel < 0 || (t.numel && !t.grad))
            return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_grad_clip: tensor %d: bad dtype, size or null pointer", i);
        if (t.numel == 0) continue;
        if (outputs >= 0 && (t.out ? 1 : 0) != outputs)
            return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_grad_clip: every tensor has an output, or none");
        outputs = t.out ? 1 : 0;
        if (t.numel >= (int64_t(1) << 36)) return fail(MXFP4_ERR_UNSUPPORTED_SHAPE, "mxfp4_grad_clip: tensor %d too large", i);
        const uintptr_t e = uintptr_t(dtype_bytes(t.dtype));
        if (!aligned_to(t.grad, e) || !aligned_to(t.out, e))
            return fail(MXFP4_ERR_MISALIGNED, "mxfp4_grad_clip: tensor %d misaligned", i);
    }
    const size_t need = mxfp4_grad_clip_workspace(tensors, count);
    if (need && (!workspace || workspace_bytes < need))
        return fail(MXFP4_ERR_INVALID_ARG, "mxfp4_grad_clip: workspace below mxfp4_grad_clip_workspace");
    const bool scale = outputs == 1;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int batches = clip_batches(count);
    Args a{};
    a.partial = static_cast<double*>(workspace);
    a.max_norm = max_norm;
    a.scale = scale ? 1 : 0;
    // one launch's tensors
    auto fill = [&](int b, int chunk_bytes) {
        a.count = 0;
        a.chunks = 0;
        for (int i = b * kBatch; i < count && i < (b + 1) * kBatch; ++i) {
            const mxfp4_grad_tensor& s = tensors[i];
            if (!s.numel) continue;
            Tensor& t = a.t[a.count++];
            t.in = s.grad;
            t.out = s.out;
            t.n = s.numel;
            t.first_chunk = a.chunks;
            t.f32 = s.dtype == MXFP4_DTYPE_F32;
            t.shift = s.out && ((reinterpret_cast<uintptr_t>(s.grad) ^ reinterpret_cast<uintptr_t>(s.out)) & 15u) != 0;
            const int64_t most = chunk_bytes / dtype_bytes(s.dtype);
            a.chunks += int32_t((s.numel + most - 1) / most);
        }
    };
    auto ctas = [&](int most) { return a.chunks < 1 ? 1 : (a.chunks < most ? a.chunks : most); };
    if (!need) {
        fill(0, kPieceBytes);
        a.norm = norm;
        return launch("mxfp4_grad_clip", clip_small_kernel, kCluster, kSmallThreads, 0, st, 0, a);
    }
    a.partials = 0;
    for (int b = 0; b < batches; ++b) {
        fill(b, kChunkBytes);
        const int grid = ctas(kMaxCtas);
        a.first_partial = a.partials;
        const mxfp4_status s = launch("mxfp4_grad_clip", norm_kernel, grid, kThreads, 0, st, 0, a);
        if (s != MXFP4_OK) return s;
        a.partials += grid;
    }
    for (int b = 0; b < (scale ? batches : 1); ++b) {
        if (scale) fill(b, kChunkBytes);
        const int grid = scale ? ctas(kScaleCtas) : 1;
        a.norm = b == 0 ? norm : nullptr;
        const mxfp4_status s = launch("mxfp4_grad_clip", scale_kernel, grid, kThreads, 0, st, 0, a);
        if (s != MXFP4_OK) return s;
    }
    return ok();
}

}  // extern "C"
