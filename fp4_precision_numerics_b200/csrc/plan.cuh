// plan.cuh -- from the experts of every token to the grouped layout: counts,
// segment offsets that are multiples of the GEMMs' alignment, the row of
// every (token, slot) and the slot of every row.
//
// A stable counting sort.  Slots n = t * top_k + j are cut into runs of one
// CTA each; plan_count_kernel leaves a histogram per run, plan_place_kernel
// adds up those before its run, turns the totals into offsets and ranks its
// own slots: a warp ranks 32 slots at a time with one match over the lanes
// and a histogram of its own, kept in slot order, so the layout is the same
// on every call.  A single run needs no first kernel.
#pragma once

#include "common.cuh"

namespace mxfp4 {
namespace plan {

constexpr int kMaxExperts = 1024;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRounds = 8;                              // slots a thread ranks per pass
constexpr int kPass = kThreads * kRounds;               // slots of one pass of a CTA
constexpr int kMaxRuns = 128;

struct Args {
    const int32_t* ids;
    int64_t slots;         // tokens * top_k
    int64_t run;           // slots of one CTA, a multiple of kPass
    int runs;
    int experts, align_log2;
    int64_t rows;
    int fill;
    int32_t* counts;
    int32_t* offsets;
    int32_t* row_of_slot;
    int32_t* slot_of_row;
    int32_t* hist;         // [runs][experts]
};

__host__ __device__ constexpr size_t smem_bytes(int experts) {
    // per-warp histograms (16 bits), bases, totals
    return size_t(kWarps) * experts * 2 + size_t(experts) * 4 * 2 + 64 * 4;
}

__global__ void __launch_bounds__(kThreads) plan_count_kernel(const Args a) {
    extern __shared__ int32_t h[];
    for (int e = threadIdx.x; e < a.experts; e += kThreads) h[e] = 0;
    __syncthreads();
    const int64_t n0 = int64_t(blockIdx.x) * a.run;
    const int64_t n1 = n0 + a.run < a.slots ? n0 + a.run : a.slots;
    for (int64_t n = n0 + threadIdx.x; n < n1; n += kThreads) {
        const int32_t e = a.ids[n];
        if (uint32_t(e) < uint32_t(a.experts)) atomicAdd(&h[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kThreads) a.hist[int64_t(blockIdx.x) * a.experts + e] = h[e];
}

__global__ void __launch_bounds__(kThreads) plan_place_kernel(const Args a) {
    extern __shared__ int32_t sm[];
    int32_t* base = sm;                                   // [experts] next row of this CTA's slots
    int32_t* total = sm + a.experts;                      // [experts]
    int32_t* scan = total + a.experts;                    // [64]
    uint16_t* wh = reinterpret_cast<uint16_t*>(scan + 64);   // [kWarps][experts]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.experts;
    const int64_t n0 = int64_t(blockIdx.x) * a.run;
    const int64_t n1 = n0 + a.run < a.slots ? n0 + a.run : a.slots;
    const int64_t mask = (int64_t(1) << a.align_log2) - 1;

    int32_t id[kRounds], rank[kRounds];
    // ranks of one pass inside each warp's part, and the warps' histograms
    auto rank_pass = [&](int64_t p0) {
        for (int i = tid; i < kWarps * E; i += kThreads) wh[i] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int64_t n = p0 + (warp * kRounds + r) * 32 + lane;
            int32_t e = n < n1 ? a.ids[n] : -1;
            if (uint32_t(e) >= uint32_t(E)) e = -1;
            id[r] = e;
            const uint32_t peers = __match_any_sync(~0u, e);
            const int lead = __ffs(peers) - 1;
            int before = 0;
            if (lane == lead && e >= 0) {
                before = wh[warp * E + e];
                wh[warp * E + e] = uint16_t(before + __popc(peers));
            }
            __syncwarp();
            before = __shfl_sync(~0u, before, lead);
            rank[r] = before + __popc(peers & ((1u << lane) - 1u));
        }
        __syncthreads();
    };

    if (a.runs == 1 && a.run <= kPass) {
        rank_pass(n0);
        for (int e = tid; e < E; e += kThreads) {
            int32_t s = 0;
            for (int w = 0; w < kWarps; ++w) s += wh[w * E + e];
            total[e] = s;
            base[e] = 0;
        }
    } else {
        for (int e = tid; e < E; e += kThreads) {
            int32_t before = 0, all = 0;
            for (int b = 0; b < a.runs; ++b) {
                const int32_t v = a.hist[int64_t(b) * E + e];
                all += v;
                before += b < int(blockIdx.x) ? v : 0;
            }
            total[e] = all;
            base[e] = before;
        }
    }
    __syncthreads();
    // exclusive scan of the padded counts, two experts a thread
    {
        const int e0 = 2 * tid;
        const int32_t p0 = e0 < E ? int32_t((total[e0] + mask) & ~mask) : 0;
        const int32_t p1 = e0 + 1 < E ? int32_t((total[e0 + 1] + mask) & ~mask) : 0;
        int32_t v = p0 + p1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(~0u, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) scan[warp] = v;
        __syncthreads();
        if (warp == 0) {
            int32_t u = lane < kWarps ? scan[lane] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t x = __shfl_up_sync(~0u, u, o);
                if (lane >= o) u += x;
            }
            if (lane < kWarps) scan[32 + lane] = u;
        }
        __syncthreads();
        const int32_t start = v - p0 - p1 + (warp ? scan[32 + warp - 1] : 0);
        const int32_t sum = scan[32 + kWarps - 1];
        if (blockIdx.x == 0) {
            if (e0 < E) a.offsets[e0] = start, a.counts[e0] = total[e0];
            if (e0 + 1 < E) a.offsets[e0 + 1] = start + p0, a.counts[e0 + 1] = total[e0 + 1];
            if (tid == 0) a.offsets[E] = a.fill ? int32_t(a.rows) : sum;
        }
        if (e0 < E) base[e0] += start;
        if (e0 + 1 < E) base[e0 + 1] += start + p0;
        // rows without a slot: each segment's padding, dealt out over the CTAs, and what lies behind the last one
        for (int q = 0; q < 2; ++q) {
            const int e = e0 + q;
            if (e < E && e % a.runs == int(blockIdx.x)) {
                const int32_t s = q ? start + p0 : start, len = q ? p1 : p0;
                for (int32_t r = s + total[e]; r < s + len; ++r) a.slot_of_row[r] = -1;
            }
        }
        for (int64_t r = sum + int64_t(blockIdx.x) * kThreads + tid; r < a.rows; r += int64_t(a.runs) * kThreads)
            a.slot_of_row[r] = -1;
    }
    __syncthreads();
    for (int64_t p0 = n0; p0 < n1; p0 += kPass) {
        if (!(a.runs == 1 && a.run <= kPass)) rank_pass(p0);
        // each warp's first row per expert
        for (int e = tid; e < E; e += kThreads) {
            int32_t s = 0;
            for (int w = 0; w < kWarps; ++w) {
                const int32_t c = wh[w * E + e];
                wh[w * E + e] = uint16_t(s);
                s += c;
            }
            total[e] = s;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int64_t n = p0 + (warp * kRounds + r) * 32 + lane;
            if (n >= n1) continue;
            const int32_t e = id[r];
            int32_t row = -1;
            if (e >= 0) {
                row = base[e] + wh[warp * E + e] + rank[r];
                a.slot_of_row[row] = int32_t(n);
            }
            a.row_of_slot[n] = row;
        }
        __syncthreads();
        for (int e = tid; e < E; e += kThreads) base[e] += total[e];
        __syncthreads();
    }
}

}  // namespace plan
}  // namespace mxfp4
