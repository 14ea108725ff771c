// plan.cuh -- from the experts of every token to the grouped layout: counts,
// segment offsets that are multiples of the GEMMs' alignment, the row of
// every (token, slot) and the slot of every row.
//
// A stable counting sort.  Slots n = t * top_k + j are cut into runs of one
// CTA each; plan_count_kernel leaves a histogram per run, plan_place_kernel
// adds up those before its run, turns the totals into offsets and places its
// own slots: a warp ranks 32 slots at a time with one match over the lanes
// and a histogram of its own, kept in slot order, so the layout is the same
// on every call.  A single run needs no first kernel.  What bounds it is
// latency, not traffic: two launches, the second of which starts early and
// ranks its slots while the first still counts.
#pragma once

#include "common.cuh"

namespace mxfp4 {
namespace plan {

constexpr int kMaxExperts = 1024;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRounds = 8;    // slots a thread ranks per pass
constexpr int kMaxRuns = 128;

struct Args {
    const int32_t* ids;
    int64_t slots;         // tokens * top_k
    int64_t run;           // slots of one CTA, whole passes
    int runs;
    int rounds;            // slots a thread ranks per pass; a pass is rounds * kThreads slots
    int experts, align_log2;
    int64_t rows;
    int fill;
    int32_t* counts;
    int32_t* offsets;
    int32_t* row_of_slot;
    int32_t* slot_of_row;
    int32_t* hist;         // [runs][hist_row(experts)], 16-byte aligned
};

// a run's histogram takes whole 16-byte vectors
__host__ __device__ constexpr int hist_row(int experts) { return (experts + 3) & ~3; }

__host__ __device__ constexpr size_t smem_bytes(int experts) {
    // next row, end and pass count per expert; scan scratch; per-warp histograms (16 bits)
    return size_t(experts) * 4 * 3 + 64 * 4 + size_t(kWarps) * experts * 2;
}

__global__ void __launch_bounds__(kThreads) plan_count_kernel(const __grid_constant__ Args a) {
    cudaTriggerProgrammaticLaunchCompletion();
    extern __shared__ int32_t h[];
    const int row = hist_row(a.experts);
    for (int e = threadIdx.x; e < row; e += kThreads) h[e] = 0;
    __syncthreads();
    const int64_t n0 = int64_t(blockIdx.x) * a.run;
    const int64_t n1 = n0 + a.run < a.slots ? n0 + a.run : a.slots;
#pragma unroll 4
    for (int64_t n = n0 + threadIdx.x; n < n1; n += kThreads) {
        const int32_t e = __ldg(a.ids + n);
        if (uint32_t(e) < uint32_t(a.experts)) atomicAdd(&h[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < row; e += kThreads) a.hist[int64_t(blockIdx.x) * row + e] = h[e];
}

__global__ void __launch_bounds__(kThreads) plan_place_kernel(const __grid_constant__ Args a) {
    extern __shared__ int32_t sm[];
    const int E = a.experts;
    int32_t* base = sm;                 // [E] next row of this CTA's slots
    int32_t* end = sm + E;              // [E] slots of the expert, then the end of its rows in use
    int32_t* cnt = sm + 2 * E;          // [E] slots of this pass
    int32_t* scan = sm + 3 * E;         // [64]
    uint16_t* wh = reinterpret_cast<uint16_t*>(scan + 64);   // [kWarps][E] slots, then first place, of each warp
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n0 = int64_t(blockIdx.x) * a.run;
    const int64_t n1 = n0 + a.run < a.slots ? n0 + a.run : a.slots;
    const int pass = a.rounds * kThreads;
    const int32_t mask = (int32_t(1) << a.align_log2) - 1;
    const bool single = a.runs == 1 && a.run <= pass;

    int32_t id[kMaxRounds], rank[kMaxRounds];
    // every slot's place among the pass's slots of its expert: rank in its warp's part, wh[warp] the places before
    auto rank_pass = [&](int64_t p0) {
        const int64_t w0 = p0 + int64_t(warp) * a.rounds * 32 + lane;
#pragma unroll
        for (int r = 0; r < kMaxRounds; ++r) {
            const int64_t n = w0 + r * 32;
            id[r] = r < a.rounds && n < n1 ? __ldg(a.ids + n) : -1;
        }
        uint32_t* z = reinterpret_cast<uint32_t*>(wh);
        for (int i = tid; i < kWarps * E / 2; i += kThreads) z[i] = 0u;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kMaxRounds; ++r) {
            if (r >= a.rounds || w0 - lane + r * 32 >= n1) break;
            int32_t e = id[r];
            if (uint32_t(e) >= uint32_t(E)) e = id[r] = -1;
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
        for (int e = tid; e < E; e += kThreads) {
            int32_t s = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int32_t c = wh[w * E + e];
                wh[w * E + e] = uint16_t(s);
                s += c;
            }
            cnt[e] = s;
            if (single) end[e] = s, base[e] = 0;
        }
        __syncthreads();
    };

    rank_pass(n0);
    if (!single) {
        for (int e = tid; e < E; e += kThreads) end[e] = base[e] = 0;
        __syncthreads();
        cudaGridDependencySynchronize();
        // The runs' histograms, four experts a load and eight loads of a
        // thread in flight; the threads that share experts take every
        // parts-th run (integer sums: any order gives the same).
        const int quads = hist_row(E) / 4;             // at most kThreads / 2
        const int parts = kThreads / quads, part = tid / quads, quad = tid - part * quads;
        if (part < parts) {
            const int4* h = reinterpret_cast<const int4*>(a.hist) + quad;
            int4 all = make_int4(0, 0, 0, 0), before = all;
            for (int b = part; b < a.runs; b += 8 * parts) {
                int4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    v[q] = b + q * parts < a.runs ? __ldcg(h + int64_t(b + q * parts) * quads) : make_int4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int32_t m = b + q * parts < int(blockIdx.x) ? -1 : 0;
                    all.x += v[q].x, all.y += v[q].y, all.z += v[q].z, all.w += v[q].w;
                    before.x += v[q].x & m, before.y += v[q].y & m, before.z += v[q].z & m, before.w += v[q].w & m;
                }
            }
            const int32_t x[4] = {all.x, all.y, all.z, all.w}, y[4] = {before.x, before.y, before.z, before.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (4 * quad + q < E) {
                    atomicAdd(&end[4 * quad + q], x[q]);
                    atomicAdd(&base[4 * quad + q], y[q]);
                }
            }
        }
        __syncthreads();
    }
    // exclusive scan of the padded counts, two experts a thread
    {
        const int e0 = 2 * tid;
        const int32_t t0 = e0 < E ? end[e0] : 0, t1 = e0 + 1 < E ? end[e0 + 1] : 0;
        const int32_t p0 = (t0 + mask) & ~mask, p1 = (t1 + mask) & ~mask;
        int32_t v = p0 + p1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(~0u, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) scan[warp] = v;
        __syncthreads();
        int32_t u = lane < kWarps ? scan[lane] : 0;
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
            const int32_t x = __shfl_up_sync(~0u, u, o);
            if (lane >= o) u += x;
        }
        const int32_t sum = __shfl_sync(~0u, u, kWarps - 1);
        const int32_t start = v - p0 - p1 + (warp ? __shfl_sync(~0u, u, warp - 1) : 0);
        if (e0 < E) base[e0] += start, end[e0] = start + t0;
        if (e0 + 1 < E) base[e0 + 1] += start + p0, end[e0 + 1] = start + p0 + t1;
        if (blockIdx.x == 0) {
            if (e0 < E) a.offsets[e0] = start, a.counts[e0] = t0;
            if (e0 + 1 < E) a.offsets[e0 + 1] = start + p0, a.counts[e0 + 1] = t1;
            if (tid == 0) a.offsets[E] = a.fill ? int32_t(a.rows) : sum;
        }
        __syncthreads();
        // rows without a slot: behind the last segment, and each segment's padding, a warp for an expert
        for (int64_t r = sum + int64_t(blockIdx.x) * kThreads + tid; r < a.rows; r += int64_t(a.runs) * kThreads)
            a.slot_of_row[r] = -1;
        for (int e = int(blockIdx.x) + warp * a.runs; e < E; e += kWarps * a.runs) {
            const int32_t s = end[e], stop = (s + mask) & ~mask;   // segments start on multiples of the alignment
            for (int32_t r = s + lane; r < stop; r += 32) a.slot_of_row[r] = -1;
        }
    }
    for (int64_t p0 = n0; p0 < n1; p0 += pass) {
        if (p0 != n0) rank_pass(p0);
#pragma unroll
        for (int r = 0; r < kMaxRounds; ++r) {
            const int64_t n = p0 + (int64_t(warp) * a.rounds + r) * 32 + lane;
            if (r >= a.rounds || n >= n1) break;
            const int32_t e = id[r];
            int32_t row = -1;
            if (e >= 0) {
                row = base[e] + wh[warp * E + e] + rank[r];
                a.slot_of_row[row] = int32_t(n);
            }
            a.row_of_slot[n] = row;
        }
        __syncthreads();
        for (int e = tid; e < E; e += kThreads) base[e] += cnt[e];
        __syncthreads();
    }
}

}  // namespace plan
}  // namespace mxfp4
