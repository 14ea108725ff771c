// plan.cuh -- from the experts of every token to the grouped layout: counts,
// segment offsets that are multiples of the GEMMs' alignment, the row of
// every (token, slot) and the slot of every row.
//
// A stable counting sort.  Slots n = t * top_k + j are cut into runs of one
// CTA each.  A placing CTA ranks its slots (a warp 32 at a time, with ballots
// and a histogram of its own, kept in slot order, so the layout is the same on
// every call), learns the slots of every expert before its run and in all,
// turns the totals into offsets and writes.  What bounds it is latency, not
// traffic, so the histograms travel as few steps as the size allows:
//  - up to kOneCta slots, one CTA;
//  - up to kOneCluster, one cluster of sixteen CTAs that read each other's
//    histograms from shared memory: one launch;
//  - beyond, up to kMaxRuns CTAs and a counting kernel before them, which in
//    clusters of eight runs leaves for every run the slots of its cluster
//    before it and for every cluster the total.  The placing kernel starts
//    early and ranks while the other counts: it reads the ids before its own
//    wait, which the counting CTAs have done for it by the time it may start.
//    (With a histogram per run to read, 128 KB a CTA for 256 experts, that
//    took 5.6k of its 19k cycles.)
#pragma once

#include "common.cuh"

namespace mxfp4 {
namespace plan {

constexpr int kMaxExperts = 1024;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRounds = 8;    // slots a thread ranks per pass
constexpr int kMaxRuns = 128;

// Most slots of a plan of one CTA, one a thread (1000 slots over 32 experts
// take it 4.8 us and a cluster 4.5, 4096 over 256 experts 10.8 and 5.3), and
// of one cluster (65536 slots over 32 experts take it 7.4 us on the device and
// 7.7 a call, over 256 experts 9.4 and 9.4; the two launches 6.5 and 7.3 on the
// device and 12.5 a call).
constexpr int64_t kOneCta = kThreads;
constexpr int64_t kOneCluster = int64_t(kThreads) * kMaxRounds * 16;

struct Args {
    const int32_t* ids;
    int64_t slots;         // tokens * top_k
    int64_t run;           // slots of one CTA, whole passes
    int runs;
    int rounds;            // slots a thread ranks per pass; a pass is rounds * kThreads slots
    int experts, align_log2, bits;   // bits: of the largest expert index
    int64_t rows;
    int fill;
    int32_t* counts;
    int32_t* offsets;
    int32_t* row_of_slot;
    int32_t* slot_of_row;
    int32_t* hist;         // [runs][hist_row(experts)] before in the cluster, then [clusters][..] totals; 16-byte aligned
};

// a run's histogram takes whole 16-byte vectors
__host__ __device__ constexpr int hist_row(int experts) { return (experts + 3) & ~3; }

constexpr int kCluster = 8;         // runs of the counting kernel's clusters
constexpr int kPlaceCluster = 16;   // runs of a plan that is one cluster
__host__ __device__ constexpr int clusters(int runs) { return (runs + kCluster - 1) / kCluster; }
__host__ __device__ constexpr size_t hist_bytes(int runs, int experts) {
    return size_t(clusters(runs)) * (kCluster + 1) * size_t(hist_row(experts)) * 4;
}

__host__ __device__ constexpr size_t smem_bytes(int experts) {
    // next row, end and pass count per expert; scan scratch; per-warp histograms (16 bits)
    return size_t(experts) * 4 * 3 + 64 * 4 + size_t(kWarps) * experts * 2;
}

// Shared memory asked for by a placing CTA of several: more than half an SM's.
// They are launched while the counting CTAs still hold their SMs, and would
// otherwise crowd on the SMs that are free (65536 x 8 slots over 256 experts
// 15.4 us so, 11.3 with one an SM).
constexpr size_t kOnePerSm = 118784;

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    plan_count_kernel(const __grid_constant__ Args a) {
    cudaGridDependencySynchronize();             // the ids are written, for the placing CTAs too
    cudaTriggerProgrammaticLaunchCompletion();   // which may take their places now
    extern __shared__ int32_t h[];
    const int row = hist_row(a.experts);
    for (int e = threadIdx.x; e < row; e += kThreads) h[e] = 0;
    __syncthreads();
    const int64_t n0 = int64_t(blockIdx.x) * a.run;
    const int64_t n1 = n0 + a.run < a.slots ? n0 + a.run : a.slots;
#pragma unroll 8
    for (int64_t n = n0 + threadIdx.x; n < n1; n += kThreads) {
        const int32_t e = __ldg(a.ids + n);
        if (uint32_t(e) < uint32_t(a.experts)) atomicAdd(&h[e], 1);
    }
    cluster_sync_all();
    const uint32_t rank = cluster_ctarank();
    int32_t* total = a.hist + int64_t(gridDim.x) * row + int64_t(blockIdx.x / kCluster) * row;
    for (int e = threadIdx.x; e < row; e += kThreads) {
        int32_t v[kCluster], before = 0, all = 0;
#pragma unroll
        for (uint32_t q = 0; q < kCluster; ++q)
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[q]) : "r"(mapa_shared(smem_u32(h + e), q)) : "memory");
#pragma unroll
        for (uint32_t q = 0; q < kCluster; ++q) {
            before += q < rank ? v[q] : 0;
            all += v[q];
        }
        a.hist[int64_t(blockIdx.x) * row + e] = before;
        if (rank == 0) total[e] = all;
    }
    cluster_sync_all();   // no CTA leaves while others read its histogram
}

template <bool CLUSTER>
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
    // one of several CTAs behind plan_count_kernel waits for it below, after its own ranking
    if (CLUSTER || single) cudaGridDependencySynchronize();

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
        // the lanes with the same expert, in rank[]: a ballot for each bit of the index and one for "none", all of them
        // independent
#pragma unroll
        for (int r = 0; r < kMaxRounds; ++r) {
            if (uint32_t(id[r]) >= uint32_t(E)) id[r] = -1;
            const uint32_t none = __ballot_sync(~0u, id[r] < 0);
            rank[r] = int32_t(id[r] < 0 ? none : ~none);
        }
        if (a.rounds == 1) {
            for (int b = 0; b < a.bits; ++b) {
                const int32_t bit = (id[0] >> b) & 1;
                const uint32_t v = __ballot_sync(~0u, bit);
                rank[0] &= int32_t(bit ? v : ~v);
            }
        } else {
            for (int b = 0; b < a.bits; ++b) {
#pragma unroll
                for (int r = 0; r < kMaxRounds; ++r) {
                    const int32_t bit = (id[r] >> b) & 1;
                    const uint32_t v = __ballot_sync(~0u, bit);
                    rank[r] &= int32_t(bit ? v : ~v);
                }
            }
        }
        __syncthreads();
        // the warp's histogram, in slot order
#pragma unroll
        for (int r = 0; r < kMaxRounds; ++r) {
            if (r >= a.rounds) break;
            const uint32_t peers = uint32_t(rank[r]);
            const int lead = __ffs(peers) - 1;
            int before = 0;
            if (lane == lead && id[r] >= 0) {
                before = wh[warp * E + id[r]];
                wh[warp * E + id[r]] = uint16_t(before + __popc(peers));
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
    if constexpr (CLUSTER) {
        cluster_sync_all();
        for (int e = tid; e < E; e += kThreads) {
            int32_t v[kPlaceCluster], before = 0, all = 0;
#pragma unroll
            for (int c = 0; c < kPlaceCluster; ++c) {
                asm volatile("ld.shared::cluster.s32 %0, [%1];"
                             : "=r"(v[c])
                             : "r"(mapa_shared(smem_u32(cnt + e), uint32_t(c)))
                             : "memory");
            }
#pragma unroll
            for (int c = 0; c < kPlaceCluster; ++c) {
                all += v[c];
                before += c < int(blockIdx.x) ? v[c] : 0;
            }
            end[e] = all;
            base[e] = before;
        }
        cluster_sync_all();   // no CTA leaves while others read its counts
    } else if (!single) {
        cudaGridDependencySynchronize();
        // the clusters' totals, at most kMaxRuns / kCluster of them, and what this run's cluster has before it
        const int row = hist_row(E), ncl = clusters(a.runs), own = int(blockIdx.x) / kCluster;
        const int32_t* totals = a.hist + int64_t(ncl) * kCluster * row;
        for (int e = tid; e < E; e += kThreads) {
            int32_t before = __ldcg(a.hist + int64_t(blockIdx.x) * row + e), all = 0;
#pragma unroll
            for (int c = 0; c < kMaxRuns / kCluster; ++c) {
                const int32_t v = c < ncl ? __ldcg(totals + int64_t(c) * row + e) : 0;
                all += v;
                before += c < own ? v : 0;
            }
            end[e] = all;
            base[e] = before;
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
