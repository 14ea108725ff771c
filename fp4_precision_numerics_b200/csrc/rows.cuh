// rows.cuh -- moving token rows into the experts' segments and back:
// dispatch (gather with zero padding rows), combine (weighted sum of a
// token's rows) and the gradient of combine.
//
// Everything here is bound by HBM.  The kernels go by tokens, so a token's
// row is read or written once and its top_k expert rows are touched once
// each; padding rows are found through slot_of_row by blocks of their own.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace mxfp4 {
namespace rows {

constexpr int kThreads = 256;
constexpr int kMaxTopK = 32;

// N consecutive elements of a row, as binary32
template <typename T, int N>
struct Vec;

template <>
struct Vec<float, 1> {
    __device__ __forceinline__ static void load(const float* p, float (&x)[1]) { x[0] = *p; }
    __device__ __forceinline__ static void store(float* p, const float (&x)[1]) { *p = x[0]; }
};
template <>
struct Vec<uint16_t, 1> {
    __device__ __forceinline__ static void load(const uint16_t* p, float (&x)[1]) {
        x[0] = __uint_as_float(uint32_t(*p) << 16);
    }
    __device__ __forceinline__ static void store(uint16_t* p, const float (&x)[1]) {
        uint16_t b;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(x[0]));
        *p = b;
    }
};
template <>
struct Vec<float, 8> {
    __device__ __forceinline__ static void load(const float* p, float (&x)[8]) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ static void store(float* p, const float (&x)[8]) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
};
// two binary32 -> packed bf16, nearest even, `lo` in the low half
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
template <>
struct Vec<uint16_t, 8> {
    __device__ __forceinline__ static void load(const uint16_t* p, float (&x)[8]) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ static void store(uint16_t* p, const float (&x)[8]) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
    }
};

// Read-only form for the expert rows.
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* p, float (&x)[N]) {
    if constexpr (N == 1) {
        Vec<T, 1>::load(p, x);
    } else if constexpr (sizeof(T) == 2) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p + 4));
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}

// How the warps of a CTA share tokens: 2^split of them take the pieces of one
// token's row, so that a few tokens still spread over the SMs.
struct Share {
    int split;   // log2 of the warps of one token
    __device__ __forceinline__ int64_t token() const {
        return int64_t(blockIdx.x) * ((kThreads / 32) >> split) + ((threadIdx.x >> 5) >> split);
    }
    __device__ __forceinline__ int part() const { return (threadIdx.x >> 5) & ((1 << split) - 1); }
};

constexpr int kPadRows = 8;   // rows a warp looks over for padding

// Zero those of a warp's kPadRows rows that have no slot.
template <typename U>
__device__ __forceinline__ void zero_padding(U* out, int64_t ldo, int64_t units, int64_t r0, int64_t rows,
                                             const int32_t* slot_of_row, int64_t slots, int lane) {
    bool mine = lane < kPadRows && r0 + lane < rows;
    if (mine) {
        const int32_t slot = slot_of_row[r0 + lane];
        mine = slot < 0 || int64_t(slot) >= slots;
    }
    uint32_t pad = __ballot_sync(~0u, mine);
    while (pad) {
        const int i = __ffs(pad) - 1;
        pad &= pad - 1;
        U* dst = out + (r0 + i) * ldo;
        for (int64_t u = lane; u < units; u += 32) dst[u] = U{};
    }
}

struct DispatchArgs {
    const uint8_t* x;
    uint8_t* out;
    int64_t tokens, rows, units;   // units of sizeof(U) bytes in a row
    int64_t ldx, ldo;              // row strides in units
    int top_k;
    const int32_t* row_of_slot;
    const int32_t* slot_of_row;
    int64_t token_blocks;
    Share share;
};

// out[row(t, j)] = x[t], and zeros on the rows without a slot (the blocks
// behind the tokens').  A token's row is read once and written top_k times.
// U: the unit of the copy, one element.
template <typename U>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const __grid_constant__ DispatchArgs a) {
    cudaGridDependencySynchronize();
    const int lane = threadIdx.x & 31;
    U* out = reinterpret_cast<U*>(a.out);
    if (int64_t(blockIdx.x) >= a.token_blocks) {
        const int64_t w = (int64_t(blockIdx.x) - a.token_blocks) * (kThreads / 32) + (threadIdx.x >> 5);
        zero_padding(out, a.ldo, a.units, w * kPadRows, a.rows, a.slot_of_row, a.tokens * a.top_k, lane);
        return;
    }
    const int64_t t = a.share.token();
    if (t >= a.tokens) return;
    int32_t row = lane < a.top_k ? a.row_of_slot[t * a.top_k + lane] : -1;
    if (row >= a.rows) row = -1;
    const U* src = reinterpret_cast<const U*>(a.x) + t * a.ldx;
    constexpr int kFly = 4;
    const int64_t step = int64_t(32 * kFly) << a.share.split;
    for (int64_t u0 = a.share.part() * 32 * kFly + lane; u0 - lane < a.units; u0 += step) {
        U v[kFly];
#pragma unroll
        for (int i = 0; i < kFly; ++i)
            if (u0 + 32 * i < a.units) v[i] = src[u0 + 32 * i];
        for (int j = 0; j < a.top_k; ++j) {
            const int32_t r = __shfl_sync(~0u, row, j);
            if (r < 0) continue;
            U* dst = out + int64_t(r) * a.ldo;
#pragma unroll
            for (int i = 0; i < kFly; ++i)
                if (u0 + 32 * i < a.units) dst[u0 + 32 * i] = v[i];
        }
    }
}

// The same for rows whose addresses and length are multiples of 16 bytes, as
// bulk copies: a warp keeps kLoads rows on their way into shared memory and
// sends each that has arrived to its top_k places, lane j to the j-th.  No
// data passes through registers, and every copy is a whole row (or an equal
// part of at most kPiece bytes), which DRAM likes.  Four fifths
// of the traffic are writes; the rows' scattered order costs 6 us of 98.
constexpr int kPiece = 8192;
constexpr int kLoads = 8, kStores = 4, kRing = kLoads + kStores;   // items being loaded, items being stored

struct BulkArgs {
    const uint8_t* x;
    uint8_t* out;
    int64_t ldx, ldo;              // row strides in bytes
    int64_t items;                 // tokens * pieces
    int64_t tokens, rows;
    uint32_t pieces, piece_bytes, last_bytes;   // of a row
    int top_k;
    int pad_rows;                  // rows a CTA looks over for padding at a time, at most 32
    const int32_t* row_of_slot;
    const int32_t* slot_of_row;
    uint32_t* status;
};

__device__ __forceinline__ void bulk_store(void* gdst, const void* smem_src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(gdst), "r"(smem_u32(smem_src)),
                 "r"(bytes)
                 : "memory");
}

// A bulk load of what nothing reads again soon: its lines leave L2 before
// those that are being written (16384 x 2880 bf16, top 4: 98 us without, 93
// with).
__device__ __forceinline__ void bulk_load_once(void* smem_dst, const void* gsrc, uint32_t bytes, uint64_t* bar) {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(smem_dst)),
        "l"(gsrc), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__global__ void __launch_bounds__(32) dispatch_bulk_kernel(const __grid_constant__ BulkArgs a) {
    extern __shared__ __align__(128) uint8_t ring[];   // kRing pieces, then one of zeros
    __shared__ uint64_t full[kRing];
    __shared__ int abort_flag;
    const int lane = threadIdx.x;
    const uint32_t slot_bytes = (a.piece_bytes + 127) & ~127u;
    if (lane == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    uint8_t* zeros = ring + kRing * slot_bytes;
    for (uint32_t i = lane * 16; i < a.piece_bytes; i += 32 * 16) *reinterpret_cast<uint4*>(zeros + i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
    cudaGridDependencySynchronize();
    const uint32_t pieces = a.pieces;
    const int64_t first = blockIdx.x, step = gridDim.x;
    const int64_t mine = first < a.items ? (a.items - first + step - 1) / step : 0;
    auto bytes_of = [&](uint32_t p) { return p + 1 == pieces ? a.last_bytes : a.piece_bytes; };
    auto load = [&](int64_t i) {   // lane 0
        const int64_t item = first + i * step;
        const int64_t t = pieces == 1 ? item : item / pieces;
        const uint32_t p = uint32_t(item - t * pieces), b = uint32_t(i % kRing);
        mbar_arrive_expect_tx(&full[b], bytes_of(p));
        bulk_load_once(ring + b * slot_bytes, a.x + t * a.ldx + int64_t(p) * a.piece_bytes, bytes_of(p), &full[b]);
    };
    auto row_for = [&](int64_t i) {
        const int64_t item = first + i * step;
        const int64_t t = pieces == 1 ? item : item / pieces;
        return i < mine && lane < a.top_k ? __ldg(a.row_of_slot + t * a.top_k + lane) : -1;
    };
    if (lane == 0)
        for (int64_t i = 0; i < kLoads && i < mine; ++i) load(i);
    int32_t next = row_for(0);
    // rows without a slot, while the first loads are under way
    for (int64_t r0 = first * a.pad_rows; r0 < a.rows; r0 += step * a.pad_rows) {
        const bool look = lane < a.pad_rows && r0 + lane < a.rows;
        const int32_t slot = look ? __ldg(a.slot_of_row + r0 + lane) : 0;
        if (look && (slot < 0 || int64_t(slot) >= a.tokens * a.top_k)) {
            uint8_t* dst = a.out + (r0 + lane) * a.ldo;
            for (uint32_t p = 0; p < pieces; ++p) bulk_store(dst + int64_t(p) * a.piece_bytes, zeros, bytes_of(p));
        }
    }
    bulk_commit();
    int64_t i = 0;
    for (; i < mine; ++i) {
        const int32_t row = next;
        next = row_for(i + 1);
        const uint32_t b = uint32_t(i % kRing);
        // the lanes give up together
        if (!__all_sync(~0u, mbar_wait_bounded(&full[b], uint32_t(i / kRing) & 1u, &abort_flag, a.status, kRoleProducer))) break;
        if (row >= 0 && row < a.rows) {
            const int64_t item = first + i * step;
            const uint32_t p = pieces == 1 ? 0u : uint32_t(item % pieces);
            bulk_store(a.out + int64_t(row) * a.ldo + int64_t(p) * a.piece_bytes, ring + b * slot_bytes, bytes_of(p));
        }
        bulk_commit();
        if (i + kLoads < mine) {
            bulk_wait_read<kStores>();   // item i - kStores has left the ring: its place takes item i + kLoads
            __syncwarp();
            if (lane == 0) load(i + kLoads);
        }
    }
    // after an expired wait: the loads still under way land before the CTA's memory is given back, or the limit passes
    const uint64_t t0 = globaltimer_ns();
    for (const int64_t stop = i + kLoads < mine ? i + kLoads : mine; i < stop; ++i)
        while (!mbar_try_wait(&full[i % kRing], uint32_t(i / kRing) & 1u) && globaltimer_ns() - t0 < kWaitBudgetNs) {}
    bulk_wait_all<0>();
}

struct CombineArgs {
    const void* y;
    void* out;
    const float* weights;          // [tokens, top_k], null: ones
    const int32_t* row_of_slot;    // [tokens, top_k]
    int64_t tokens, rows, cols, ldy, ldo;
    int top_k;
    Share share;
};

// Slots whose rows a lane has in flight together.  Four cost registers and so
// warps: 16384 x 2880 f32 rows, top 4, ran 185 us with four (24 warps an SM)
// and 142 us with two.
constexpr int kSlots = 2;

// out[t] = sum over the slots j of w[t, j] y[row(t, j)] in binary32, j ascending; a slot without a row adds nothing.
template <typename TY, typename TO, int N>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineArgs a) {
    cudaGridDependencySynchronize();
    const int lane = threadIdx.x & 31;
    const int64_t t = a.share.token();
    if (t >= a.tokens) return;
    const TY* y = static_cast<const TY*>(a.y);
    TO* out = static_cast<TO*>(a.out) + t * a.ldo;
    int32_t row = lane < a.top_k ? a.row_of_slot[t * a.top_k + lane] : -1;
    if (row >= a.rows) row = -1;
    const float w = lane < a.top_k && a.weights ? a.weights[t * a.top_k + lane] : 1.0f;
    const int64_t step = int64_t(32 * N) << a.share.split;
    for (int64_t c = (a.share.part() * 32 + lane) * N; c - lane * N < a.cols; c += step) {
        float s[N];
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = 0.0f;
        for (int j0 = 0; j0 < a.top_k; j0 += kSlots) {
            float v[kSlots][N];
            int32_t r[kSlots];
#pragma unroll
            for (int q = 0; q < kSlots; ++q) {
                r[q] = __shfl_sync(~0u, row, (j0 + q) & 31);
                if (j0 + q >= a.top_k || c >= a.cols) r[q] = -1;
                if (r[q] >= 0) load_row<TY, N>(y + int64_t(r[q]) * a.ldy + c, v[q]);
            }
#pragma unroll
            for (int q = 0; q < kSlots; ++q) {
                const float wq = __shfl_sync(~0u, w, (j0 + q) & 31);
                if (r[q] < 0) continue;
#pragma unroll
                for (int i = 0; i < N; ++i) s[i] = fmaf(wq, v[q][i], s[i]);
            }
        }
        if (c < a.cols) Vec<TO, N>::store(out + c, s);
    }
}

struct CombineBwdArgs {
    const uint8_t* d;              // d_out
    const uint8_t* y;
    uint8_t* dy;
    int64_t ldd, ldy, lddy;        // row strides in bytes
    const float* weights;
    float* d_weights;
    const int32_t* row_of_slot;
    const int32_t* slot_of_row;
    int64_t tokens, rows, cols;
    int top_k;
    Share share;                   // element-wise kernel
    int64_t slot_blocks;
    uint32_t groups, pieces;       // bulk kernel: groups of slots, pieces of a row
    uint32_t piece_cols, last_cols;
    int pad_rows;                  // rows a CTA looks over for padding at a time, at most 32
    uint32_t* status;
};

// dy[row(t, j)] = w[t, j] d_out[t], dw[t, j] = <d_out[t], y[row(t, j)]>, and
// zeros on the rows without a slot (the blocks behind the slots').  2^split
// warps take one slot, N columns a lane; the products are added up per lane,
// then over the lanes and the warps of the slot in a fixed order.  For short
// rows, and for rows that the kernel below cannot copy.
template <typename TY, typename TD, int N>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(const __grid_constant__ CombineBwdArgs a) {
    cudaGridDependencySynchronize();
    __shared__ float part[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (int64_t(blockIdx.x) >= a.slot_blocks) {
        using U = std::conditional_t<N == 1, TD, uint4>;
        constexpr int64_t kUnit = sizeof(U);
        const int64_t w = (int64_t(blockIdx.x) - a.slot_blocks) * (kThreads / 32) + warp;
        zero_padding(reinterpret_cast<U*>(a.dy), a.lddy / kUnit, a.cols * int64_t(sizeof(TD)) / kUnit, w * kPadRows, a.rows,
                     a.slot_of_row, a.tokens * a.top_k, lane);
        return;
    }
    const int64_t n = a.share.token();                // slot
    const bool live = n < a.tokens * a.top_k;         // idle warps stay for the barrier
    const int64_t row = live ? a.row_of_slot[n] : -1;
    float dot = 0.0f;
    if (row >= 0 && row < a.rows) {
        const float w = a.weights[n];
        const TY* y = reinterpret_cast<const TY*>(a.y + row * a.ldy);
        const TD* d = reinterpret_cast<const TD*>(a.d + n / a.top_k * a.ldd);
        TD* o = reinterpret_cast<TD*>(a.dy + row * a.lddy);
#pragma unroll(N == 1 ? 4 : 1)
        for (int64_t c = (a.share.part() * 32 + lane) * N; c < a.cols; c += int64_t(32 * N) << a.share.split) {
            float g[N], v[N];
            Vec<TD, N>::load(d + c, g);
            Vec<TY, N>::load(y + c, v);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                dot = fmaf(g[i], v[i], dot);
                g[i] *= w;
            }
            Vec<TD, N>::store(o + c, g);
        }
#pragma unroll
        for (int i = 16; i; i >>= 1) dot += __shfl_xor_sync(~0u, dot, i);
    }
    if (a.share.split == 0) {   // the same for the whole CTA
        if (lane == 0 && live) a.d_weights[n] = dot;
        return;
    }
    if (lane == 0) part[warp] = dot;
    __syncthreads();
    if (a.share.part() == 0 && lane == 0 && live) {
        float s = 0.0f;
        for (int i = 0; i < (1 << a.share.split); ++i) s += part[warp + i];
        a.d_weights[n] = s;
    }
}

// The same for rows of whole 16-byte pieces.  A warp of a CTA copies a
// token's d_out row and the y rows of up to kGroup of its slots into a ring of
// shared memory (bulk copies, bounded waits), kGroup warps take a slot each:
// d_out comes from HBM once, the dot product stays in one warp, and the loads
// in flight cost no registers.  The rows without a slot get bulk copies of
// zeros meanwhile.  16384 x 2880 bf16, top 4: 146 us, 6.0 TB/s, with one CTA
// an SM and four stages (153 with two CTAs of three); 164 us with a warp a
// token, two slots at a time in registers, 201 with one.
constexpr int kGroup = 4;
constexpr int kBwdRing = 4;
constexpr int kBwdThreads = 32 * (1 + kGroup);
constexpr uint32_t kBwdStage = 32768;        // bytes of a stage at most

struct BwdStage {                            // offsets inside a stage
    uint32_t y, y_bytes, total;
};

template <typename TY, typename TD>
__host__ __device__ __forceinline__ BwdStage bwd_stage(uint32_t piece_cols) {
    BwdStage s;
    s.y = (piece_cols * uint32_t(sizeof(TD)) + 127) & ~127u;
    s.y_bytes = (piece_cols * uint32_t(sizeof(TY)) + 127) & ~127u;
    s.total = s.y + kGroup * s.y_bytes;
    return s;
}

template <typename TY, typename TD>
__global__ void __launch_bounds__(kBwdThreads, 1) combine_bwd_bulk_kernel(const __grid_constant__ CombineBwdArgs a) {
    extern __shared__ __align__(128) uint8_t ring[];   // kBwdRing stages, then a piece of zeros
    __shared__ uint64_t full[kBwdRing], empty[kBwdRing];
    __shared__ int32_t s_row[kBwdRing][kGroup];
    __shared__ float s_weight[kBwdRing][kGroup];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const BwdStage st = bwd_stage<TY, TD>(a.piece_cols);
    uint8_t* zeros = ring + kBwdRing * st.total;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kBwdRing; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kGroup);
        }
        abort_flag = 0;
        fence_barrier_init();
    }
    for (uint32_t i = threadIdx.x * 16; i < st.y; i += kBwdThreads * 16)
        *reinterpret_cast<uint4*>(zeros + i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncthreads();
    cudaGridDependencySynchronize();
    const int64_t units = a.tokens * a.groups;   // a token's group of slots
    const uint32_t pieces = a.pieces;
    uint32_t it = 0;                             // pieces so far
    if (warp == 0) {
        auto slot_of = [&](int64_t u) {          // lane q: slot of the unit's q-th, -1
            const int64_t t = a.groups == 1 ? u : u / a.groups;
            const int j = int(u - t * a.groups) * kGroup + lane;
            return u < units && lane < kGroup && j < a.top_k ? t * a.top_k + j : int64_t(-1);
        };
        int64_t slot = slot_of(blockIdx.x);
        int32_t next_row = slot >= 0 ? __ldg(a.row_of_slot + slot) : -1;
        float next_w = slot >= 0 ? __ldg(a.weights + slot) : 0.0f;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
            int32_t row = next_row >= a.rows ? -1 : next_row;
            const float w = next_w;
            slot = slot_of(u + gridDim.x);
            next_row = slot >= 0 ? __ldg(a.row_of_slot + slot) : -1;
            next_w = slot >= 0 ? __ldg(a.weights + slot) : 0.0f;
            const int64_t t = a.groups == 1 ? u : u / a.groups;
            const uint32_t live = __ballot_sync(~0u, row >= 0);
            for (uint32_t p = 0; p < pieces && ok; ++p, ++it) {
                const uint32_t b = it % kBwdRing;
                if (it >= kBwdRing)
                    ok = __all_sync(~0u, mbar_wait_bounded(&empty[b], (it / kBwdRing - 1) & 1u, &abort_flag, a.status,
                                                           kRoleProducer));   // the lanes give up together
                if (!ok) break;
                if (lane < kGroup) {
                    s_row[b][lane] = row;
                    s_weight[b][lane] = w;
                }
                __syncwarp();
                const uint32_t cols = p + 1 == pieces ? a.last_cols : a.piece_cols;
                const uint32_t db = cols * uint32_t(sizeof(TD)), yb = cols * uint32_t(sizeof(TY));
                uint8_t* stage = ring + b * st.total;
                if (lane == 0) mbar_arrive_expect_tx(&full[b], live ? db + __popc(live) * yb : 0u);
                __syncwarp();
                const int64_t c0 = int64_t(p) * a.piece_cols;
                if (lane == kGroup && live) bulk_load_once(stage, a.d + t * a.ldd + c0 * int64_t(sizeof(TD)), db, &full[b]);
                if (row >= 0)
                    bulk_load_once(stage + st.y + lane * st.y_bytes, a.y + int64_t(row) * a.ldy + c0 * int64_t(sizeof(TY)), yb,
                              &full[b]);
            }
        }
        for (int64_t r0 = int64_t(blockIdx.x) * a.pad_rows; r0 < a.rows; r0 += int64_t(gridDim.x) * a.pad_rows) {
            const bool look = lane < a.pad_rows && r0 + lane < a.rows;
            const int32_t n = look ? __ldg(a.slot_of_row + r0 + lane) : 0;
            if (look && (n < 0 || int64_t(n) >= a.tokens * a.top_k)) {
                uint8_t* dst = a.dy + (r0 + lane) * a.lddy;
                for (uint32_t p = 0; p < pieces; ++p)
                    bulk_store(dst + int64_t(p) * a.piece_cols * int64_t(sizeof(TD)), zeros,
                               (p + 1 == pieces ? a.last_cols : a.piece_cols) * uint32_t(sizeof(TD)));
            }
        }
        bulk_commit();
        // every load has landed before the CTA's memory is given back
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t i = it > kBwdRing ? it - kBwdRing : 0u; i < it; ++i)
            while (!mbar_try_wait(&full[i % kBwdRing], (i / kBwdRing) & 1u) && globaltimer_ns() - t0 < kWaitBudgetNs) {}
        bulk_wait_all<0>();
        return;
    }
    const int q = warp - 1;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t t = a.groups == 1 ? u : u / a.groups;
        const int j = int(u - t * a.groups) * kGroup + q;
        float dot = 0.0f;
        for (uint32_t p = 0; p < pieces; ++p, ++it) {
            const uint32_t b = it % kBwdRing;
            // the lanes give up together, here and below
            if (!__all_sync(~0u, mbar_wait_bounded(&full[b], (it / kBwdRing) & 1u, &abort_flag, a.status, kRoleEpilogue))) return;
            const int32_t row = s_row[b][q];
            const float w = s_weight[b][q];
            if (row >= 0) {
                const uint8_t* stage = ring + b * st.total;
                const TD* d = reinterpret_cast<const TD*>(stage);
                const TY* y = reinterpret_cast<const TY*>(stage + st.y + q * st.y_bytes);
                TD* o = reinterpret_cast<TD*>(a.dy + int64_t(row) * a.lddy) + int64_t(p) * a.piece_cols;
                const int cols = int(p + 1 == pieces ? a.last_cols : a.piece_cols);
#pragma unroll 2
                for (int c = lane * 8; c < cols; c += 256) {
                    float g[8], v[8];
                    Vec<TD, 8>::load(d + c, g);
                    Vec<TY, 8>::load(y + c, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot = fmaf(g[i], v[i], dot);
                        g[i] *= w;
                    }
                    Vec<TD, 8>::store(o + c, g);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[b]);
        }
#pragma unroll
        for (int i = 16; i; i >>= 1) dot += __shfl_xor_sync(~0u, dot, i);
        if (lane == 0 && j < a.top_k) a.d_weights[t * a.top_k + j] = dot;
    }
}

// combine for rows of whole 16-byte pieces.  A warp copies the rows of up to
// kGroup of a token's slots into a ring of shared memory (bulk copies, bounded
// waits; the next tokens' rows and weights are fetched two tokens ahead), six
// warps add 256 columns of a piece each.  16384 x 2880 f32, top 4: 133 us, 6.4
// TB/s (142 with a warp a token and vector loads); 4000 tokens 34 and 49, where
// the other kernel's warps fill the device 1.1 times.  A token costs a CTA 0.8
// us at least, so short rows stay with the other kernel.
constexpr int kSumWarps = 6;                      // of 256 columns each
constexpr int kSumCols = kSumWarps * 256;         // of a piece at most
constexpr int kSumThreads = 32 * (1 + kSumWarps);
constexpr int kSumRingBytes = 53248;   // four CTAs an SM
constexpr int kSumRingMost = 16;

struct CombineBulkArgs {
    const uint8_t* y;
    void* out;
    const float* weights;
    const int32_t* row_of_slot;
    int64_t tokens, rows, ldy, ldo;       // ldy in bytes, ldo in elements
    int top_k;
    uint32_t groups, pieces, piece_cols, last_cols, ring, row_bytes;   // row_bytes: of a row's piece in a stage
    uint32_t* status;
};

template <typename TY, typename TO>
__global__ void __launch_bounds__(kSumThreads, 4) combine_bulk_kernel(const __grid_constant__ CombineBulkArgs a) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kSumRingMost], empty[kSumRingMost];
    __shared__ int32_t s_row[kSumRingMost][kGroup];
    __shared__ float s_weight[kSumRingMost][kGroup];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t R = a.ring, stage_bytes = kGroup * a.row_bytes;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < R; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kSumWarps);
        }
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    cudaGridDependencySynchronize();
    uint32_t b = 0, phase = 0, it = 0;
    if (warp == 0) {
        bool ok = true;
        // a token's rows and weights are fetched two tokens ahead
        auto row_for = [&](int64_t t) {
            return t < a.tokens && lane < a.top_k ? __ldg(a.row_of_slot + t * a.top_k + lane) : -1;
        };
        auto weight_for = [&](int64_t t) {
            return t < a.tokens && lane < a.top_k && a.weights ? __ldg(a.weights + t * a.top_k + lane) : 1.0f;
        };
        int32_t r1 = row_for(blockIdx.x), r2 = row_for(blockIdx.x + gridDim.x);
        float w1 = weight_for(blockIdx.x), w2 = weight_for(blockIdx.x + gridDim.x);
        for (int64_t t = blockIdx.x; t < a.tokens && ok; t += gridDim.x) {
            const int32_t rows_l = r1 >= a.rows ? -1 : r1;
            const float w_l = w1;
            r1 = r2, w1 = w2;
            r2 = row_for(t + 2 * int64_t(gridDim.x)), w2 = weight_for(t + 2 * int64_t(gridDim.x));
            for (uint32_t p = 0; p < a.pieces && ok; ++p) {
                const uint32_t yb = (p + 1 == a.pieces ? a.last_cols : a.piece_cols) * uint32_t(sizeof(TY));
                for (uint32_t g = 0; g < a.groups; ++g, ++it) {
                    if (it >= R)   // the lanes give up together
                        ok = __all_sync(~0u, mbar_wait_bounded(&empty[b], phase ^ 1u, &abort_flag, a.status, kRoleProducer));
                    if (!ok) break;
                    const int32_t row = __shfl_sync(~0u, rows_l, (g * kGroup + lane) & 31);
                    const float w = __shfl_sync(~0u, w_l, (g * kGroup + lane) & 31);
                    const bool mine = lane < kGroup && g * kGroup + lane < uint32_t(a.top_k) && row >= 0;
                    const uint32_t live = __ballot_sync(~0u, mine);
                    if (lane < kGroup) {
                        s_row[b][lane] = mine ? row : -1;
                        s_weight[b][lane] = w;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(&full[b], __popc(live) * yb);
                    __syncwarp();
                    if (mine)
                        bulk_load_once(ring + b * stage_bytes + lane * a.row_bytes,
                                       a.y + int64_t(row) * a.ldy + int64_t(p) * a.piece_cols * int64_t(sizeof(TY)), yb,
                                       &full[b]);
                    if (++b == R) b = 0, phase ^= 1u;
                }
            }
        }
        // every load has landed before the CTA's memory is given back
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t i = it > R ? it - R : 0u; i < it; ++i)
            while (!mbar_try_wait(&full[i % R], (i / R) & 1u) && globaltimer_ns() - t0 < kWaitBudgetNs) {}
        return;
    }
    // columns of this lane in a piece: 8 together, or for binary32 4 and, 128 behind, 4 (16-byte reads without conflicts)
    constexpr bool kHalves = sizeof(TY) == 4;
    const uint32_t c0 = (warp - 1) * 256 + lane * (kHalves ? 4 : 8);
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        for (uint32_t p = 0; p < a.pieces; ++p) {
            const uint32_t cols = p + 1 == a.pieces ? a.last_cols : a.piece_cols;
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = 0.0f;
            for (uint32_t g = 0; g < a.groups; ++g) {
                if (!__all_sync(~0u, mbar_wait_bounded(&full[b], phase, &abort_flag, a.status, kRoleEpilogue))) return;
                const uint8_t* stage = ring + b * stage_bytes;
#pragma unroll
                for (int q = 0; q < kGroup; ++q) {
                    if (s_row[b][q] < 0) continue;
                    const float w = s_weight[b][q];
                    const TY* y = reinterpret_cast<const TY*>(stage + q * a.row_bytes);
                    if constexpr (kHalves) {
                        if (c0 < cols) {
                            const float4 v = *reinterpret_cast<const float4*>(y + c0);
                            s[0] = fmaf(w, v.x, s[0]), s[1] = fmaf(w, v.y, s[1]);
                            s[2] = fmaf(w, v.z, s[2]), s[3] = fmaf(w, v.w, s[3]);
                        }
                        if (c0 + 128 < cols) {
                            const float4 v = *reinterpret_cast<const float4*>(y + c0 + 128);
                            s[4] = fmaf(w, v.x, s[4]), s[5] = fmaf(w, v.y, s[5]);
                            s[6] = fmaf(w, v.z, s[6]), s[7] = fmaf(w, v.w, s[7]);
                        }
                    } else if (c0 < cols) {
                        float v[8];
                        Vec<TY, 8>::load(y + c0, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) s[i] = fmaf(w, v[i], s[i]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[b]);
                if (++b == R) b = 0, phase ^= 1u;
            }
            TO* o = static_cast<TO*>(a.out) + t * a.ldo + int64_t(p) * a.piece_cols + c0;
            if constexpr (kHalves) {
                if constexpr (sizeof(TO) == 2) {
                    if (c0 < cols) *reinterpret_cast<uint2*>(o) = make_uint2(bf16x2(s[0], s[1]), bf16x2(s[2], s[3]));
                    if (c0 + 128 < cols) *reinterpret_cast<uint2*>(o + 128) = make_uint2(bf16x2(s[4], s[5]), bf16x2(s[6], s[7]));
                } else {
                    if (c0 < cols) *reinterpret_cast<float4*>(o) = make_float4(s[0], s[1], s[2], s[3]);
                    if (c0 + 128 < cols) *reinterpret_cast<float4*>(o + 128) = make_float4(s[4], s[5], s[6], s[7]);
                }
            } else if (c0 < cols) {
                Vec<TO, 8>::store(o, s);
            }
        }
    }
}

}  // namespace rows
}  // namespace mxfp4
