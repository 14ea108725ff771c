// rows.cuh -- moving token rows into the experts' segments and back:
// dispatch (gather with zero padding rows), combine (weighted sum of a
// token's rows) and the gradient of combine.
//
// Everything here is bound by HBM.  The kernels go by tokens, so a token's
// row is read or written once and its top_k expert rows are touched once
// each; padding rows are found through slot_of_row by blocks of their own.
#pragma once

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

// Streaming forms: what is read or written once should not push the rows that
// are read again out of L2.
template <typename T, int N>
__device__ __forceinline__ void load_once(const T* p, float (&x)[N]) {
    if constexpr (N == 1) {
        Vec<T, 1>::load(p, x);
    } else if constexpr (sizeof(T) == 2) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p + 4));
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}

template <typename U>
__device__ __forceinline__ void store_once(U* p, U v) { __stcs(p, v); }

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
        for (int64_t u = lane; u < units; u += 32) store_once(dst + u, U{});
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
// behind the tokens').  A token's row is read once and written top_k times,
// four pieces of 512 bytes of a warp in flight.  U: the unit of the copy.
template <typename U>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const __grid_constant__ DispatchArgs a) {
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
            if (u0 + 32 * i < a.units) v[i] = __ldcs(src + u0 + 32 * i);
        for (int j = 0; j < a.top_k; ++j) {
            const int32_t r = __shfl_sync(~0u, row, j);
            if (r < 0) continue;
            U* dst = out + int64_t(r) * a.ldo;
#pragma unroll
            for (int i = 0; i < kFly; ++i)
                if (u0 + 32 * i < a.units) store_once(dst + u0 + 32 * i, v[i]);
        }
    }
}

struct CombineArgs {
    const void* y;
    void* out;
    const float* weights;          // [tokens, top_k], null: ones
    const int32_t* row_of_slot;    // [tokens, top_k]
    int64_t tokens, rows, cols, ldy, ldo;
    int top_k;
    Share share;
    // gradient
    const void* d_out;
    int64_t ldd;
    void* dy;
    int64_t lddy;
    float* d_weights;
    const int32_t* slot_of_row;
    int64_t token_blocks;
};

constexpr int kSlots = 4;   // slots whose rows are in flight together

// out[t] = sum over the slots j of w[t, j] y[row(t, j)] in binary32, j ascending; a slot without a row adds nothing.
template <typename TY, typename TO, int N>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineArgs a) {
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
                if (r[q] >= 0) load_once<TY, N>(y + int64_t(r[q]) * a.ldy + c, v[q]);
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

// dy[row(t, j)] = w[t, j] d_out[t], dw[t, j] = <d_out[t], y[row(t, j)]>;
// blocks behind the tokens' zero the rows without a slot.  The products are
// added up per lane, then over the lanes and the warps of the token in a
// fixed order.
template <typename TY, typename TD, int N>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(const __grid_constant__ CombineArgs a) {
    __shared__ float part[kThreads / 32][kSlots];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    TD* dy = static_cast<TD*>(a.dy);
    if (int64_t(blockIdx.x) >= a.token_blocks) {
        const int64_t w = (int64_t(blockIdx.x) - a.token_blocks) * (kThreads / 32) + warp;
        if constexpr (N == 1) {
            zero_padding(dy, a.lddy, a.cols, w * kPadRows, a.rows, a.slot_of_row, a.tokens * a.top_k, lane);
        } else {
            constexpr int kPer = 16 / int(sizeof(TD));
            zero_padding(reinterpret_cast<uint4*>(dy), a.lddy / kPer, a.cols / kPer, w * kPadRows, a.rows, a.slot_of_row,
                         a.tokens * a.top_k, lane);
        }
        return;
    }
    const int64_t t = a.share.token();
    const bool live = t < a.tokens;   // idle warps stay for the barriers
    const TY* y = static_cast<const TY*>(a.y);
    const TD* d = static_cast<const TD*>(a.d_out) + (live ? t : 0) * a.ldd;
    int32_t row = live && lane < a.top_k ? a.row_of_slot[t * a.top_k + lane] : -1;
    if (row >= a.rows) row = -1;
    const float w = live && lane < a.top_k ? a.weights[t * a.top_k + lane] : 0.0f;
    const int64_t step = int64_t(32 * N) << a.share.split;
    const int64_t cols = live ? a.cols : 0;
    for (int j0 = 0; j0 < a.top_k; j0 += kSlots) {
        float dot[kSlots], wj[kSlots];
        int32_t r[kSlots];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            dot[q] = 0.0f;
            r[q] = __shfl_sync(~0u, row, (j0 + q) & 31);
            wj[q] = __shfl_sync(~0u, w, (j0 + q) & 31);
            if (j0 + q >= a.top_k) r[q] = -1;
        }
        for (int64_t c = (a.share.part() * 32 + lane) * N; c < cols; c += step) {
            float g[N], v[kSlots][N];
            Vec<TD, N>::load(d + c, g);
#pragma unroll
            for (int q = 0; q < kSlots; ++q)
                if (r[q] >= 0) load_once<TY, N>(y + int64_t(r[q]) * a.ldy + c, v[q]);
#pragma unroll
            for (int q = 0; q < kSlots; ++q) {
                if (r[q] < 0) continue;
                float o[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    dot[q] = fmaf(g[i], v[q][i], dot[q]);
                    o[i] = g[i] * wj[q];
                }
                Vec<TD, N>::store(dy + int64_t(r[q]) * a.lddy + c, o);
            }
        }
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
#pragma unroll
            for (int o = 16; o; o >>= 1) dot[q] += __shfl_xor_sync(~0u, dot[q], o);
        }
        if (a.share.split) {   // the same for the whole CTA
            if (lane == 0) {
#pragma unroll
                for (int q = 0; q < kSlots; ++q) part[warp][q] = dot[q];
            }
            __syncthreads();
            if (a.share.part() == 0 && lane < kSlots) {
                float s = 0.0f;
                for (int i = 0; i < (1 << a.share.split); ++i) s += part[warp + i][lane];
                if (live && j0 + lane < a.top_k) a.d_weights[t * a.top_k + j0 + lane] = s;
            }
            __syncthreads();
        } else if (lane < kSlots && live && j0 + lane < a.top_k) {
            a.d_weights[t * a.top_k + j0 + lane] = lane == 0 ? dot[0] : lane == 1 ? dot[1] : lane == 2 ? dot[2] : dot[3];
        }
    }
}

}  // namespace rows
}  // namespace mxfp4
