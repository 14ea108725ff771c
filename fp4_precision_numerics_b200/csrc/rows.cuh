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

struct DispatchArgs {
    const uint8_t* x;
    uint8_t* out;
    int64_t tokens, rows, units;   // units of sizeof(U) bytes in a row
    int64_t ldx, ldo;              // row strides in units
    int top_k;
    const int32_t* slot_of_row;
};

// out[r] = x[slot_of_row[r] / top_k], zeros where the row has no slot.  U: the unit of the copy.
template <typename U>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t r = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (r >= a.rows) return;
    const int32_t slot = a.slot_of_row[r];
    U* dst = reinterpret_cast<U*>(a.out) + r * a.ldo;
    if (slot < 0 || int64_t(slot) >= a.tokens * a.top_k) {
        for (int64_t i = lane; i < a.units; i += 32) dst[i] = U{};
        return;
    }
    const U* src = reinterpret_cast<const U*>(a.x) + int64_t(slot / a.top_k) * a.ldx;
    for (int64_t i = lane; i < a.units; i += 32) dst[i] = src[i];
}

struct CombineArgs {
    const void* y;
    void* out;
    const float* weights;          // [tokens, top_k], null: ones
    const int32_t* row_of_slot;    // [tokens, top_k]
    int64_t tokens, rows, cols, ldy, ldo;
    int top_k;
    // gradient
    const void* d_out;
    int64_t ldd;
    void* dy;
    int64_t lddy;
    float* d_weights;
    const int32_t* slot_of_row;
    int64_t token_blocks;
};

// out[t] = sum over the slots j of w[t, j] y[row(t, j)] in binary32, j ascending; a slot without a row adds nothing.
template <typename TY, typename TO, int N>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.tokens) return;
    const TY* y = static_cast<const TY*>(a.y);
    TO* out = static_cast<TO*>(a.out) + t * a.ldo;
    int32_t row = lane < a.top_k ? a.row_of_slot[t * a.top_k + lane] : -1;
    if (row >= a.rows) row = -1;
    const float w = lane < a.top_k && a.weights ? a.weights[t * a.top_k + lane] : 1.0f;
    for (int64_t c0 = 0; c0 < a.cols; c0 += 32 * N) {
        const int64_t c = c0 + lane * N;
        float s[N];
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const int32_t r = __shfl_sync(~0u, row, j);
            const float wj = __shfl_sync(~0u, w, j);
            if (r >= 0 && c < a.cols) {
                float v[N];
                Vec<TY, N>::load(y + int64_t(r) * a.ldy + c, v);
#pragma unroll
                for (int i = 0; i < N; ++i) s[i] = fmaf(wj, v[i], s[i]);
            }
        }
        if (c < a.cols) Vec<TO, N>::store(out + c, s);
    }
}

// dy[row(t, j)] = w[t, j] d_out[t], dw[t, j] = <d_out[t], y[row(t, j)]>;
// blocks behind the tokens' zero the rows without a slot.
template <typename TY, typename TD, int N>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(const CombineArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    TD* dy = static_cast<TD*>(a.dy);
    if (int64_t(blockIdx.x) >= a.token_blocks) {
        const int64_t r = (int64_t(blockIdx.x) - a.token_blocks) * (kThreads / 32) + warp;
        if (r >= a.rows) return;
        const int32_t slot = a.slot_of_row[r];
        if (slot >= 0 && int64_t(slot) < a.tokens * a.top_k) return;
        float z[N] = {};
        for (int64_t c = lane * N; c < a.cols; c += 32 * N) Vec<TD, N>::store(dy + r * a.lddy + c, z);
        return;
    }
    const int64_t t = int64_t(blockIdx.x) * (kThreads / 32) + warp;
    if (t >= a.tokens) return;
    const TY* y = static_cast<const TY*>(a.y);
    const TD* d = static_cast<const TD*>(a.d_out) + t * a.ldd;
    for (int j = 0; j < a.top_k; ++j) {
        const int32_t r = a.row_of_slot[t * a.top_k + j];
        float dot = 0.0f;
        if (r >= 0 && r < a.rows) {
            const float w = a.weights ? a.weights[t * a.top_k + j] : 1.0f;
            for (int64_t c = lane * N; c < a.cols; c += 32 * N) {
                float g[N], v[N];
                Vec<TD, N>::load(d + c, g);
                Vec<TY, N>::load(y + int64_t(r) * a.ldy + c, v);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    dot = fmaf(g[i], v[i], dot);
                    g[i] *= w;
                }
                Vec<TD, N>::store(dy + int64_t(r) * a.lddy + c, g);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
        if (lane == 0) a.d_weights[t * a.top_k + j] = dot;
    }
}

}  // namespace rows
}  // namespace mxfp4
