// clip.cuh -- the global norm of many gradient tensors and their scaling.
//
// norm = sqrt(sum g^2) over all tensors; where norm > max_norm (and finite)
// every gradient is multiplied by max_norm / norm.  Two passes: each CTA
// leaves the sum of squares of its chunks, then each CTA of the second pass
// adds up those partial sums in their order (no atomics: the same bits on
// every call) and scales its chunks.  Squares are summed in binary64.
#pragma once

#include "common.cuh"

namespace mxfp4 {
namespace clip {

constexpr int kThreads = 512;
constexpr int kChunk = 16384;        // elements of one CTA's piece of a tensor
constexpr int kBatch = 96;           // tensors of one launch (their table travels as kernel parameters)
constexpr int kMaxCtas = 592;        // partial sums of one launch

struct Tensor {
    const void* in;
    void* out;
    int64_t n;
    int32_t first_chunk;
    int16_t f32, wide;               // dtype; 16-byte accesses possible
};

struct Args {
    Tensor t[kBatch];
    int count;
    int32_t chunks;
    double* partial;                 // all launches' partial sums
    int partials;                    // how many
    int first_partial;               // this launch's first
    float max_norm;
    float* norm;                     // may be null
    int scale;                       // 0: the norm alone
};

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[kThreads / 32];
    __shared__ double all;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        double s = threadIdx.x < kThreads / 32 ? part[threadIdx.x] : 0.0;
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (threadIdx.x == 0) all = s;
    }
    __syncthreads();
    return all;
}

__device__ __forceinline__ float load_one(const Tensor& t, int64_t i) {
    return t.f32 ? static_cast<const float*>(t.in)[i]
                 : __uint_as_float(uint32_t(static_cast<const uint16_t*>(t.in)[i]) << 16);
}

__device__ __forceinline__ int tensor_of(const Args& a, int32_t chunk) {
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.t[mid].first_chunk <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Args a) {
    double s = 0.0;
    for (int32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const Tensor& t = a.t[tensor_of(a, c)];
        const int64_t i0 = int64_t(c - t.first_chunk) * kChunk;
        const int64_t i1 = i0 + kChunk < t.n ? i0 + kChunk : t.n;
        for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
            const double v = double(load_one(t, i));
            s = fma(v, v, s);
        }
    }
    s = block_sum(s);
    if (threadIdx.x == 0) a.partial[a.first_partial + blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Args a) {
    double s = 0.0;
    for (int i = threadIdx.x; i < a.partials; i += kThreads) s += a.partial[i];
    s = sqrt(block_sum(s));
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.norm) *a.norm = float(s);
    if (!a.scale) return;
    const bool over = s > double(a.max_norm) && s < double(INFINITY);
    const float coef = over ? float(double(a.max_norm) / s) : 1.0f;
    for (int32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const Tensor& t = a.t[tensor_of(a, c)];
        if (!over && t.out == t.in) continue;
        const int64_t i0 = int64_t(c - t.first_chunk) * kChunk;
        const int64_t i1 = i0 + kChunk < t.n ? i0 + kChunk : t.n;
        for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
            const float v = load_one(t, i) * coef;
            if (!over) {   // the same bits, a NaN's too
                if (t.f32) static_cast<uint32_t*>(t.out)[i] = static_cast<const uint32_t*>(t.in)[i];
                else static_cast<uint16_t*>(t.out)[i] = static_cast<const uint16_t*>(t.in)[i];
            } else if (t.f32) {
                static_cast<float*>(t.out)[i] = v;
            } else {
                uint16_t b;
                asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
                static_cast<uint16_t*>(t.out)[i] = b;
            }
        }
    }
}

}  // namespace clip
}  // namespace mxfp4
