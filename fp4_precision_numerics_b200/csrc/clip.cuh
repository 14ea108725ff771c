// clip.cuh -- the global norm of many gradient tensors and their scaling.
//
// norm = sqrt(sum g^2) over all tensors; where norm > max_norm (and finite)
// every gradient is multiplied by max_norm / norm.  The norm has to be known
// before the first product, so the gradients are read twice: 3 passes of HBM
// traffic against the 2 that on-chip memory for all of them would take.
//  - Two launches: each CTA of the first leaves the sum of squares of its
//    chunks, each CTA of the second adds up those partial sums in their order
//    and scales its chunks, last chunk first, so that it begins with what the
//    first pass left in L2.  24 tensors, 274M binary32 elements: 499 us, 6.6
//    TB/s.  The first runs on CTAs that stay (8 per SM), the second on many
//    short ones, which keep closer to chunk order (543 us with 8 per SM).
//  - Up to kSmallPieces pieces of 4 KB: one launch of one cluster, a warp a
//    piece, with the partial sums exchanged through shared memory; the second
//    reading hits L2.
// No atomics: the same bits on every call.
//
// Squares are taken and added in binary64: neither range nor count costs
// precision, and the norm is off by its one rounding to binary32.  Against
// binary32 sums of 16 elements that is 0.6 us of 8 on the device for small
// lists and 1% of large ones.
#pragma once

#include "common.cuh"

namespace mxfp4 {
namespace clip {

constexpr int kThreads = 256;
constexpr int kVecs = 8;                             // 16-byte vectors a thread has in flight
constexpr int kChunkBytes = kThreads * kVecs * 16;   // one CTA's piece of a tensor
constexpr int kPieceBytes = 32 * kVecs * 16;         // one warp's
constexpr int kCluster = 8, kSmallThreads = 1024;    // of the single launch
constexpr int kSmallPieces = kCluster * kSmallThreads / 32 * 2;
constexpr int kBatch = 96;                           // tensors of one launch (their table travels as kernel parameters)
constexpr int kMaxCtas = 148 * 8;                    // of the first launch: as many partial sums
constexpr int kScaleCtas = 148 * 64;                 // of the second

struct Tensor {
    const void* in;
    void* out;
    int64_t n;
    int32_t first_chunk;
    int16_t f32;         // dtype
    int16_t shift;       // in and out sit differently on 16 bytes: element by element
};

struct Args {
    Tensor t[kBatch];
    int count;
    int32_t chunks;
    double* partial;     // all launches' partial sums
    int partials;        // how many
    int first_partial;   // this launch's first
    float max_norm;
    float* norm;         // may be null
    int scale;           // 0: the norm alone
};

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    return s;
}

// A chunk (of kBytes bytes) as [head elements up to 16 bytes][vectors][tail elements].
struct Piece {
    int64_t first;      // its first element
    int n, head, vecs, per;
};

template <int kBytes>
__device__ __forceinline__ Piece piece_of(const Tensor& t, int32_t chunk, bool shifted) {
    Piece p;
    const int esz = t.f32 ? 4 : 2;
    const int most = kBytes / esz;
    p.per = 16 / esz;
    p.first = int64_t(chunk - t.first_chunk) * most;
    p.n = int(t.n - p.first < most ? t.n - p.first : most);
    const uintptr_t at = reinterpret_cast<uintptr_t>(t.in) + p.first * esz;
    p.head = shifted ? p.n : int((16 - (at & 15)) & 15) / esz;
    if (p.head > p.n) p.head = p.n;
    p.vecs = (p.n - p.head) / p.per;
    return p;
}

// The squares are exact in binary64.
template <bool F32>
__device__ __forceinline__ double squares(const uint4 (&w)[kVecs]) {
    double d[4] = {0.0, 0.0, 0.0, 0.0};   // four chains: an addition takes longer than its issue
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const double hi = double(__uint_as_float(F32 ? u[q] : u[q] & 0xFFFF0000u));
            d[q] = fma(hi, hi, d[q]);
            if (!F32) {
                const double lo = double(__uint_as_float(u[q] << 16));
                d[q] = fma(lo, lo, d[q]);
            }
        }
    }
    return (d[0] + d[1]) + (d[2] + d[3]);
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

// Sum of the squares of thread `tid`'s part of a chunk of N threads.
template <int N>
__device__ __forceinline__ double chunk_squares(const Tensor& t, int32_t chunk, int tid) {
    const Piece p = piece_of<N * kVecs * 16>(t, chunk, false);
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(t.in) +
                                                    (p.first + p.head) * (t.f32 ? 4 : 2));
    uint4 w[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int q = tid + i * N;
        w[i] = q < p.vecs ? v[q] : make_uint4(0u, 0u, 0u, 0u);
    }
    double s = 0.0;
    // what the vectors leave over: fewer than 16 elements a chunk
    const int body = p.vecs * p.per, rest = p.n - body;
    for (int r = tid; r < rest; r += N) {
        const double x = double(load_one(t, p.first + (r < p.head ? r : r + body)));
        s = fma(x, x, s);
    }
    if (tid < p.vecs) s += t.f32 ? squares<true>(w) : squares<false>(w);
    return s;
}

__device__ __forceinline__ uint32_t scaled(uint32_t u, float coef, bool f32) {
    if (f32) return __float_as_uint(__uint_as_float(u) * coef);
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
        : "=r"(d)
        : "f"(__uint_as_float(u & 0xFFFF0000u) * coef), "f"(__uint_as_float(u << 16) * coef));
    return d;
}

// out = in * coef (or in's bits, a NaN's too, where nothing is over) on thread `tid`'s part of a chunk of N threads.
template <int N>
__device__ __forceinline__ void chunk_scale(const Tensor& t, int32_t chunk, int tid, bool over, float coef) {
    const Piece p = piece_of<N * kVecs * 16>(t, chunk, t.shift);
    const bool f32 = t.f32;
    const int64_t at = (p.first + p.head) * (f32 ? 4 : 2);
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(t.in) + at);
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(t.out) + at);
    uint4 w[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int q = tid + i * N;
        if (q < p.vecs) w[i] = v[q];
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int q = tid + i * N;
        if (q >= p.vecs) continue;
        if (over) {
            w[i].x = scaled(w[i].x, coef, f32);
            w[i].y = scaled(w[i].y, coef, f32);
            w[i].z = scaled(w[i].z, coef, f32);
            w[i].w = scaled(w[i].w, coef, f32);
        }
        __stcs(o + q, w[i]);
    }
    const int body = p.vecs * p.per, rest = p.n - body;
    for (int r = tid; r < rest; r += N) {
        const int64_t i = p.first + (r < p.head ? r : r + body);
        if (f32) {
            const uint32_t u = static_cast<const uint32_t*>(t.in)[i];
            static_cast<uint32_t*>(t.out)[i] = over ? scaled(u, coef, true) : u;
        } else {
            const uint32_t u = static_cast<const uint16_t*>(t.in)[i];
            static_cast<uint16_t*>(t.out)[i] = uint16_t(over ? scaled(u, coef, false) : u);
        }
    }
}

__device__ __forceinline__ bool is_over(double norm, float max_norm) {
    return norm > double(max_norm) && float(norm) < INFINITY;   // as the caller reads it
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Args a) {
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();   // the scaling CTAs may take their places and wait
    double s = 0.0;
    int ti = 0;
    for (int32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        while (ti + 1 < a.count && a.t[ti + 1].first_chunk <= c) ++ti;
        s += chunk_squares<kThreads>(a.t[ti], c, threadIdx.x);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) a.partial[a.first_partial + blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Args a) {
    cudaGridDependencySynchronize();
    double s = 0.0;
    for (int i = threadIdx.x; i < a.partials; i += kThreads) s += a.partial[i];
    s = sqrt(block_sum(s));
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.norm) *a.norm = float(s);
    if (!a.scale) return;
    const bool over = is_over(s, a.max_norm);
    const float coef = over ? float(double(a.max_norm) / s) : 1.0f;
    int ti = a.count - 1;
    for (int32_t c = a.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        while (a.t[ti].first_chunk > c) --ti;
        const Tensor& t = a.t[ti];
        if (over || t.out != t.in) chunk_scale<kThreads>(t, c, threadIdx.x, over, coef);
    }
}

// Both passes in one cluster, chunks of kPieceBytes.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSmallThreads)
    clip_small_kernel(const __grid_constant__ Args a) {
    cudaGridDependencySynchronize();
    __shared__ double part[kSmallThreads / 32];
    __shared__ double mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t first = int32_t(blockIdx.x) + warp * kCluster, step = kCluster * kSmallThreads / 32;
    double s = 0.0;
    for (int32_t c = first; c < a.chunks; c += step) s += chunk_squares<32>(a.t[tensor_of(a, c)], c, lane);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (lane == 0) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        s = part[lane];
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (lane == 0) mine = s;
    }
    cluster_sync_all();
    s = 0.0;
#pragma unroll
    for (uint32_t r = 0; r < kCluster; ++r) {
        double v;
        asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(mapa_shared(smem_u32(&mine), r)) : "memory");
        s += v;
    }
    s = sqrt(s);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = float(s);
    cluster_sync_all();   // no CTA leaves while others read its sum
    if (!a.scale) return;
    const bool over = is_over(s, a.max_norm);
    const float coef = over ? float(double(a.max_norm) / s) : 1.0f;
    for (int32_t c = first; c < a.chunks; c += step) {
        const Tensor& t = a.t[tensor_of(a, c)];
        if (over || t.out != t.in) chunk_scale<32>(t, c, lane, over, coef);
    }
}

}  // namespace clip
}  // namespace mxfp4
