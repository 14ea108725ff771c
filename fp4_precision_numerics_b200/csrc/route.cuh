// route.cuh -- routing of tokens to experts: scores, choice of the top k,
// weights, and the gradient of the weights with respect to the logits.
//
// One warp per token; lane i holds the logits of experts i, i + 32, ...
// Where nothing is added to the scores the choice goes by the logits (softmax
// and the sigmoid keep their order), else by the scores in binary64, so that
// it never hangs on the last bits of an exponential: provisional binary32
// scores decide wherever they are far enough apart.  Ties go to the lowest
// expert index, NaN ranks lowest.
#pragma once

#include "common.cuh"

namespace mxfp4 {
namespace route {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;     // lane j of the token's warp holds slot j
constexpr int kMaxGroups = 32;   // lane g holds group g
constexpr int kWarps = 4;

struct Args {
    const void* logits;
    int64_t tokens, ld;
    int experts, top_k;
    const float* bias;      // may be null
    const uint8_t* mask;    // may be null
    int groups, group_size, top_groups, group_best;
    uint32_t group_magic;   // ceil(2^22 / group_size)
    int group_lanes, group_shift;   // largest power of two <= 32 / groups, and its log2
    int renormalise;
    float scale;
    int32_t* ids;           // [tokens, top_k]
    float* weights;         // [tokens, top_k]
    // backward
    const int32_t* ids_in;
    const float* d_weights;
    void* d_logits;
    int64_t ldd;
};

__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float load_logit(const float* p) { return *p; }

// nearest-even binary32 -> bf16; a NaN stays a NaN
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
    uint16_t b;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
    *p = b;
}
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }

constexpr long long kKeyNone = LLONG_MIN;   // not to be chosen

// Integer whose order is that of the doubles, NaN below -infinity.
__device__ __forceinline__ long long key_of(double v) {
    if (isnan(v)) return kKeyNone + 1;
    const long long b = __double_as_longlong(v + 0.0);   // -0 and +0 are one value
    return b < 0 ? (b ^ 0x7FFFFFFFFFFFFFFFll) : b;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// The largest (key, lowest index) of the warp, in every lane.
__device__ __forceinline__ void warp_best(long long& key, int& idx) {
#pragma unroll 1
    for (int o = 16; o; o >>= 1) {
        const long long k2 = __shfl_xor_sync(~0u, key, o);
        const int i2 = __shfl_xor_sync(~0u, idx, o);
        if (k2 > key || (k2 == key && i2 < idx)) {
            key = k2;
            idx = i2;
        }
    }
}

// ---------------------------------------------------------------------------
// 32-bit keys in the order of binary32 values, for the warp's integer
// reductions: 0 is "not to be chosen", 1 a NaN.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t key32(float v) {
    if (isnan(v)) return 1u;
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 and +0 are one value
    return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    if (key < 0x007FFFFFu) return NAN;   // -infinity's key is 0x007FFFFF
    return __uint_as_float((key >> 31) ? (key & 0x7FFFFFFFu) : ~key);
}

// The largest value whose key, its low bits cut, is `key`; both infinities stay
// what they are (+infinity's key ends in zeros, and above it lie the NaNs).
__device__ __forceinline__ float upper_value(uint32_t key, uint32_t low) {
    return key >= 0xFF800000u ? INFINITY : value_of(key | low);
}

// Group of expert e, e / group_size, by the rounded-up reciprocal 2^22 /
// group_size: it is off by less than 1 / 2^12 for e < 1024 and the quotient
// stays 1 / group_size away from the next integer.
__device__ __forceinline__ int group_of(int e, uint32_t group_magic) { return int((uint32_t(e) * group_magic) >> 22); }

__device__ __forceinline__ double value_of(long long key) {   // of key_of
    return key == kKeyNone + 1 ? double(NAN) : __longlong_as_double(key < 0 ? (key ^ 0x7FFFFFFFFFFFFFFFll) : key);
}

// The provisional scores' exponential and reciprocal: the hardware's
// approximations (2 ulp, results below 2^-126 flushed to 0), which the bound
// on the scores allows for.
__device__ __forceinline__ float fast_exp(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}
__device__ __forceinline__ float fast_sigmoid(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + fast_exp(-x)));
    return y;
}

// sigmoid(x) e^-m for m <= 0: the weights' common factor is taken out before
// they leave binary32 (at x = -88.7).  0 from -708 down, where binary64 ends.
// For rows with a chosen logit below kLowLogit, above which binary32's sigmoid
// has all its bits (taken by every row, 0.1 to 0.5 us of 7 to 13; the test for it 0.1 to 0.2).
constexpr float kLowLogit = -80.0f;
__device__ __forceinline__ float sigmoid_over(float x, float m) {
    const float v = expf(fminf(x, 0.0f) - m) / (1.0f + expf(-fabsf(x)));   // a NaN comes through the second factor
    return x < -708.0f ? 0.0f : v;
}

// Does (k, i) come before (k2, i2) in the order of choice?
__device__ __forceinline__ bool before(long long k, int i, long long k2, int i2) { return k > k2 || (k == k2 && i < i2); }

// ---------------------------------------------------------------------------
// Rows whose binary32 scores lie too close together.  There are few of them,
// but a launch that fits the device in one or two waves ends with them, and
// their code is cold: it is kept short (rolled loops, one exponential), and the
// common cases evaluate only what is in doubt.  8191 tokens x 256 experts in 8
// groups, top 8, 10.4 us without such rows: 29 us with all scores and the
// whole choice in binary64 in registers, 17 with rolled loops over shared
// memory, 12.5 with the two settle_ functions.
// ---------------------------------------------------------------------------
__device__ __noinline__ double exact_sigmoid(float x) { return 1.0 / (1.0 + exp(-double(x))); }

template <typename T>
__device__ __forceinline__ long long exact_key(const Args& a, const T* row, int e) {
    return key_of(exact_sigmoid(load_logit(row + e)) + (a.bias ? double(a.bias[e]) : 0.0));
}

// Join two lanes' best and second best.
__device__ __forceinline__ void join_best(long long& b1, long long& b2, int o) {
    const long long o1 = __shfl_xor_sync(~0u, b1, o), o2 = __shfl_xor_sync(~0u, b2, o);
    b2 = max(max(b2, o2), min(b1, o1));
    b1 = max(b1, o1);
}

// Sigmoid: which of two groups stays, `in` (so far) or `out`, the only two in
// doubt; returns the kept groups.
template <typename T>
__device__ __noinline__ uint32_t settle_groups(const Args& a, const T* row, int lane, uint32_t kept, int in, int out) {
    long long first = 0, key = 0;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const int g = side ? out : in;
        long long b1 = kKeyNone, b2 = kKeyNone;
#pragma unroll 1
        for (int q = lane; q < a.group_size; q += 32) {
            const long long k = exact_key(a, row, g * a.group_size + q);
            b2 = max(b2, min(b1, k));
            b1 = max(b1, k);
        }
        __syncwarp();
#pragma unroll 1
        for (int o = 16; o; o >>= 1) join_best(b1, b2, o);
        key = a.group_best > 1 && a.group_size > 1 ? key_of(value_of(b1) + value_of(b2)) : b1;
        if (side == 0) first = key;
    }
    return before(key, out, first, in) ? (kept ^ (1u << in)) | (1u << out) : kept;
}

// Sigmoid: the order of the top_k + 1 experts in lanes 0..top_k (-1: none),
// which hold the whole choice; returns slot j's in lane j.
template <typename T>
__device__ __noinline__ int settle_picks(const Args& a, const T* row, int lane, int id) {
    if (lane > a.top_k) id = -1;
    long long mine = kKeyNone;
    if (id >= 0) mine = exact_key(a, row, id);
    __syncwarp();
    int rank = 0;
#pragma unroll 1
    for (int j = 0; j <= a.top_k; ++j)
        rank += before(__shfl_sync(~0u, mine, j), __shfl_sync(~0u, id, j), mine, id) ? 1 : 0;
    int out = 0;
#pragma unroll 1
    for (int j = 0; j <= a.top_k; ++j) {
        const int r = __shfl_sync(~0u, rank, j), i = __shfl_sync(~0u, id, j);
        if (r == lane) out = i;
    }
    return out;
}

// Experts of one token by the binary64 selection scores of all of them.
// Called by whole warps; `z` is the warp's [experts] of shared memory, `id`
// the choice by binary32 scores with the first one not chosen in lane top_k.
template <typename T, bool SIGMOID>
__device__ __noinline__ int choose_exact(const Args& a, const T* row, int lane, long long* z, int id) {
    float m = -INFINITY;
    bool bad = false;
    double sum = 1.0;
    if (!SIGMOID) {
#pragma unroll 1
        for (int e = lane; e < a.experts; e += 32) {
            const float l = load_logit(row + e);
            m = fmaxf(m, l);
            bad |= !(l < INFINITY);
        }
        m = warp_max(m);
        bad = __any_sync(~0u, bad);
        sum = 0.0;
    }
#pragma unroll 1
    for (int e = lane; e < a.experts; e += 32) {
        const double x = double(load_logit(row + e));
        const double v = SIGMOID ? exp(-x) : (m == -INFINITY ? 0.0 : exp(x - double(m)));
        if (!SIGMOID) sum += v;
        z[e] = __double_as_longlong(v);
    }
    if (!SIGMOID) sum = warp_sum(sum);
#pragma unroll 1
    for (int e = lane; e < a.experts; e += 32) {
        const double v = __longlong_as_double(z[e]);
        double s = SIGMOID ? 1.0 / (1.0 + v) : v / sum;
        if (!SIGMOID) s = bad ? double(NAN) : (sum > 0.0 ? s : 0.0);
        if (a.bias) s += double(a.bias[e]);
        z[e] = key_of(s);
    }
    __syncwarp();
    if (a.groups > 1) {
        const int g = lane >> a.group_shift, p = lane & (a.group_lanes - 1);
        long long b1 = kKeyNone, b2 = kKeyNone;
        if (g < a.groups) {
#pragma unroll 1
            for (int q = p; q < a.group_size; q += a.group_lanes) {
                const long long k = z[g * a.group_size + q];
                b2 = max(b2, min(b1, k));
                b1 = max(b1, k);
            }
        }
#pragma unroll 1
        for (int o = a.group_lanes >> 1; o; o >>= 1) join_best(b1, b2, o);
        if (a.group_best > 1 && a.group_size > 1 && b1 != kKeyNone) b1 = key_of(value_of(b1) + value_of(b2));
        int rank = 0;   // of this lane's group
#pragma unroll 1
        for (int h = 0; h < a.groups; ++h)
            rank += before(__shfl_sync(~0u, b1, h << a.group_shift), h, b1, g) ? 1 : 0;
        const uint32_t kept = __ballot_sync(~0u, g < a.groups && rank < a.top_groups);
#pragma unroll 1
        for (int e = lane; e < a.experts; e += 32)
            if (!((kept >> (group_of(e, a.group_magic) << a.group_shift)) & 1u)) z[e] = kKeyNone;
        __syncwarp();
    }
    // Most often the binary32 choice and its first loser only change places.
    const int k = a.top_k;
    if (k < 32) {
        if (lane > k) id = -1;
        const long long mine = id >= 0 ? z[id] : kKeyNone;
        int rank = 0;
#pragma unroll 1
        for (int j = 0; j <= k; ++j)
            rank += before(__shfl_sync(~0u, mine, j), __shfl_sync(~0u, id, j), mine, id) ? 1 : 0;
        int out = -1;
        long long key = kKeyNone;
#pragma unroll 1
        for (int j = 0; j <= k; ++j) {
            const int r = __shfl_sync(~0u, rank, j), i = __shfl_sync(~0u, id, j);
            const long long v = __shfl_sync(~0u, mine, j);
            if (r == lane) out = i, key = v;
        }
        const long long last = __shfl_sync(~0u, key, k - 1);
        const int last_id = __shfl_sync(~0u, out, k - 1);
        int ahead = 0;   // experts before the last one chosen
#pragma unroll 1
        for (int e = lane; e < a.experts; e += 32) ahead += z[e] != kKeyNone && before(z[e], e, last, last_id) ? 1 : 0;
        ahead = warp_sum(ahead);
        if (last != kKeyNone && ahead == k - 1) return out;
    }
    id = 0;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        long long b = kKeyNone;
        int e = INT_MAX;
#pragma unroll 1
        for (int q = lane; q < a.experts; q += 32) {
            if (z[q] > b) {
                b = z[q];
                e = q;
            }
        }
        warp_best(b, e);
        if (lane == j) id = e;
        if ((e & 31) == lane) z[e] = kKeyNone;
        __syncwarp();
    }
    return id;
}

// Is the key of a score h known to be above that of a score l, both with their
// low bits cut?  slack + c2 (|h| + |l|) bounds the scores' error.
__device__ __forceinline__ bool clear_scores(uint32_t h, uint32_t l, uint32_t low, float slack, float c2) {
    const float hi = value_of(h & ~low), lo = value_of(l | low);
    return hi - lo > slack + c2 * (fabsf(hi) + fabsf(lo));
}

// The last slot's expert `last`, of key `won`, and its rival are an exact tie,
// the order is certain up to there and others have keys as good: are they all
// ties as well?  Called by whole warps; kept: the groups, ~0 without; m and
// inv: the softmax's largest logit and reciprocal sum.
template <typename T, bool SIGMOID, bool BY_LOGIT>
__device__ __noinline__ bool ties_at_cut(const Args& a, const T* row, int lane, uint32_t kept, float m, float inv,
                                         uint32_t won, int last, uint32_t low, float slack, float c2) {
    const float x0 = load_logit(row + last), b0 = a.bias ? a.bias[last] : 0.0f;
    bool all = true;
#pragma unroll 1
    for (int e = lane; e < a.experts; e += 32) {
        if (!((kept >> (a.groups > 1 ? group_of(e, a.group_magic) : 0)) & 1u)) continue;
        const float x = load_logit(row + e), b = a.bias ? a.bias[e] : 0.0f;
        if (x == x0 && b == b0) continue;
        const float s = BY_LOGIT ? x : (SIGMOID ? fast_sigmoid(x) : fast_exp(x - m) * inv) + b;
        const uint32_t k = isnan(s) ? low + 1u : key32(s) & ~low;
        if (BY_LOGIT) all = all && k != (won & ~low);
        else all = all && (k > (won & ~low) ? clear_scores(k, won, low, slack, c2) : clear_scores(won, k, low, slack, c2));
    }
    __syncwarp();
    return __all_sync(~0u, all);
}

// Experts of one token by its logits, on whole 32-bit keys; for the rare rows
// with different logits that share a shortened key.
template <typename T, int V>
__device__ __noinline__ int choose_by_logit(const Args& a, const T* row, int lane, uint32_t kept) {
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        const bool in = e < a.experts && (a.groups == 1 || ((kept >> group_of(e, a.group_magic)) & 1u));
        key[i] = in ? key32(load_logit(row + e)) : 0u;
    }
    int id = 0;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(~0u, best);
        uint32_t mine = ~0u;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (key[i] == best) mine = uint32_t(lane + 32 * i);
        const int e = int(__reduce_min_sync(~0u, mine));
        if (lane == j) id = e;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i == e) key[i] = 0u;
    }
    return id;
}

__host__ __device__ constexpr int bits_of(int v) { return v <= 1 ? 0 : 1 + bits_of((v + 1) / 2); }

// Sort a lane's keys, largest first: the odd-even merge network, step (P, D)
// of which compares x with x + D.
template <int P, int D, int V>
__device__ __forceinline__ void sort_desc(uint32_t (&k)[V]) {
    if constexpr (P < V) {
#pragma unroll
        for (int x = D % P; x + D < V; ++x) {
            if ((x - D % P) % (2 * D) < D && x / (2 * P) == (x + D) / (2 * P)) {
                const uint32_t hi = max(k[x], k[x + D]), lo = min(k[x], k[x + D]);
                k[x] = hi;
                k[x + D] = lo;
            }
        }
        if constexpr (D > 1) sort_desc<P, D / 2>(k);
        else sort_desc<2 * P, 2 * P>(k);
    }
}

// A lane sorts its keys once; then a slot costs one warp reduction over the
// lanes' first keys, one ballot and the winner's step to its next key.  The
// low bits of a key hold V - 1 - i (expert lane + 32 i), so the key names the
// register, the ballot the lane, and equal keys fall to the lowest index.  The
// keys' upper bits are
//  BY_LOGIT (nothing is added to the scores, whose order is the logits'): the
//    logit.  bf16 logits fit whole.  Of binary32 ones the last bits are cut;
//    rows where a cut decided between different logits (equal keys among the
//    winners and the first loser) are redone on whole keys.
//  else: binary32 scores s~ + b by the fast exponential and division, good to
//    c1 max(s) + 2^-24 |s + b| (the exponential of an argument rounded to
//    2^-24: |x| e^-|x| <= 0.37 of a step; 2 ulp each for the instructions;
//    the softmax's sum of up to 1024 terms 37 roundings) plus the cut bits.
//    Where neighbours of the order that matter, or the last group kept and
//    the first one dropped, are further apart than twice that, the order is
//    the exact one; the other rows (about two in a thousand of random ones)
//    are settled in binary64.
// Neighbours with the same logit and the same bias are an exact tie; where the
// last slot and its rival are one, everyone behind them has to be clear of
// them or a tie as well (ties_at_cut: 0.1 us of 7 to 13 where there are none;
// 8191 x 256 bf16 under one bias, with ties in many rows, 8.2 -> 9.9 us).
// Bound by instruction issue and the latency of a row, not by traffic: 8191
// tokens x 256 binary32 logits in 8 groups, sigmoid with bias, top 8, 13.0 us
// (0.7 TB/s), 16384 x 256 top 8 12.8 us, 16384 x 32 bf16 top 4 5.9 us of
// which 2 are the launch.
template <typename T, bool SIGMOID, int V, bool BY_LOGIT>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ Args a) {
    cudaGridDependencySynchronize();
    constexpr bool WHOLE = BY_LOGIT && sizeof(T) == 2;
    constexpr uint32_t LOW = (1u << bits_of(V)) - 1u;
    constexpr float c1 = SIGMOID ? 0x1p-19f : 0x1p-17f, c2 = 0x1p-21f + 0x1p-23f * float(LOW);
    extern __shared__ __align__(16) uint32_t staged[];   // [kWarps][experts] keys, of the groups or of choose_exact
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.tokens) return;
    if (a.mask && !a.mask[t]) {
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = -1;
            a.weights[t * a.top_k + lane] = 0.0f;
        }
        return;
    }
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    float l[V];
    float m = -INFINITY;
    bool bad = false;   // a NaN or +infinity: every softmax score of the row is NaN
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < a.experts ? load_logit(row + e) : -INFINITY;
        if (!SIGMOID) {
            m = fmaxf(m, l[i]);
            bad |= !(l[i] < INFINITY);
        }
    }
    if (!SIGMOID) {
        m = warp_max(m);
        bad = __any_sync(~0u, bad);
    }
    float z = 0.0f;   // softmax: the sum of exp(l - m); of provisional terms where the weights do not need it
    if (!SIGMOID && !a.renormalise) {
#pragma unroll
        for (int i = 0; i < V; ++i) z += m == -INFINITY ? 0.0f : expf(l[i] - m);
        z = warp_sum(z);
    }
    float inv = 1.0f;
    if constexpr (!BY_LOGIT) {
        float s[V];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (SIGMOID) {
                s[i] = fast_sigmoid(l[i]);
            } else {
                s[i] = m == -INFINITY ? 0.0f : fast_exp(l[i] - m);
                sum += s[i];
            }
        }
        if (!SIGMOID) {
            if (a.renormalise) z = warp_sum(sum);
            inv = bad ? NAN : z > 0.0f ? 1.0f / z : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            l[i] = (SIGMOID ? s[i] : s[i] * inv) + (a.bias && e < a.experts ? a.bias[e] : 0.0f);
        }
    }
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        // a NaN's key is LOW + 1 and more, 0 is "not to be chosen"
        const uint32_t k = isnan(l[i]) ? LOW + 1u : key32(l[i]) & ~LOW;
        key[i] = lane + 32 * i < a.experts ? k | uint32_t(V - 1 - i) : 0u;
    }
    const float top = SIGMOID ? 1.0f : (z > 0.0f ? 1.0f / z : 0.0f);   // no score is larger
    bool near = false;   // warp-uniform: the order is not certain

    uint32_t kept = 0;
    if (a.groups > 1) {
        // group_lanes lanes (a power of two) take one group's keys from shared
        // memory and join their two best.
        uint32_t* mine = staged + (threadIdx.x >> 5) * a.experts * (BY_LOGIT ? 1 : 2);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i < a.experts) mine[lane + 32 * i] = key[i] & ~LOW;
        __syncwarp();
        const int g = lane >> a.group_shift, p = lane & (a.group_lanes - 1);
        uint32_t b1 = 0u, b2 = 0u;
        if (g < a.groups) {
            for (int q = p; q < a.group_size; q += a.group_lanes) {
                const uint32_t k = mine[g * a.group_size + q];
                b2 = max(b2, min(b1, k));
                b1 = max(b1, k);
            }
        }
        for (int o = a.group_lanes >> 1; o; o >>= 1) {
            const uint32_t c1st = __shfl_xor_sync(~0u, b1, o), c2nd = __shfl_xor_sync(~0u, b2, o);
            b2 = max(max(b2, c2nd), min(b1, c1st));
            b1 = max(b1, c1st);
        }
        uint32_t gkey = g < a.groups && p == 0 ? b1 : 0u;
        float mag = 0.0f;     // the terms added for a group
        if (!BY_LOGIT && gkey) {
            const float v1 = upper_value(b1, LOW);
            float terms = fabsf(v1);
            if (a.group_best > 1 && a.group_size > 1) {
                const float v2 = upper_value(b2, LOW);
                gkey = key32(v1 + v2);
                terms += fabsf(v2);
            } else {
                gkey = key32(v1);
            }
            if (terms < INFINITY) mag = terms;
        }
        const float sum = value_of(gkey);
        uint32_t last = 0;
        int w = 0;
        bool stays = false;
        for (int j = 0; j < a.top_groups; ++j) {
            last = __reduce_max_sync(~0u, gkey);
            w = __ffs(__ballot_sync(~0u, gkey == last)) - 1;
            kept |= 1u << (w >> a.group_shift);
            if (lane == w) gkey = 0u, stays = true;
        }
        const uint32_t lost = __reduce_max_sync(~0u, gkey);
        if (!BY_LOGIT) {
            mag = warp_max(mag);
            // a sum is off by both terms' errors and its own rounding
            const float lo = value_of(lost), hi = value_of(last);
            const float bound = 2.0f * (c1 * top + c2 * mag);
            near = !(hi - lo > bound);
            if (near && SIGMOID) {
                // only the last group kept and the first one dropped in doubt?
                const uint32_t in = __ballot_sync(~0u, stays && !(sum - lo > bound));
                const uint32_t out = __ballot_sync(~0u, gkey != 0u && !(hi - sum > bound));
                if (__popc(in) == 1 && __popc(out) == 1) {
                    kept = settle_groups<T>(a, row, lane, kept, (__ffs(in) - 1) >> a.group_shift,
                                            (__ffs(out) - 1) >> a.group_shift);
                    near = false;
                }
            }
        } else if (!WHOLE) {
            near = lost == last;   // cut keys: the groups' best may differ
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (!((kept >> min(group_of(lane + 32 * i, a.group_magic), 31)) & 1u)) key[i] = 0u;
    }
    if (BY_LOGIT && !WHOLE && near) {
        // groups by their whole best logits
        near = false;
        kept = 0;
        uint32_t gkey = 0u;
        for (int g = 0; g < a.groups; ++g) {
            uint32_t b = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                if (e < a.experts && group_of(e, a.group_magic) == g) b = max(b, key32(load_logit(row + e)));
            }
            b = __reduce_max_sync(~0u, b);
            if (lane == g) gkey = b;
        }
        for (int j = 0; j < a.top_groups; ++j) {
            const uint32_t b = __reduce_max_sync(~0u, gkey);
            const int w = __ffs(__ballot_sync(~0u, gkey == b)) - 1;
            kept |= 1u << w;
            if (lane == w) gkey = 0u;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            const bool in = e < a.experts && ((kept >> group_of(e, a.group_magic)) & 1u);
            key[i] = in ? (isnan(l[i]) ? LOW + 1u : key32(l[i]) & ~LOW) | uint32_t(V - 1 - i) : 0u;
        }
    }

    sort_desc<1, 1>(key);
    int id = 0;               // lane j: expert of slot j
    uint32_t won = 0u;        // its key
    // one slot more than asked for: what the last one won against
    const int slots = a.top_k + (WHOLE ? 0 : 1);
    int e = -1;
    uint32_t best = 0u;
    for (int j = 0; j < slots; ++j) {
        best = __reduce_max_sync(~0u, key[0]);
        const int w = __ffs(__ballot_sync(~0u, key[0] == best)) - 1;
        e = best ? w + 32 * (V - 1 - int(best & LOW)) : -1;
        if (lane == w) {
#pragma unroll
            for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
            key[V - 1] = 0u;
        }
        if (lane == j) {
            id = e;
            won = best;
        }
    }
    if (!WHOLE) {
        // lane j against lane j + 1; the last winner's rival is still in e and best (lane 31 has no lane above it)
        uint32_t next = __shfl_down_sync(~0u, won, 1);
        int rival = __shfl_down_sync(~0u, id, 1);
        if (lane + 1 == a.top_k) next = best, rival = e;
        const float slack = BY_LOGIT ? 0.0f : c1 * top;
        // is the expert of key `l` known to come after the one of key `h`?
        auto clear = [&](uint32_t h, uint32_t l) {
            return BY_LOGIT ? (h & ~LOW) != (l & ~LOW) : clear_scores(h, l, LOW, slack, c2);
        };
        bool close = lane < a.top_k && rival >= 0 && !clear(won, next);
        // An exact tie is in order, but at the cut it says nothing of the experts behind the rival: one whose key is as
        // good may have the larger score.
        const bool tie = close && load_logit(row + id) == load_logit(row + rival) && (!a.bias || a.bias[id] == a.bias[rival]);
        if (tie && lane + 1 != a.top_k) close = false;
        const bool unsure = near;   // of the groups
        near = near || __any_sync(~0u, close);
        uint32_t rest = 0u, last = 0u;
        if (near) {
            rest = __reduce_max_sync(~0u, key[0]);
            last = __shfl_sync(~0u, won, a.top_k - 1);
            near = unsure || __any_sync(~0u, close && !tie);
            // (a logit's key that is not cut is equal for ties only)
            if (!near && rest != 0u && !clear(last, rest) && !(BY_LOGIT && V == 1))
                near = !ties_at_cut<T, SIGMOID, BY_LOGIT>(a, row, lane, a.groups > 1 ? kept : ~0u, m, inv, last,
                                                          __shfl_sync(~0u, id, a.top_k - 1), LOW, slack, c2);
        }
        if (near) {
            __syncwarp();
            if constexpr (BY_LOGIT) {
                id = choose_by_logit<T, V>(a, row, lane, kept);
            } else {
                if (lane == a.top_k) id = e;
                // do the slots and the first loser hold the whole choice, the last slot being clear of everyone else?
                if (SIGMOID && !unsure && a.top_k < 32 && (rest == 0u || clear(last, rest)))
                    id = settle_picks<T>(a, row, lane, id);
                else
                    id = choose_exact<T, SIGMOID>(a, row, lane,
                                                  reinterpret_cast<long long*>(staged) + (threadIdx.x >> 5) * a.experts, id);
            }
        }
    }

    const bool live = lane < a.top_k;
    const float x = live ? load_logit(row + id) : -INFINITY;
    float w;
    if (SIGMOID) {
        w = live ? 1.0f / (1.0f + expf(-x)) : 0.0f;
        if (__any_sync(~0u, live && x < kLowLogit)) {
            const float mx = a.renormalise ? fminf(warp_max(x), 0.0f) : 0.0f;
            w = sigmoid_over(x, mx);   // 0 where nothing is chosen
        }
    } else if (a.renormalise) {
        const float mx = warp_max(x);
        w = mx == -INFINITY ? 0.0f : expf(x - mx);
    } else {
        w = z > 0.0f ? expf(x - m) / z : 0.0f;
    }
    if (a.renormalise) {
        const float s = warp_sum(live ? w : 0.0f);
        w = s != 0.0f ? w / s : 0.0f;
    }
    if (!SIGMOID && bad) w = NAN;
    if (live) {
        a.ids[t * a.top_k + lane] = id;
        a.weights[t * a.top_k + lane] = w * a.scale;
    }
}

// d logits of the weights, with the scores recomputed from the logits.  With
// p the chosen scores (divided by their sum when renormalised), c = scale
// and D = sum_j p_j dw_j over the slots:
//   softmax, renormalised   c p_j (dw_j - D)           on chosen experts
//   softmax                 c s_e ([e chosen] dw_e - D)   on every expert
//   sigmoid, renormalised   c p_j (1 - s_j) (dw_j - D)  on chosen experts
//   sigmoid                 c s_j (1 - s_j) dw_j        on chosen experts
// A slot whose id lies outside [0, experts) carries no weight.
// 16384 x 128 bf16 top 6, plain softmax, 6.6 us; beyond 512 experts that form
// spills 136 bytes a thread (16384 x 1024 bf16 24.1 us, 2.8 TB/s, against 11.8
// renormalised).
template <typename T, bool SIGMOID, int V>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const __grid_constant__ Args a) {
    cudaGridDependencySynchronize();
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.tokens) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    T* out = static_cast<T*>(a.d_logits) + t * a.ldd;
    const bool whole = !SIGMOID && !a.renormalise;   // every logit gets a gradient, where a slot is live
    int id = lane < a.top_k ? a.ids_in[t * a.top_k + lane] : -1;
    float dw = lane < a.top_k ? a.d_weights[t * a.top_k + lane] : 0.0f;
    float g[V];
    float m = -INFINITY;
    if (whole) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            g[i] = e < a.experts ? load_logit(row + e) : -INFINITY;
            m = fmaxf(m, g[i]);
        }
    }
    const bool live = id >= 0 && id < a.experts;
    const bool any = __any_sync(~0u, live);
    if (!live) id = -1, dw = 0.0f;
    const float x = live ? load_logit(row + id) : -INFINITY;

    float add = 0.0f;      // lane j: what its slot gives its expert
    float base = 0.0f;     // and what the expert gets besides
    if (SIGMOID) {
        float s = live ? 1.0f / (1.0f + expf(-x)) : 0.0f;
        float r = live ? 1.0f / (1.0f + expf(x)) : 0.0f;   // 1 - s
        if (__any_sync(~0u, live && fabsf(x) > -kLowLogit)) {
            const float mx = a.renormalise ? fminf(warp_max(x), 0.0f) : 0.0f;
            s = sigmoid_over(x, mx);   // 0 where nothing is chosen, as is what the other factor is multiplied with
            r = sigmoid_over(-x, 0.0f);
        }
        if (a.renormalise) {
            const float sum = warp_sum(s);
            const float p = sum != 0.0f ? s / sum : 0.0f;
            const float d = warp_sum(p * dw);
            add = p * r * (dw - d);
        } else {
            add = s * r * dw;
        }
    } else if (a.renormalise) {
        const float mx = warp_max(x);
        const float e = mx == -INFINITY ? 0.0f : (live ? expf(x - mx) : 0.0f);
        const float sum = warp_sum(e);
        const float p = sum != 0.0f ? e / sum : 0.0f;
        const float d = warp_sum(p * dw);
        add = p * (dw - d);
    } else {
        m = warp_max(m);
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            g[i] = m == -INFINITY ? 0.0f : expf(g[i] - m);
            z += g[i];
        }
        z = warp_sum(z);
        const float inv = z != 0.0f ? 1.0f / z : 0.0f;
        const float s = live && m != -INFINITY ? expf(x - m) * inv : 0.0f;
        add = s * dw;
        const float d = warp_sum(add) * a.scale;
        base = -s * d;
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] *= -d * inv;
    }
    add *= a.scale;
    // what a chosen expert gets in all, from each slot that names it
    float sum = base;
    for (int j = 0; j < a.top_k; ++j) {
        const int ej = __shfl_sync(~0u, id, j);
        const float gj = __shfl_sync(~0u, add, j);
        if (ej == id) sum += gj;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        if (e < a.experts) store_logit(out + e, whole && any ? g[i] : 0.0f);
    }
    __syncwarp();   // the chosen experts' lanes store over what stands there
    if (live) store_logit(out + id, sum);
}

}  // namespace route
}  // namespace mxfp4
