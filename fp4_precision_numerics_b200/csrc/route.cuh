// route.cuh -- routing of tokens to experts: scores, choice of the top k,
// weights, and the gradient of the weights with respect to the logits.
//
// One warp per token; lane i holds the logits of experts i, i + 32, ...
// The choice is made on 64-bit keys whose integer order is the order of the
// selection scores: the logits themselves where scores are not added to
// anything (softmax and the sigmoid keep their order), else the scores in
// binary64, so that the choice never hangs on the last bits of an
// exponential.  Ties go to the lowest expert index, NaN ranks lowest.
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
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const long long k2 = __shfl_xor_sync(~0u, key, o);
        const int i2 = __shfl_xor_sync(~0u, idx, o);
        if (k2 > key || (k2 == key && i2 < idx)) {
            key = k2;
            idx = i2;
        }
    }
}

template <typename T, bool SIGMOID, int V>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const Args a) {
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
        m = fmaxf(m, l[i]);
        bad |= !(l[i] < INFINITY);
    }
    m = warp_max(m);
    bad = __any_sync(~0u, bad);

    const bool by_logit = !a.bias && (a.groups == 1 || a.group_best == 1);
    double v[V];
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = double(l[i]);
    } else {
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const double x = double(l[i]);
            if (SIGMOID) {
                v[i] = 1.0 / (1.0 + exp(-x));
            } else {
                v[i] = m == -INFINITY ? 0.0 : exp(x - double(m));   // a padding lane adds exp(-inf) = 0
                z += v[i];
            }
        }
        if (!SIGMOID) {
            z = warp_sum(z);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = bad ? double(NAN) : (z > 0.0 ? v[i] / z : 0.0);
        }
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                if (e < a.experts) v[i] += double(a.bias[e]);
            }
        }
    }
    long long key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < a.experts ? key_of(v[i]) : kKeyNone;

    if (a.groups > 1) {
        long long gkey = kKeyNone;   // lane g: group g's score
        for (int g = 0; g < a.groups; ++g) {
            long long b1 = kKeyNone, b2 = kKeyNone;
            int i1 = INT_MAX;
            double v1 = 0.0, v2 = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                if (e >= a.experts || e / a.group_size != g) continue;
                if (key[i] > b1) {
                    b2 = b1, v2 = v1;
                    b1 = key[i], v1 = v[i], i1 = e;
                } else if (key[i] > b2) {
                    b2 = key[i], v2 = v[i];
                }
            }
            long long w1 = b1;
            int wi = i1;
            warp_best(w1, wi);
            double s = __shfl_sync(~0u, v1, wi & 31);   // expert wi is held by lane wi % 32
            if (a.group_best > 1 && a.group_size > 1) {
                const bool mine = i1 == wi;
                long long c = mine ? b2 : b1;
                const double cv = mine ? v2 : v1;
                int cl = lane;
                warp_best(c, cl);
                s += __shfl_sync(~0u, cv, cl);
            }
            if (lane == g) gkey = key_of(s);
        }
        uint32_t kept = 0;
        for (int j = 0; j < a.top_groups; ++j) {
            long long b = gkey;
            int g = lane;
            warp_best(b, g);
            kept |= 1u << g;
            if (lane == g) gkey = kKeyNone;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (e < a.experts && !((kept >> (e / a.group_size)) & 1u)) key[i] = kKeyNone;
        }
    }

    int id = 0;   // lane j: expert of slot j
    for (int j = 0; j < a.top_k; ++j) {
        long long b = kKeyNone;
        int e = INT_MAX;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (key[i] > b) {
                b = key[i];
                e = lane + 32 * i;
            }
        }
        warp_best(b, e);
        if (lane == j) id = e;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i == e) key[i] = kKeyNone;
    }

    const bool live = lane < a.top_k;
    const float x = live ? load_logit(row + id) : -INFINITY;
    float w;
    if (SIGMOID) {
        w = live ? 1.0f / (1.0f + expf(-x)) : 0.0f;
    } else if (a.renormalise) {
        const float mx = warp_max(x);
        w = mx == -INFINITY ? 0.0f : expf(x - mx);
    } else {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) z += m == -INFINITY ? 0.0f : expf(l[i] - m);
        z = warp_sum(z);
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
template <typename T, bool SIGMOID, int V>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const Args a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.tokens) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    T* out = static_cast<T*>(a.d_logits) + t * a.ldd;
    int id = lane < a.top_k ? a.ids_in[t * a.top_k + lane] : -1;
    const bool live = id >= 0 && id < a.experts;
    if (!live) id = -1;
    const bool any = __any_sync(~0u, live);
    const float dw = live ? a.d_weights[t * a.top_k + lane] : 0.0f;
    const float x = live ? load_logit(row + id) : -INFINITY;

    float add = 0.0f;      // lane j: the part of its expert alone
    float every = 0.0f;    // plain softmax: -c D, times s_e
    float m = -INFINITY, inv = 0.0f;
    if (SIGMOID) {
        const float s = live ? 1.0f / (1.0f + expf(-x)) : 0.0f;
        const float r = live ? 1.0f / (1.0f + expf(x)) : 0.0f;   // 1 - s
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
    } else if (any) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (e < a.experts) m = fmaxf(m, load_logit(row + e));
        }
        m = warp_max(m);
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (e < a.experts && m != -INFINITY) z += expf(load_logit(row + e) - m);
        }
        z = warp_sum(z);
        inv = z != 0.0f ? 1.0f / z : 0.0f;
        const float s = live && m != -INFINITY ? expf(x - m) * inv : 0.0f;
        every = -warp_sum(s * dw);
        add = s * dw;
    }
    add *= a.scale;
    every *= a.scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        float g = 0.0f;
        if (!SIGMOID && !a.renormalise && any && e < a.experts && m != -INFINITY)
            g = expf(load_logit(row + e) - m) * inv * every;
        for (int j = 0; j < a.top_k; ++j) {
            const int ej = __shfl_sync(~0u, id, j);
            const float gj = __shfl_sync(~0u, add, j);
            if (ej == e) g += gj;
        }
        if (e < a.experts) store_logit(out + e, g);
    }
}

}  // namespace route
}  // namespace mxfp4
