// Router of a mixture-of-experts layer for any number of tokens, its gradient, and the sorting of a routing by expert, for
// gfx950.
//
//   s = softmax(z) or sigmoid(z);  rank = s + bias (z without a bias);  the top_k by rank in the top_groups groups of
//   experts whose two largest s + bias sum highest;  w = scale s, or scale s / (sum of the chosen s)
//
// One wave per token, expert e in lane e % 64.  Which of two ranks is larger is decided in binary64, so that a choice does
// not hang on the rounding of s.
#include <cmath>

#include "qk_device.h"
#include "qk_internal.h"

namespace qk {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 64;       // of a workgroup

__device__ __forceinline__ float load_logit(const void* p, int32_t dtype, int64_t i) {
    float v;
    if (dtype == QK_F32) v = static_cast<const float*>(p)[i];
    else if (dtype == QK_F16) v = (float)static_cast<const _Float16*>(p)[i];
    else v = as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    return v == v ? fminf(v, 3.402823466e38f) : -INFINITY;         // a NaN masks as -inf does
}

__device__ __forceinline__ void store_logit(void* p, int32_t dtype, int64_t i, float v) {
    if (dtype == QK_F32) static_cast<float*>(p)[i] = v;
    else if (dtype == QK_F16) static_cast<_Float16*>(p)[i] = (_Float16)v;
    else static_cast<__bf16*>(p)[i] = (__bf16)v;
}

template <class T>
__device__ __forceinline__ T wave_xor(T v, int mask) {
    return __shfl_xor(v, mask, 64);
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = fmax(v, wave_xor(v, m));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += wave_xor(v, m);
    return v;
}

// The place of the largest of v[i] at lane l, as 64 i + l, the lowest of equal ones; best: its value.
template <int V>
__device__ __forceinline__ int wave_argmax(const double (&v)[V], double& best) {
    double m = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmax(m, v[i]);
    best = wave_max(m);
    int at = -1;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) {
        const uint64_t b = __ballot(v[i] == best);
        if (b) at = 64 * i + __builtin_ctzll(b);
    }
    return at;
}

template <int V>
__device__ __forceinline__ double pick(const double (&v)[V], int e) {
    double r = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i)
        if (e >> 6 == i) r = v[i];
    return __shfl(r, e & 63, 64);
}

// softmax: s of every expert, 0 for the masked; sigmoid: the same
template <int V>
__device__ __forceinline__ void scores(const double (&z)[V], bool sigmoid, double (&s)[V]) {
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = 1.0 / (1.0 + exp(-z[i]));
        return;
    }
    double m = z[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmax(m, z[i]);
    m = wave_max(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s[i] = z[i] == -INFINITY ? 0.0 : exp(z[i] - m);
        sum += s[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
}

// Shares of the chosen experts (one a lane; z = -inf: none): s_j / sum of s.  Relative to the largest, so that scores too
// small for a number still have a ratio.
__device__ __forceinline__ double share_of(double z, bool sigmoid) {
    const double top = sigmoid ? fmin(wave_max(z), 0.0) : wave_max(z);
    double r = 0.0;
    if (z != -INFINITY) r = sigmoid && z >= 0.0 ? 1.0 / (1.0 + exp(-z)) : exp(z - top) / (sigmoid ? 1.0 + exp(z) : 1.0);
    const double total = wave_sum(r);
    return total > 0.0 ? r / total : 0.0;
}

template <int V>
__global__ __launch_bounds__(kThreads) void moe_route_kernel(MoeRouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / 64;
    if (t >= a.T) return;
    double z[V], s[V], key[V], ranked[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 64 * i + lane;
        z[i] = e < a.E ? (double)load_logit(a.logits, a.dtype, t * a.E + e) : -INFINITY;
    }
    scores<V>(z, a.score == QK_SIGMOID, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 64 * i + lane;
        float b = a.bias && e < a.E ? a.bias[e] : 0.0f;
        b = b == b ? fminf(b, 3.402823466e38f) : -INFINITY;
        ranked[i] = z[i] == -INFINITY ? -INFINITY : s[i] + (double)b;
        key[i] = a.bias ? ranked[i] : z[i];
    }
    if (a.groups > 1) {
        const int per = a.E / a.groups;
        double mine = -INFINITY;                                    // lane g: the sum of group g's two largest
        for (int g = 0; g < a.groups; ++g) {
            double v[V], best;
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = (64 * i + lane) / per == g ? ranked[i] : -INFINITY;
            const int at = wave_argmax<V>(v, best);
            double sum = best;
            if (best != -INFINITY) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (64 * i + lane == at) v[i] = -INFINITY;
                double second;
                wave_argmax<V>(v, second);
                if (second != -INFINITY) sum += second;
            }
            if (lane == g) mine = sum;
        }
        uint64_t kept = 0;
        for (int j = 0; j < a.top_groups; ++j) {
            const double m[1] = {mine};
            double best;
            const int g = wave_argmax<1>(m, best);
            if (best == -INFINITY) break;
            kept |= 1ull << g;
            if (lane == g) mine = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = 64 * i + lane;
            if (e < a.E && !(kept >> (e / per) & 1)) key[i] = -INFINITY;
        }
    }
    int id = -1;
    double zj = -INFINITY, sj = 0.0;
    for (int j = 0; j < a.top_k; ++j) {
        double best;
        const int e = wave_argmax<V>(key, best);
        if (best == -INFINITY) break;
        const double ze = pick<V>(z, e), se = pick<V>(s, e);
        if (lane == j) {
            id = e;
            zj = ze;
            sj = se;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (64 * i + lane == e) key[i] = -INFINITY;
    }
    const double w = a.renorm ? share_of(zj, a.score == QK_SIGMOID) : sj;
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = id;
        a.weights[t * a.top_k + lane] = (float)(w * (double)a.scale);
    }
}

template <int V>
__global__ __launch_bounds__(kThreads) void moe_route_backward_kernel(MoeRouteBackwardArgs a) {
    __shared__ float dz_lds[kTokens][64 * V];
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / 64;
    if (t >= a.T) return;
    float* dz = dz_lds[threadIdx.x / 64];
    const bool sigmoid = a.score == QK_SIGMOID;
    int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
    if (id >= a.E) id = -1;
    const double z = id >= 0 ? (double)load_logit(a.logits, a.dtype, t * a.E + id) : -INFINITY;
    const double d = id >= 0 ? (double)a.scale * (double)a.dweights[t * a.top_k + lane] : 0.0;
    double all = 0.0, own;                                          // dz = own at the chosen, all * s at every expert
    double s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 0.0;
    if (a.renorm) {
        const double p = share_of(z, sigmoid), mean = wave_sum(d * p);
        // softmax: p (d - mean); sigmoid: (d - mean) / total * s (1 - s) = (d - mean) p (1 - s)
        own = (d - mean) * p * (sigmoid ? 1.0 / (1.0 + exp(z)) : 1.0);
    } else if (sigmoid) {
        own = z == -INFINITY ? 0.0 : d / (1.0 + exp(-z)) / (1.0 + exp(z));
    } else {
        double zz[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = 64 * i + lane;
            zz[i] = e < a.E ? (double)load_logit(a.logits, a.dtype, t * a.E + e) : -INFINITY;
        }
        scores<V>(zz, false, s);
        double se = 0.0;
        for (int j = 0; j < a.top_k; ++j) {
            const int e = __shfl(id, j, 64);
            if (e < 0) continue;
            const double v = pick<V>(s, e);
            if (lane == j) se = v;
        }
        own = d * se;
        all = -wave_sum(own);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) dz[64 * i + lane] = 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (id >= 0 && z != -INFINITY) dz[id] = (float)own;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 64 * i + lane;
        if (e < a.E) store_logit(a.dlogits, a.dtype, t * a.E + e, (float)((double)dz[e] + all * s[i]));
    }
}

// ---------------------------------------------------------------------------
// Plan: workgroup e finds where expert e starts (how many slots go to lower experts) and lists its slots in order;
// workgroup E those without an expert.  Nothing is shared between workgroups, so nothing depends on their order.
// ---------------------------------------------------------------------------
template <int kBlock>
__global__ __launch_bounds__(kBlock) void moe_plan_kernel(const int32_t* __restrict__ ids, int32_t slots, int32_t E,
                                                          int32_t* __restrict__ plan) {
    constexpr int kWaves = kBlock / 64;
    __shared__ int32_t part[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int e = (int)blockIdx.x;
    // expert of a slot, E for none
    auto expert = [&](int i) {
        const int v = ids[i];
        return v < 0 || v >= E ? E : v;
    };
    int less = 0;
    for (int i = tid; i < slots; i += kBlock) less += expert(i) < e;
    less = wave_scan(less);
    if (lane == 63) part[wave] = less;
    __syncthreads();
    int at = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) at += part[w];
    if (tid == 0) plan[e] = at;
    int32_t* list = plan + moe_plan_list(E);
    for (int base = 0; base < slots; base += kBlock) {
        const int i = base + tid;
        const bool mine = i < slots && expert(i) == e;
        const uint64_t b = __ballot(mine);
        __syncthreads();
        if (lane == 0) part[wave] = __builtin_popcountll(b);
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            before += w < wave ? part[w] : 0;
            all += part[w];
        }
        if (mine) list[at + before + __builtin_popcountll(b & ((1ull << lane) - 1))] = i;
        at += all;
    }
}

unsigned token_grid(int64_t T) { return (unsigned)((T + kTokens - 1) / kTokens); }

}  // namespace

hipError_t launch_moe_route(const MoeRouteArgs& a, hipStream_t s) {
    const dim3 grid(token_grid(a.T));
    if (a.E <= 64) moe_route_kernel<1><<<grid, kThreads, 0, s>>>(a);
    else if (a.E <= 128) moe_route_kernel<2><<<grid, kThreads, 0, s>>>(a);
    else if (a.E <= 256) moe_route_kernel<4><<<grid, kThreads, 0, s>>>(a);
    else moe_route_kernel<8><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_route_backward(const MoeRouteBackwardArgs& a, hipStream_t s) {
    const dim3 grid(token_grid(a.T));
    if (a.E <= 64) moe_route_backward_kernel<1><<<grid, kThreads, 0, s>>>(a);
    else if (a.E <= 128) moe_route_backward_kernel<2><<<grid, kThreads, 0, s>>>(a);
    else if (a.E <= 256) moe_route_backward_kernel<4><<<grid, kThreads, 0, s>>>(a);
    else moe_route_backward_kernel<8><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_plan(const int32_t* ids, int64_t slots, int32_t E, int32_t* plan, hipStream_t s) {
    if (slots <= 2048) moe_plan_kernel<256><<<dim3((unsigned)E + 1), 256, 0, s>>>(ids, (int32_t)slots, E, plan);
    else moe_plan_kernel<1024><<<dim3((unsigned)E + 1), 1024, 0, s>>>(ids, (int32_t)slots, E, plan);
    return hipGetLastError();
}

}  // namespace qk
