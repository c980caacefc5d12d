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
// Plan: every workgroup counts the slots of all experts (whole numbers in LDS: their order does not matter) and finds from
// the sums where each expert starts; workgroup e lists the slots of expert e in order and cuts them into tiles, workgroup E
// those without an expert.  Nothing is shared between workgroups.  A thread takes kPer consecutive slots at a time.
// ---------------------------------------------------------------------------
template <int kBlock, int kPer>
__global__ __launch_bounds__(kBlock) void moe_plan_kernel(const int32_t* __restrict__ ids, int32_t slots, int32_t E, int32_t rows,
                                                          int32_t* __restrict__ plan) {
    constexpr int kWaves = kBlock / 64, kBins = 576;               // of E + 1 <= 513, in whole waves
    __shared__ int32_t bins[kBins];
    __shared__ int32_t part[2][kBins / 64], part2[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int e = (int)blockIdx.x;
    for (int i = tid; i < kBins; i += kBlock) bins[i] = 0;
    __syncthreads();
    // the experts (E: none) of slots base .. base + kPer - 1; -1 past the end
    auto load = [&](int64_t base, int (&v)[kPer]) {
        if (base + kPer <= slots) {
            __builtin_memcpy(v, ids + base, 4 * kPer);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = base + i < slots ? ids[base + i] : 0;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = base + i >= slots ? -1 : v[i] < 0 || v[i] >= E ? E : v[i];
    };
    for (int64_t base = (int64_t)tid * kPer; base < slots; base += kBlock * kPer) {
        int v[kPer];
        load(base, v);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (v[i] >= 0) atomicAdd(&bins[v[i]], 1);
    }
    __syncthreads();
    // sums of the slots and the tiles of the bins below one's own, 64 bins a wave
    constexpr int kTurns = (kBins / 64 + kWaves - 1) / kWaves;
    int n[kTurns], before[kTurns], tiles[kTurns];
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        const int g = wave + kWaves * u;
        n[u] = before[u] = tiles[u] = 0;
        if (g >= kBins / 64) continue;
        n[u] = bins[64 * g + lane];
        before[u] = wave_scan(n[u]);
        tiles[u] = wave_scan((n[u] + rows - 1) / rows);
        if (lane == 63) {
            part[0][g] = before[u];
            part[1][g] = tiles[u];
        }
    }
    __syncthreads();
    int at = 0, tile0 = 0, mine = 0;
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        const int g = wave + kWaves * u;
        if (g >= kBins / 64) continue;
        for (int w = 0; w < g; ++w) {
            before[u] += part[0][w];
            tiles[u] += part[1][w];
        }
        if (64 * g + lane == e) {                                   // hands its numbers to the workgroup
            bins[0] = before[u] - n[u];
            bins[1] = tiles[u] - (n[u] + rows - 1) / rows;
            bins[2] = n[u];
        }
    }
    __syncthreads();
    at = bins[0];
    tile0 = bins[1];
    mine = bins[2];
    int32_t* const tiles_at = plan + moe_plan_tiles(E, slots);
    const int own_tiles = (mine + rows - 1) / rows;
    if (tid == 0) {
        plan[e] = at;
        if (e == E) tiles_at[0] = tile0 + own_tiles;
    }
    MoeTile* const table = reinterpret_cast<MoeTile*>(tiles_at + 4);
    for (int i = tid; i < own_tiles; i += kBlock)
        table[tile0 + i] = MoeTile{at + i * rows, e | (mine - i * rows < rows ? mine - i * rows : rows) << 16};
    int32_t* list = plan + moe_plan_list(E);
    for (int64_t first = 0; first < slots; first += kBlock * kPer) {
        const int64_t base = first + (int64_t)tid * kPer;
        int v[kPer], count = 0;
        load(base, v);
#pragma unroll
        for (int i = 0; i < kPer; ++i) count += v[i] == e;
        const int incl = wave_scan(count);
        __syncthreads();
        if (lane == 63) part2[wave] = incl;
        __syncthreads();
        int place = at + incl - count;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            place += w < wave ? part2[w] : 0;
            at += part2[w];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (v[i] == e) list[place++] = (int32_t)(base + i);
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
    const int32_t rows = (int32_t)moe_tile_rows(slots, E);
    const dim3 grid((unsigned)E + 1);
    if (slots <= 512) moe_plan_kernel<256, 2><<<grid, 256, 0, s>>>(ids, (int32_t)slots, E, rows, plan);
    else moe_plan_kernel<1024, 16><<<grid, 1024, 0, s>>>(ids, (int32_t)slots, E, rows, plan);
    return hipGetLastError();
}

}  // namespace qk
