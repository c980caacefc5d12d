// Router of a mixture-of-experts layer for any number of tokens, its gradient, and the sorting of a routing by expert, for
// gfx950.
//
//   s = softmax(z) or sigmoid(z);  rank = s + bias (z without a bias);  the top_k by rank in the top_groups groups of
//   experts whose two largest s + bias sum highest;  w = scale s, or scale s / (sum of the chosen s)
//
// One wave per token, expert e in lane e % 64.  Which of two ranks is larger is decided in binary64, so that a choice does
// not hang on the rounding of s: the choice is made in 32 bits, and where two ranks or two groups are closer than the error of
// that, made again in 64.  (8192 tokens of 256 experts in 8 groups, top 8: 17.1 us in a captured graph, 18.7 under the
// profiler, instructions, VALU busy 72 %; all in 64 bits 44.)
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
template <int kCtrl, int kRows = 0xF>
__device__ __forceinline__ double dpp_move(double old, double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v), o = __builtin_bit_cast(uint64_t, old);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)o, (int)(uint32_t)u, kCtrl, kRows, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)(o >> 32), (int)(uint32_t)(u >> 32), kCtrl, kRows, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Over the wave, in every lane: inside the rows of 16, then rows 0 and 2 into 1 and 3, then the lower half into the upper.
template <class Op>
__device__ __forceinline__ double wave_reduce(double v, double none, Op&& op) {
    v = op(v, dpp_move<0xB1>(none, v));
    v = op(v, dpp_move<0x4E>(none, v));
    v = op(v, dpp_move<0x141>(none, v));
    v = op(v, dpp_move<0x140>(none, v));
    v = op(v, dpp_move<0x142, 0xA>(none, v));
    v = op(v, dpp_move<0x143, 0xC>(none, v));
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_max(double v) {
    return wave_reduce(v, -INFINITY, [](double a, double b) { return fmax(a, b); });
}
__device__ __forceinline__ double wave_sum(double v) {
    return wave_reduce(v, 0.0, [](double a, double b) { return a + b; });
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

// Whole numbers in the order of the floats (of equal zeros one), 0 below all of them but -NaN.
__device__ __forceinline__ uint32_t order_of(float f) {
    const uint32_t u = as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t k) { return as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kNone = 0x007FFFFFu;                             // order_of(-inf)

// Largest of the wave, as a scalar: inside the rows of 16 lanes, then of the four rows.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = group_max_u32<16>(v);
    const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16));
    const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48));
    return max(a, b);
}
__device__ __forceinline__ float wave_sum(float v) {
    v += as_float(__builtin_amdgcn_mov_dpp(as_uint(v), 0xB1, 0xF, 0xF, false));
    v += as_float(__builtin_amdgcn_mov_dpp(as_uint(v), 0x4E, 0xF, 0xF, false));
    v += as_float(__builtin_amdgcn_mov_dpp(as_uint(v), 0x141, 0xF, 0xF, false));
    v += as_float(__builtin_amdgcn_mov_dpp(as_uint(v), 0x140, 0xF, 0xF, false));
    auto row = [&](int l) { return as_float((uint32_t)__builtin_amdgcn_readlane((int)as_uint(v), l)); };
    return (row(0) + row(16)) + (row(32) + row(48));
}

__device__ __forceinline__ float sigmoid_of(float z) { return z >= 0.0f ? 1.0f / (1.0f + expf(-z)) : expf(z) / (1.0f + expf(z)); }

// Shares of the chosen experts (one a lane; z = -inf: none): s_j / sum of s.  Relative to the largest, so that scores too
// small for a number still have a ratio.
__device__ __forceinline__ float share_of(float z, bool sigmoid) {
    const float most = float_of(wave_max(order_of(z))), top = sigmoid ? fminf(most, 0.0f) : most;
    float r = 0.0f;
    if (z != -INFINITY) r = sigmoid && z >= 0.0f ? 1.0f / (1.0f + expf(-z)) : expf(z - top) / (sigmoid ? 1.0f + expf(z) : 1.0f);
    const float total = wave_sum(r);
    return total > 0.0f ? r / total : 0.0f;
}

// The two largest of groups of 2^n experts, in every lane and register of the group: joined across the lanes that a DPP
// pattern pairs, then across registers.
template <class K>
__device__ __forceinline__ void join(K& a1, K& a2, K b1, K b2) {
    const K low = a1 < b1 ? a1 : b1, second = a2 < b2 ? b2 : a2;
    a2 = low < second ? second : low;
    a1 = a1 < b1 ? b1 : a1;
}
template <int kCtrl>
__device__ __forceinline__ double dpp_pair(double v) {
    return dpp_move<kCtrl>(v, v);
}
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_pair(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}
template <int V, class K>
__device__ __forceinline__ void join_groups(K (&m1)[V], K (&m2)[V], int per) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (per > 1) join(m1[i], m2[i], dpp_pair<0xB1>(m1[i]), dpp_pair<0xB1>(m2[i]));       // lane ^ 1
        if (per > 2) join(m1[i], m2[i], dpp_pair<0x4E>(m1[i]), dpp_pair<0x4E>(m2[i]));       // lane ^ 2
        if (per > 4) join(m1[i], m2[i], dpp_pair<0x141>(m1[i]), dpp_pair<0x141>(m2[i]));     // 7 - lane of 8
        if (per > 8) join(m1[i], m2[i], dpp_pair<0x140>(m1[i]), dpp_pair<0x140>(m2[i]));     // 15 - lane of 16
        if (per > 16) join(m1[i], m2[i], wave_xor(m1[i], 16), wave_xor(m2[i], 16));
        if (per > 32) join(m1[i], m2[i], wave_xor(m1[i], 32), wave_xor(m2[i], 32));
    }
#pragma unroll
    for (int d = 1; d < V; d <<= 1) {
        if (64 * d >= per) break;
        K b1[V], b2[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            b1[i] = m1[i ^ d];
            b2[i] = m2[i ^ d];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) join(m1[i], m2[i], b1[i], b2[i]);
    }
}

// v[e / 64] of lane e % 64, e a lane's own.
template <int V, class K>
__device__ __forceinline__ K gather(const K (&v)[V], int e) {
    K r = v[0];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const K x = __shfl(v[i], e & 63, 64);
        r = e >> 6 == i ? x : r;
    }
    return r;
}

// What a token's choice leaves in lane j: its expert j, that one's logit and, where weights are not renormalized, its score.
struct Choice {
    int id;
    float z;
    float s;
};

__device__ __forceinline__ float load_bias(const float* bias, int e, int E) {
    const float b = bias && e < E ? bias[e] : 0.0f;
    return b == b ? fminf(b, 3.402823466e38f) : -INFINITY;
}

// The choice in binary64 throughout.
template <int V>
__device__ __forceinline__ Choice choose_exactly(const MoeRouteArgs& a, int64_t t, int group_shift) {
    const int lane = threadIdx.x & 63;
    double z[V], s[V], key[V], ranked[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 64 * i + lane;
        z[i] = e < a.E ? (double)load_logit(a.logits, a.dtype, t * a.E + e) : -INFINITY;
    }
    scores<V>(z, a.score == QK_SIGMOID, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        ranked[i] = z[i] == -INFINITY ? -INFINITY : s[i] + (double)load_bias(a.bias, 64 * i + lane, a.E);
        key[i] = a.bias ? ranked[i] : z[i];
    }
    if (a.groups > 1) {
        const int per = a.E / a.groups;
        double sum = -INFINITY;                                     // lane g: of group g's two largest
        if (group_shift >= 0) {
            double m1[V], m2[V], both[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                m1[i] = ranked[i];
                m2[i] = -INFINITY;
            }
            join_groups<V>(m1, m2, per);
#pragma unroll
            for (int i = 0; i < V; ++i) both[i] = m2[i] == -INFINITY ? m1[i] : m1[i] + m2[i];
            const double v = gather<V>(both, lane << group_shift);
            if (lane < a.groups) sum = v;
        } else {
            for (int g = 0; g < a.groups; ++g) {
                double v[V], best, second;
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = (64 * i + lane) / per == g ? ranked[i] : -INFINITY;
                const int at = wave_argmax<V>(v, best);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (64 * i + lane == at) v[i] = -INFINITY;
                wave_argmax<V>(v, second);
                if (lane == g) sum = second == -INFINITY ? best : best + second;
            }
        }
        uint64_t kept = 0;
        for (int j = 0; j < a.top_groups; ++j) {
            const double m[1] = {sum};
            double best;
            const int g = wave_argmax<1>(m, best);
            if (best == -INFINITY) break;
            kept |= 1ull << g;
            if (lane == g) sum = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = 64 * i + lane;
            if (e < a.E && !(kept >> (e / per) & 1)) key[i] = -INFINITY;
        }
    }
    Choice c{-1, -INFINITY, 0.0f};
    for (int j = 0; j < a.top_k; ++j) {
        double best;
        const int e = wave_argmax<V>(key, best);
        if (best == -INFINITY) break;
        const double ze = pick<V>(z, e), se = pick<V>(s, e);
        if (lane == j) c = Choice{e, (float)ze, (float)se};
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (64 * i + lane == e) key[i] = -INFINITY;
    }
    return c;
}

// The largest key and the lowest place that has it (64 i + lane), which is taken out.
template <int V>
__device__ __forceinline__ int take_best(uint32_t (&key)[V], uint32_t& best) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, key[i]);
    best = wave_max(m);
    int at = 0;
    uint64_t who = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) {
        const uint64_t b = __ballot(key[i] == best);
        if (b) {
            at = i;
            who = b;
        }
    }
    who &= -who;
    const bool mine = (threadIdx.x & 63) == (uint32_t)__builtin_ctzll(who);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = at == i && mine ? kNone : key[i];
    return 64 * at + (int)__builtin_ctzll(who);
}

// The choice with ranks in 32 bits, for groups of 2^n experts.  Where ranks in it are too close for that, the best ones up to
// a clear gap behind the last one wanted are put in order by their ranks in 64 bits, one in each lane; false where that does
// not do: a group too close to another, or more than 64 such ranks.
//   A score in 32 bits is off by less than 2^-21 (sigmoid: its exponential by the rounding of the argument, 2^-24 |z| of itself,
// of which x exp(-x) < 0.4 is left, and two steps, the reciprocal by one) or 2^-20 (softmax: the sum of 512, made in a tree, by
// 2^-21 of itself more).  Added to a bias it is rounded to 2^-24 of itself.
__device__ __forceinline__ float slack(float rank, bool sigmoid) {
    return (sigmoid ? 4.76837158e-7f : 9.53674316e-7f) + 1.1920929e-7f * fabsf(rank);
}

template <int V>
__device__ __forceinline__ bool choose_fast(const MoeRouteArgs& a, int64_t t, int group_shift, Choice& c) {
    const int lane = threadIdx.x & 63;
    const bool sigmoid = a.score == QK_SIGMOID;
    float z[V];
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 64 * i + lane;
        z[i] = e < a.E ? load_logit(a.logits, a.dtype, t * a.E + e) : -INFINITY;
        key[i] = order_of(z[i]);
    }
    float top = 0.0f, inv = 0.0f;                                   // of the softmax
    if (a.bias || a.groups > 1 || !(a.renorm || sigmoid)) {
        float s[V];
        if (sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float e = __expf(-fabsf(z[i])), r = __builtin_amdgcn_rcpf(1.0f + e);
                s[i] = z[i] >= 0.0f ? r : e * r;
            }
        } else {
            uint32_t m = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) m = max(m, key[i]);
            top = float_of(wave_max(m));
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[i] = z[i] == -INFINITY ? 0.0f : __expf(z[i] - top);
                sum += s[i];
            }
            inv = 1.0f / wave_sum(sum);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = s[i] > 0.0f ? s[i] * inv : 0.0f;
        }
        uint32_t ranked[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            ranked[i] = z[i] == -INFINITY ? kNone : order_of(a.bias ? s[i] + load_bias(a.bias, 64 * i + lane, a.E) : s[i]);
            if (a.bias) key[i] = ranked[i];
        }
        if (a.groups > 1) {
            uint32_t m1[V], m2[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                m1[i] = ranked[i];
                m2[i] = kNone;
            }
            join_groups<V>(m1, m2, 1 << group_shift);
            // Group g in lane g: its sum, and what 32 bits may have that off by.  The two ranks may cancel, their errors do not.
            // A sum past the largest numbers counts as one of them, from which its error reaches to an infinity: two such are
            // never clear of each other.
            const uint32_t k1 = gather<V>(m1, lane << group_shift), k2 = gather<V>(m2, lane << group_shift);
            const bool one = k2 <= kNone;
            const float v1 = float_of(k1), v2 = one ? 0.0f : float_of(k2);
            const float sum = fminf(fmaxf(v1 + v2, -3.402823466e38f), 3.402823466e38f);
            const float off = slack(v1, sigmoid) + (one ? 0.0f : slack(v2, sigmoid)) + 1.1920929e-7f * fabsf(sum);
            uint32_t g = lane < a.groups && k1 > kNone ? order_of(sum) : 0u;
            uint64_t kept = 0;                                      // the best top_groups
            for (int j = 0; j < a.top_groups; ++j) {
                const uint32_t best = wave_max(g);
                if (best == 0) break;
                const int at = (int)__builtin_ctzll(__ballot(g == best));
                kept |= 1ull << at;
                g = lane == at ? 0u : g;
            }
            // a clear gap between the least that one of them may be and the most that one of the others may be
            const uint32_t most = wave_max(g ? order_of(sum + off) : 0u);
            if (most) {
                if (~wave_max(kept >> lane & 1 ? ~order_of(sum - off) : 0u) <= most) return false;
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (!(kept >> ((64 * i + lane) >> group_shift) & 1)) key[i] = kNone;
        }
    }
    int id = -1, n = 0;                                             // candidate j in lane j
    uint32_t mine = 0;
    float wanted = 0.0f;                                            // rank of the last one wanted
    while (true) {
        uint32_t best;
        const int e = take_best<V>(key, best);
        if (best <= kNone) break;
        if (a.bias) {
            const float v = float_of(best);
            if (n >= a.top_k && wanted - v > slack(wanted, sigmoid) + slack(v, sigmoid)) break;
            if (n == 64) return false;
            wanted = n == a.top_k - 1 ? v : wanted;
        }
        if (lane == n) {
            id = e;
            mine = best;
        }
        if (++n == a.top_k && !a.bias) break;
    }
    if (a.bias) {
        const float v = float_of(mine), next = __shfl_down(v, 1, 64);
        const bool close = lane + 1 < n && !(v - next > slack(v, sigmoid) + slack(next, sigmoid));
        if (__ballot(close)) {
            const int e = id < 0 ? 0 : id;
            const double ze = (double)gather<V>(z, e);
            double s;
            if (sigmoid) {
                s = 1.0 / (1.0 + exp(-ze));
            } else {
                double sum = 0.0;
#pragma unroll
                for (int i = 0; i < V; ++i) sum += z[i] == -INFINITY ? 0.0 : exp((double)z[i] - (double)top);
                s = exp(ze - (double)top) / wave_sum(sum);
            }
            const double r = s + (double)load_bias(a.bias, e, a.E);
            int place = 0;
            for (int i = 0; i < n; ++i) {
                const double ri = __shfl(r, i, 64);
                const int ei = __shfl(id, i, 64);
                place += ri > r || (ri == r && ei < id);
            }
            id = __builtin_amdgcn_ds_permute(4 * (lane < n ? place : lane), id);
        }
        if (lane >= a.top_k) id = -1;
    }
    c.id = id;
    c.z = gather<V>(z, id < 0 ? 0 : id);
    if (id < 0) c.z = -INFINITY;
    c.s = a.renorm || sigmoid || id < 0 ? 0.0f : expf(c.z - top) * inv;
    return true;
}

// (Sixteen waves a SIMD would need 32 registers; what the choice in 64 bits has beyond 64 goes to memory.)
template <int V>
__global__ __launch_bounds__(kThreads, V <= 4 ? 8 : 4) void moe_route_kernel(MoeRouteArgs a, int group_shift) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kTokens + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (t >= a.T) return;
    Choice c;
    if (group_shift < 0 || !choose_fast<V>(a, t, group_shift, c)) c = choose_exactly<V>(a, t, group_shift);
    const bool sigmoid = a.score == QK_SIGMOID;
    const float w = a.renorm ? share_of(c.z, sigmoid) : sigmoid ? sigmoid_of(c.z) : c.s;
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = c.id;
        a.weights[t * a.top_k + lane] = w * a.scale;
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
    const float z = id >= 0 ? load_logit(a.logits, a.dtype, t * a.E + id) : -INFINITY;
    const float d = id >= 0 ? a.scale * a.dweights[t * a.top_k + lane] : 0.0f;
    float all = 0.0f, own;                                          // dz = own at the chosen, all * s at every expert
    float s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 0.0f;
    if (a.renorm) {
        // softmax: p (d - mean); sigmoid: (d - mean) / total * s (1 - s) = (d - mean) p (1 - s).  Both relative to the d of the
        // largest p: of one near 1 only what the others have is left, and d - mean would be the rounding of d.
        const float p = share_of(z, sigmoid);
        const int most = (int)__builtin_ctzll(__ballot(order_of(z) == wave_max(order_of(z))));
        const float rel = d - as_float((uint32_t)__builtin_amdgcn_readlane((int)as_uint(d), most));
        own = (rel - wave_sum(rel * p)) * p * (sigmoid ? sigmoid_of(-z) : 1.0f);
    } else if (sigmoid) {
        own = z == -INFINITY ? 0.0f : d * sigmoid_of(z) * sigmoid_of(-z);
    } else {
        float zz[V];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = 64 * i + lane;
            zz[i] = e < a.E ? load_logit(a.logits, a.dtype, t * a.E + e) : -INFINITY;
            m = max(m, order_of(zz[i]));
        }
        const float top = float_of(wave_max(m));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = zz[i] == -INFINITY ? 0.0f : expf(zz[i] - top);
            sum += s[i];
        }
        sum = wave_sum(sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] *= inv;
        const float p = z == -INFINITY ? 0.0f : expf(z - top) * inv;
        own = d * p;
        all = -wave_sum(own);
        // p (d - sum d p) of one near 1 would be the rounding of d, too: p (d (1 - p) - the others' sum), 1 - p from their s
        const uint64_t near_one = __ballot(p > 0.5f);
        if (near_one) {
            const int at = (int)__builtin_ctzll(near_one), e = __builtin_amdgcn_readlane(id, at);
            float rest = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[i] = 64 * i + lane == e ? 0.0f : s[i];
                rest += s[i];
            }
            rest = wave_sum(rest);
            const float others = wave_sum(lane == at ? 0.0f : own);
            own = lane == at ? p * (d * rest - others) : own;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) dz[64 * i + lane] = 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (id >= 0 && z != -INFINITY) dz[id] = own;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 64 * i + lane;
        if (e < a.E) store_logit(a.dlogits, a.dtype, t * a.E + e, fmaf(all, s[i], dz[e]));
    }
}

// ---------------------------------------------------------------------------
// Plan: every workgroup counts the slots of all experts (whole numbers in LDS: their order does not matter) and finds from
// the sums where each expert starts; workgroup e lists the slots of expert e in order and cuts them into tiles, workgroup E
// those without an expert.  Nothing is shared between workgroups.  A thread takes kPer consecutive slots at a time.
// Bound by latency (4096 tokens, top 8 of 64, 9.7 us): the first two runs of slots are loaded at once and kept for the list, 12.5 where
// each is loaded twice; 512 tokens, top 2 of 8, 4.2 us with 4 slots a thread, 6.7 with 16.
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
    auto count_in = [&](const int (&v)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (v[i] >= 0) atomicAdd(&bins[v[i]], 1);
    };
    // the first kKept runs are loaded together and stay in registers
    constexpr int kRun = kBlock * kPer, kKept = 2;
    int kept[kKept][kPer];
#pragma unroll
    for (int c = 0; c < kKept; ++c) load((int64_t)c * kRun + tid * kPer, kept[c]);
#pragma unroll
    for (int c = 0; c < kKept; ++c) count_in(kept[c]);
    for (int64_t first = kKept * kRun; first < slots; first += kRun) {
        int v[kPer];
        load(first + tid * kPer, v);
        count_in(v);
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
    auto list_run = [&](int64_t first, const int (&v)[kPer]) {
        const int64_t base = first + (int64_t)tid * kPer;
        int count = 0;
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
    };
#pragma unroll
    for (int c = 0; c < kKept; ++c)
        if (c * kRun < slots) list_run((int64_t)c * kRun, kept[c]);
    for (int64_t first = kKept * kRun; first < slots; first += kRun) {
        int v[kPer];
        load(first + tid * kPer, v);
        list_run(first, v);
    }
}

unsigned token_grid(int64_t T) { return (unsigned)((T + kTokens - 1) / kTokens); }

// Launches over tokens in pieces (a launch has fewer than 2^32 threads): launch(arguments of the piece).
template <class Args, class Launch>
hipError_t by_tokens(const Args& a, Launch&& launch) {
    constexpr int64_t kMost = (int64_t)1 << 24;
    for (int64_t t = 0; t < a.T; t += kMost) {
        Args p = a;
        p.T = a.T - t < kMost ? a.T - t : kMost;
        p.move(t);
        launch(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_moe_route(const MoeRouteArgs& all, hipStream_t s) {
    // log2 of the experts of a group; groups of other sizes are chosen in 64 bits
    const int per = all.E / all.groups;
    const int shift = all.groups == 1 ? 0 : (per & (per - 1)) == 0 ? __builtin_ctz((unsigned)per) : -1;
    return by_tokens(all, [&](const MoeRouteArgs& a) {
        const dim3 grid(token_grid(a.T));
        if (a.E <= 64) moe_route_kernel<1><<<grid, kThreads, 0, s>>>(a, shift);
        else if (a.E <= 128) moe_route_kernel<2><<<grid, kThreads, 0, s>>>(a, shift);
        else if (a.E <= 256) moe_route_kernel<4><<<grid, kThreads, 0, s>>>(a, shift);
        else moe_route_kernel<8><<<grid, kThreads, 0, s>>>(a, shift);
    });
}

hipError_t launch_moe_route_backward(const MoeRouteBackwardArgs& all, hipStream_t s) {
    return by_tokens(all, [&](const MoeRouteBackwardArgs& a) {
        const dim3 grid(token_grid(a.T));
        if (a.E <= 64) moe_route_backward_kernel<1><<<grid, kThreads, 0, s>>>(a);
        else if (a.E <= 128) moe_route_backward_kernel<2><<<grid, kThreads, 0, s>>>(a);
        else if (a.E <= 256) moe_route_backward_kernel<4><<<grid, kThreads, 0, s>>>(a);
        else moe_route_backward_kernel<8><<<grid, kThreads, 0, s>>>(a);
    });
}

hipError_t launch_moe_plan(const int32_t* ids, int64_t slots, int32_t E, int32_t* plan, hipStream_t s) {
    const int32_t rows = (int32_t)moe_tile_rows(slots, E);
    const dim3 grid((unsigned)E + 1);
    if (slots <= 512) moe_plan_kernel<256, 2><<<grid, 256, 0, s>>>(ids, (int32_t)slots, E, rows, plan);
    else if (slots <= 8192) moe_plan_kernel<1024, 4><<<grid, 1024, 0, s>>>(ids, (int32_t)slots, E, rows, plan);
    else moe_plan_kernel<1024, 16><<<grid, 1024, 0, s>>>(ids, (int32_t)slots, E, rows, plan);
    return hipGetLastError();
}

}  // namespace qk
