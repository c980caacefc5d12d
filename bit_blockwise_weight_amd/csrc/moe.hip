// A mixture-of-experts layer for a few tokens over 4-bit experts, for gfx950:
//     S_t     = the top_k largest of logits[t, :], ties to the lower index
//     w[t, e] = exp(L[t, e] - max) / sum (over S_t, or over every expert)
//     h[t, e] = silu(x_t Wg_e^T) * (x_t Wu_e^T)
//     y_t     = sum over e in S_t of w[t, e] h[t, e] Wd_e^T
// with the weights of all experts stacked in two quantized tensors, gate and up rows of an
// expert one after the other in the first.
//
//   moe_route_kernel  one workgroup: each wave selects one token's experts, then the
//                     experts with a token are listed in increasing order, each with its
//                     tokens (for the up kernel) and with a weight and a row of h per
//                     token (for the down kernel).
//   moe_up_kernel     a workgroup per (listed expert, 16 rows of gate and the 16 of up):
//                     only the expert's own tokens are staged in LDS; each wave takes
//                     128-k chunks of the rows, the partial sums are added in wave order.
//                     h is kept as two bf16 values (hi + lo, 16 bits of mantissa): the
//                     down product then loses nothing against the bf16 or fp16 output.
//   moe_down_kernel   a workgroup per 16 outputs; its waves take the (expert, chunk) steps in
//                     turn and keep one accumulator per token, the token's weight being
//                     applied with the row scale: no partial sums in memory, no atomics.
// Every weight of a listed expert is read once per layer; that is the bound.
#include <algorithm>

#include "qk_device.h"
#include "qk_internal.h"
#include "w4_tile.h"

namespace qk {
namespace {

using namespace w4;

constexpr int kMaxT = 16;
constexpr int kMaxE = 256;
constexpr int kMaxK = 16;

// Routing result, in the workspace.
struct Routes {
    int32_t nactive;
    int32_t pad[3];
    int32_t expert[kMaxE];            // listed experts, increasing
    int32_t count[kMaxE];             // tokens of each
    uint8_t tok[kMaxE][kMaxT];        // those tokens, increasing
    int16_t row[kMaxE][kMaxT];        // row of h of each: t * top_k + position
    float w[kMaxE][kMaxT];            // weight per token, 0 for the others
    int16_t hrow[kMaxE][kMaxT];       // row of h per token, -1 for the others
};

struct RouteArgs {
    const void* logits;
    int32_t dtype;
    int32_t T, E, top_k, renorm;
};

__device__ __forceinline__ float load_logit(const void* p, int32_t dtype, int64_t i) {
    float v;
    if (dtype == QK_F32) v = static_cast<const float*>(p)[i];
    else if (dtype == QK_F16) v = f16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
    else v = bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
    return v == v ? v : -INFINITY;                       // a NaN logit is never chosen
}

__global__ __launch_bounds__(kMaxT * 64) void moe_route_kernel(RouteArgs a, Routes* out) {
    __shared__ int ids[kMaxT][kMaxK];
    __shared__ float wt[kMaxT][kMaxK];
    __shared__ uint32_t mask[kMaxE];
    __shared__ int wcount[4];
    const int tid = threadIdx.x, lane = tid & 63, t = tid >> 6;
    if (tid < kMaxE) mask[tid] = 0;
    __syncthreads();
    if (t < a.T) {
        float v[4];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = lane + 64 * i;
            v[i] = e < a.E ? load_logit(a.logits, a.dtype, (int64_t)t * a.E + e) : -INFINITY;
            top = fmaxf(top, v[i]);
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
        float den = 0.0f;
        if (!a.renorm) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v[i] != -INFINITY) den += expf(v[i] - top);
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) den += __shfl_xor(den, d);
        }
        float mine = 0.0f;                               // lane k: weight of the k-th choice
        int id = -1;
        for (int k = 0; k < a.top_k; ++k) {
            float best = v[0];
            int e = lane;
#pragma unroll
            for (int i = 1; i < 4; ++i)
                if (v[i] > best) {
                    best = v[i];
                    e = lane + 64 * i;
                }
            float m = best;
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
            if (m == -INFINITY) break;                   // nothing left that may be chosen
            int c = best == m ? e : kMaxE;
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) c = min(c, __shfl_xor(c, d));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c == lane + 64 * i) v[i] = -INFINITY;
            const float p = expf(m - top);
            if (a.renorm) den += p;
            if (lane == k) {
                mine = p;
                id = c;
            }
        }
        if (lane < a.top_k) {
            ids[t][lane] = id;
            wt[t][lane] = id >= 0 ? mine / den : 0.0f;
            if (id >= 0) atomicOr(&mask[id], 1u << t);
        }
    }
    __syncthreads();
    const uint32_t mk = tid < kMaxE ? mask[tid] : 0u;
    const unsigned long long bal = __ballot(mk != 0);
    if (tid < kMaxE && lane == 0) wcount[t] = __popcll(bal);
    __syncthreads();
    if (tid >= kMaxE) return;
    int rank = __popcll(bal & ((1ull << lane) - 1));
    int total = 0;
    for (int w = 0; w < 4; ++w) {
        if (w < t) rank += wcount[w];
        total += wcount[w];
    }
    if (tid == 0) out->nactive = total;
    if (!mk) return;
    out->expert[rank] = tid;
    out->count[rank] = __popc(mk);
    int pos = 0;
    for (int tt = 0; tt < kMaxT; ++tt) {
        float w = 0.0f;
        int r = -1;
        if ((mk >> tt) & 1u) {
            for (int k = 0; k < a.top_k; ++k)
                if (ids[tt][k] == tid) {
                    w = wt[tt][k];
                    r = tt * a.top_k + k;
                }
            out->tok[rank][pos] = (uint8_t)tt;
            out->row[rank][pos] = (int16_t)r;
            ++pos;
        }
        out->w[rank][tt] = w;
        out->hrow[rank][tt] = (int16_t)r;
    }
}

// A weight view of either form, with the calls the kernels make of it.
template <int F>
struct View {
    typedef Int4View type;
};
template <>
struct View<kLevels> {
    typedef LevelsView type;
};

template <int F, int NG>
struct Scales {
    typedef GroupScales<NG> type;
};
template <int NG>
struct Scales<kLevels, NG> {
    typedef LevelScales type;
};

template <int F>
struct UpArgs {
    const uint16_t* x;       // [T, H]
    typename View<F>::type w;
    const Routes* routes;
    uint16_t* h;             // [T * top_k, 2 * Ipad]: per 8 values, 8 hi then 8 lo
    int64_t H;
    int64_t I;
    int64_t Ipad;            // I rounded up to a chunk
    int32_t T;
    int32_t x_aligned;
};

template <int F>
constexpr int kUpWaves = F == kLevels ? 16 : 8;
template <int F>
constexpr int kUpPitch = kUpWaves<F> * kChunk * 2 + 16;

template <int F, int NG>
__global__ __launch_bounds__(kUpWaves<F> * 64) void moe_up_kernel(UpArgs<F> p) {
    extern __shared__ __align__(16) uint8_t lds[];
    constexpr int W = kUpWaves<F>, kThreads = W * 64;
    constexpr int kWinUnits = W * kChunk / 8;
    constexpr int kPitch = kUpPitch<F>;
    constexpr int kGroupMfmas = 4 / NG;
    const int a = blockIdx.y;
    if (a >= p.routes->nactive) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, hq = lane >> 4;
    const int M = p.routes->count[a];
    const int64_t e = p.routes->expert[a];
    const int64_t i0 = (int64_t)blockIdx.x * 16;
    uint8_t* xlds = lds + (F == kLevels ? kTabBytes : 0);
    // rows of gate and of up (past the last one of the expert: its last row, never stored)
    const int64_t in = i0 + n < p.I ? i0 + n : p.I - 1;
    const int64_t row[2] = {e * 2 * p.I + in, e * 2 * p.I + p.I + in};
    const uint8_t* codes[2] = {p.w.codes + row[0] * p.w.stride, p.w.codes + row[1] * p.w.stride};
    const int nchunk = (int)((p.H + kChunk - 1) / kChunk);
    const int nwin = (nchunk + W - 1) / W;
    float mean = 0.0f;
    if constexpr (F == kLevels) {
        build_table(lds, p.w.levels, tid, kThreads);
        if (p.w.nested) mean = *p.w.dq_mean;
    }

    floatx4_t y[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    u32x4_t cw[2][2];
    typename Scales<F, NG>::type sc[2][2];
    auto fetch = [&](int buf, int win) {
        int c = win * W + wave;
        c = c < nchunk ? c : nchunk - 1;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            cw[buf][r] = load_codes(codes[r], p.w.stride, c, hq);
            sc[buf][r].load(p.w, row[r], c);
        }
    };
    auto stage = [&](int win) {
        for (int i = tid; i < M * kWinUnits; i += kThreads) {
            const int m = i / kWinUnits, u = i % kWinUnits;
            u32x4_t v = load_x8(p.x + (int64_t)p.routes->tok[a][m] * p.H, (int64_t)win * (W * kChunk) + 8 * u, p.H,
                                p.x_aligned);
            if constexpr (F != kLevels) v = int4_order(v);
            *reinterpret_cast<u32x4_t*>(xlds + m * kPitch + 16 * u) = v;
        }
    };
    const uint8_t* arow = xlds + (n < M ? n : M - 1) * kPitch + wave * (kChunk * 2) + 16 * hq;
    auto compute = [&](int buf, int win) {
        if (win * W + wave >= nchunk) return;
        u32x4_t w[2] = {cw[buf][0], cw[buf][1]};
        transpose_groups(w[0]);
        transpose_groups(w[1]);
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            floatx4_t acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}}, xs = {0, 0, 0, 0};
#pragma unroll
            for (int j = q * kGroupMfmas; j < (q + 1) * kGroupMfmas; ++j) {
                const u32x4_t av = *reinterpret_cast<const u32x4_t*>(arow + 64 * j);
                if constexpr (F == kLevels) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) acc[r] = mfma<F>(av, decode8_table(lds, w[r][j], 4 * lane), acc[r]);
                } else {
                    xs = mfma<F>(av, ones<F>(), xs);
#pragma unroll
                    for (int r = 0; r < 2; ++r) acc[r] = mfma<F>(av, decode8<F>(w[r][j]), acc[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if constexpr (F == kLevels) {
                    const float s = sc[buf][r].scale(p.w, mean, q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[r][i] = fmaf(s, acc[r][i], y[r][i]);
                } else {
                    const float s = sc[buf][r].scale(p.w, q);
                    const float zb = (float)sc[buf][r].z[q] + kCodeBias<F>;
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[r][i] = fmaf(s, fmaf(-zb, xs[i], acc[r][i]), y[r][i]);
                }
            }
        }
    };

    fetch(0, 0);
    for (int win = 0; win < nwin; win += 2) {
        stage(win);
        if (win + 1 < nwin) fetch(1, win + 1);
        __syncthreads();
        compute(0, win);
        __syncthreads();
        if (win + 1 < nwin) {
            stage(win + 1);
            if (win + 2 < nwin) fetch(0, win + 2);
            __syncthreads();
            compute(1, win + 1);
            __syncthreads();
        }
    }

    floatx4_t* red = reinterpret_cast<floatx4_t*>(lds);
#pragma unroll
    for (int r = 0; r < 2; ++r) red[(wave * 2 + r) * 64 + lane] = y[r];
    __syncthreads();
    const float* redf = reinterpret_cast<const float*>(lds);
    if (tid < 256) {
        float gate = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            gate += redf[w * 512 + tid];
            up += redf[w * 512 + 256 + tid];
        }
        const int l = tid >> 2, m = 4 * (l >> 4) + (tid & 3), i = (int)i0 + (l & 15);
        if (m < M) {
            float v = gate / (1.0f + expf(-gate)) * up;
            if (i >= p.I) v = 0.0f;                      // the padding of h takes part in the down product
            const uint16_t hi = float_to_bits16(v, false);
            const uint16_t lo = float_to_bits16(v - bf16_bits_to_float(hi), false);
            uint16_t* dst = p.h + (int64_t)p.routes->row[a][m] * (2 * p.Ipad) + (i >> 3) * 16 +
                            (F == kLevels ? (i & 7) : int4_slot(i));
            dst[0] = hi;
            dst[8] = lo;
        }
    }
}

template <int F>
struct DownArgs {
    const uint16_t* h;
    typename View<F>::type w;
    const Routes* routes;
    uint16_t* y;             // [T, H]
    int64_t H;
    int64_t Ipad;
    int32_t nchunk;
    int32_t T;
    int32_t y_f16;
    int32_t pad;
};

constexpr int kDownWaves = 16;

// Two: more than 8 tokens, hi and lo of h in products of their own; otherwise rows 0..7 of the
// activation operand are the tokens' hi parts and rows 8..15 their lo parts.
template <int F, int NG, bool Two>
__global__ __launch_bounds__(kDownWaves * 64) void moe_down_kernel(DownArgs<F> p) {
    extern __shared__ __align__(16) uint8_t lds[];
    constexpr int W = kDownWaves, kThreads = W * 64;
    constexpr int kGroupMfmas = 4 / NG;
    constexpr int kParts = Two ? 2 : 1;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, hq = lane >> 4;
    const int nact = p.routes->nactive;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t nn = n0 + n < p.H ? n0 + n : p.H - 1;
    float mean = 0.0f;
    if constexpr (F == kLevels) {
        build_table(lds, p.w.levels, tid, kThreads);
        if (p.w.nested) mean = *p.w.dq_mean;
        __syncthreads();
    }
    const int tok = Two ? n : (n & 7);                   // token of the lane's activation row
    const int wt0 = Two ? 4 * hq : (4 * hq) & 7;         // token of the lane's first accumulator

    floatx4_t y = {0, 0, 0, 0};
    struct Job {
        u32x4_t code;
        u32x4_t a[kParts][4];
        typename Scales<F, NG>::type sc;
        floatx4_t wt;
    };
    Job job[2];
    const int njobs = nact * p.nchunk;
    auto fetch = [&](Job& jb, int q) {
        const int a = q / p.nchunk, c = q % p.nchunk;
        const int64_t row = (int64_t)p.routes->expert[a] * p.H + nn;
        jb.code = load_codes(p.w.codes + row * p.w.stride, p.w.stride, c, hq);
        jb.sc.load(p.w, row, c);
        jb.wt = *reinterpret_cast<const floatx4_t*>(&p.routes->w[a][wt0]);
        const int r = p.routes->hrow[a][tok];
        const uint16_t* src = p.h + (int64_t)r * (2 * p.Ipad) + (c * kChunk + 8 * hq) * 2 + (Two ? 0 : 8 * (n >> 3));
#pragma unroll
        for (int s = 0; s < kParts; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                jb.a[s][j] = (u32x4_t){0, 0, 0, 0};
                if (r >= 0) jb.a[s][j] = *reinterpret_cast<const u32x4_t*>(src + 64 * j + 8 * s);
            }
    };
    auto compute = [&](Job& jb) {
        u32x4_t w = jb.code;
        transpose_groups(w);
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            floatx4_t acc = {0, 0, 0, 0}, xs = {0, 0, 0, 0};
#pragma unroll
            for (int j = q * kGroupMfmas; j < (q + 1) * kGroupMfmas; ++j) {
                u32x4_t b;
                if constexpr (F == kLevels) b = decode8_table(lds, w[j], 4 * lane);
                else b = decode8<F>(w[j]);
#pragma unroll
                for (int s = 0; s < kParts; ++s) {
                    acc = mfma<F>(jb.a[s][j], b, acc);
                    if constexpr (F != kLevels) xs = mfma<F>(jb.a[s][j], ones<F>(), xs);
                }
            }
            float s;
            if constexpr (F == kLevels) s = jb.sc.scale(p.w, mean, q);
            else s = jb.sc.scale(p.w, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = acc[i];
                if constexpr (F != kLevels) v = fmaf(-((float)jb.sc.z[q] + kCodeBias<F>), xs[i], v);
                y[i] = fmaf(s * jb.wt[i], v, y[i]);
            }
        }
    };

    if (wave < njobs) fetch(job[0], wave);
    for (int q = wave; q < njobs; q += 2 * W) {
        if (q + W < njobs) fetch(job[1], q + W);
        compute(job[0]);
        if (q + W < njobs) {
            if (q + 2 * W < njobs) fetch(job[0], q + 2 * W);
            compute(job[1]);
        }
    }

    __syncthreads();                                     // the last table reads
    floatx4_t* red = reinterpret_cast<floatx4_t*>(lds);
    red[wave * 64 + lane] = y;
    __syncthreads();
    if (tid < 256) {
        const int l = tid >> 2, m = 4 * (l >> 4) + (tid & 3);
        const float* redf = reinterpret_cast<const float*>(lds);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            float u = redf[w * 256 + tid];
            if (!Two && tid < 128) u += redf[w * 256 + tid + 128];     // the lo part: lane + 32
            v += u;
        }
        const int64_t o = n0 + (l & 15);
        if (m < p.T && o < p.H) p.y[m * p.H + o] = float_to_bits16(v, p.y_f16);
    }
}

template <int F, int NG>
hipError_t launch_up(const UpArgs<F>& p, int32_t amax, hipStream_t s) {
    constexpr int W = kUpWaves<F>;
    const size_t lds = std::max<size_t>((F == kLevels ? kTabBytes : 0) + (size_t)p.T * kUpPitch<F>,
                                        (size_t)W * 2 * 64 * 16);
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&moe_up_kernel<F, NG>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    moe_up_kernel<F, NG><<<dim3((unsigned)(p.Ipad / 16), (unsigned)amax), dim3(W * 64), lds, s>>>(p);
    return hipGetLastError();
}

template <int F, int NG>
hipError_t launch_down(const DownArgs<F>& p, hipStream_t s) {
    const size_t lds = F == kLevels ? kTabBytes : kDownWaves * 64 * 16;
    const dim3 grid((unsigned)((p.H + 15) / 16));
    if (p.T > 8) moe_down_kernel<F, NG, true><<<grid, dim3(kDownWaves * 64), lds, s>>>(p);
    else moe_down_kernel<F, NG, false><<<grid, dim3(kDownWaves * 64), lds, s>>>(p);
    return hipGetLastError();
}

LevelsView levels_view(const MatArgs& w) {
    LevelsView v;
    v.codes = w.w.codes;
    v.absmax = w.w.absmax;
    v.q8 = w.w.q8;
    v.dq_scale = w.w.dq_scale;
    v.dq_mean = w.w.dq_mean;
    v.stride = w.K / 2;
    v.last_block = (w.w.n + w.w.blocksize - 1) / w.w.blocksize - 1;
    v.bshift = w.w.blocksize_log2;
    v.nested = w.w.nested;
    for (int i = 0; i < 16; ++i) v.levels[i] = w.w.levels[i];
    return v;
}

constexpr size_t kRoutesBytes = (sizeof(Routes) + 255) / 256 * 256;

struct Buffers {
    Routes* routes;
    uint16_t* h;
};
Buffers buffers(void* workspace) {
    uint8_t* b = static_cast<uint8_t*>(workspace);
    return {reinterpret_cast<Routes*>(b), reinterpret_cast<uint16_t*>(b + kRoutesBytes)};
}

template <int F>
UpArgs<F> up_args(const MoeItem& m, const Buffers& b) {
    UpArgs<F> p;
    p.x = static_cast<const uint16_t*>(m.x);
    p.routes = b.routes;
    p.h = b.h;
    p.H = m.H;
    p.I = m.I;
    p.Ipad = (m.I + kChunk - 1) / kChunk * kChunk;
    p.T = m.T;
    p.x_aligned = m.H % 8 == 0 && reinterpret_cast<uintptr_t>(m.x) % 16 == 0;
    return p;
}

template <int F>
DownArgs<F> down_args(const MoeItem& m, const Buffers& b) {
    DownArgs<F> p;
    p.h = b.h;
    p.routes = b.routes;
    p.y = static_cast<uint16_t*>(m.y);
    p.H = m.H;
    p.Ipad = (m.I + kChunk - 1) / kChunk * kChunk;
    p.nchunk = (int32_t)(p.Ipad / kChunk);
    p.T = m.T;
    p.y_f16 = m.f16;
    p.pad = 0;
    return p;
}

template <int F>
hipError_t launch_up_int4(const MoeItem& m, const Buffers& b, const qk_int4_state* w, int32_t amax, hipStream_t s) {
    UpArgs<F> p = up_args<F>(m, b);
    p.w = int4_view(w);
    const int ng = int4_groups_per_chunk(w->group);
    if (ng == 4) return launch_up<F, 4>(p, amax, s);
    if (ng == 2) return launch_up<F, 2>(p, amax, s);
    return launch_up<F, 1>(p, amax, s);
}

hipError_t launch_route(const MoeItem& m, const Buffers& b, hipStream_t s) {
    RouteArgs r{m.logits, m.logits_dtype, m.T, m.E, m.top_k, m.renorm};
    moe_route_kernel<<<dim3(1), dim3(kMaxT * 64), 0, s>>>(r, b.routes);
    return hipGetLastError();
}

}  // namespace

size_t moe_workspace_bytes(int32_t T, int32_t top_k, int64_t I) {
    const size_t ipad = ((size_t)I + kChunk - 1) / kChunk * kChunk;
    return kRoutesBytes + (size_t)T * (size_t)top_k * ipad * 4;
}

hipError_t launch_moe_int4(const MoeItem& m, const qk_int4_state* gate_up, const qk_int4_state* down, void* workspace,
                           hipStream_t s) {
    const Buffers b = buffers(workspace);
    const int32_t amax = std::min(m.E, m.T * m.top_k);
    hipError_t e = launch_route(m, b, s);
    if (e != hipSuccess) return e;
    e = m.f16 ? launch_up_int4<kInt4F16>(m, b, gate_up, amax, s) : launch_up_int4<kInt4Bf16>(m, b, gate_up, amax, s);
    if (e != hipSuccess) return e;
    DownArgs<kInt4Bf16> p = down_args<kInt4Bf16>(m, b);
    p.w = int4_view(down);
    const int ng = int4_groups_per_chunk(down->group);
    if (ng == 4) return launch_down<kInt4Bf16, 4>(p, s);
    if (ng == 2) return launch_down<kInt4Bf16, 2>(p, s);
    return launch_down<kInt4Bf16, 1>(p, s);
}

hipError_t launch_moe_levels(const MoeItem& m, const MatArgs& gate_up, const MatArgs& down, void* workspace,
                             hipStream_t s) {
    const Buffers b = buffers(workspace);
    const int32_t amax = std::min(m.E, m.T * m.top_k);
    hipError_t e = launch_route(m, b, s);
    if (e != hipSuccess) return e;
    UpArgs<kLevels> u = up_args<kLevels>(m, b);
    u.w = levels_view(gate_up);
    e = launch_up<kLevels, 2>(u, amax, s);
    if (e != hipSuccess) return e;
    DownArgs<kLevels> d = down_args<kLevels>(m, b);
    d.w = levels_view(down);
    return launch_down<kLevels, 2>(d, s);
}

}  // namespace qk
