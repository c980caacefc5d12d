// A mixture-of-experts layer for a few tokens over 4-bit experts, for gfx950:
//     S_t     = the top_k largest of logits[t, :], ties to the lower index
//     w[t, e] = exp(L[t, e] - max) / sum (over S_t, or over every expert)
//     h[t, e] = silu(x_t Wg_e^T) * (x_t Wu_e^T)
//     y_t     = sum over e in S_t of w[t, e] h[t, e] Wd_e^T
// with the weights of all experts stacked in two quantized tensors, gate and up rows of an
// expert one after the other in the first.
//
//   moe_up_kernel       routes first: selects each token's experts and lists the experts that have a token in
//                       increasing order, each with its tokens, their weights and their pairs (token, position).
//                       Then items of 16 rows of gate and the same 16 of up of a listed expert (RowTiles,
//                       w4_tile.h), dealt in equal shares; only the expert's own tokens are staged.  h is fp32.
//   moe_down_kernel     items of rows of Wd of a listed expert times its tokens' h, which enters the matrix cores as two
//                       values, hi + lo (w4_tile.h: 24 bits of mantissa); w h Wd^T goes to memory in fp32.
//   moe_combine_kernel  adds each token's parts in the order of its choices: no atomics.  Adding them in the down
//                       kernel, by the wave that stores the last part, made that 82 us instead of 22 (16 tokens, top
//                       8 of 64, 2048 x 1024): every wave then waits for its stores to reach memory.
// Every weight of a listed expert is read once per listing; that is the bound.  At 6 TB/s, which a read of large
// weights reaches, one token's top 2 of 8 experts of 4096 x 11008 take 24 us, measured 40; of 64 experts of
// 2048 x 1024 with top 8 one token takes 4.4, measured 19.3 (three launches, one round of loads each), sixteen
// tokens 31, measured 59 in int4 and 66 in NF4, whose table reads from LDS take as long as the loads.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "qk_device.h"
#include "qk_internal.h"
#include "w4_tile.h"

namespace qk {
namespace {

using namespace w4;

constexpr int kMaxT = 16;
constexpr int kMaxE = 256;
constexpr int kMaxK = 16;
constexpr int kMaxPairs = kMaxT * kMaxK;
template <int F>
constexpr int kThreads = 64 * w4_waves((Form)F);

// Routing result: the experts that have a token, in increasing order, and their tokens, in increasing
// order, one after the other.  An expert with more tokens than the up kernel takes at once is listed again for
// the rest of them, so that every listing is the same work (its weights are then read more than once, from cache
// mostly).
struct Routes {
    int32_t listed;
    int32_t pad[3];
    int32_t chosen[kMaxT];                // experts of each token (its positions 0, 1, ... are taken)
    int32_t expert[kMaxPairs];
    int32_t start[kMaxPairs + 4];         // first entry of each listed expert below; one more ends the last
    float w[kMaxPairs];                   // weight of the entry
    uint8_t tok[kMaxPairs];               // its token
    uint8_t pair[kMaxPairs];              // its row of h: t * top_k + position
};
static_assert(sizeof(Routes) % 16 == 0);

struct RouteArgs {
    const void* logits;
    int32_t dtype;
    int32_t T, E, top_k, renorm;
    int32_t most;                         // tokens of a listing, at most
};

__device__ __forceinline__ float load_logit(const void* p, int32_t dtype, int i) {
    float v;
    if (dtype == QK_F32) v = static_cast<const float*>(p)[i];
    else if (dtype == QK_F16) v = f16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
    else v = bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
    return v == v ? v : -INFINITY;                       // a NaN logit is never chosen
}

// Scratch of route(), in LDS.
struct RouteScratch {
    int32_t who[kMaxT][kMaxK];            // the experts of a token, by position
    float w[kMaxT][kMaxK];                // their weights
    uint32_t mask[kMaxE];                 // tokens of each expert
    int32_t first[kMaxE];                 // its first entry
    int32_t total[4];
};

// Sum over 16 lanes, in every one of them.
__device__ __forceinline__ float row_sum(float v) {
    v += as_float(__builtin_amdgcn_mov_dpp(as_uint(v), 0xB1, 0xF, 0xF, false));    // xor 1
    v += as_float(__builtin_amdgcn_mov_dpp(as_uint(v), 0x4E, 0xF, 0xF, false));    // xor 2
    v += as_float(__builtin_amdgcn_mov_dpp(as_uint(v), 0x141, 0xF, 0xF, false));   // half mirror
    v += as_float(__builtin_amdgcn_mov_dpp(as_uint(v), 0x140, 0xF, 0xF, false));   // mirror
    return v;
}

template <int kCtrl, int kRows = 0xF>
__device__ __forceinline__ float dpp_max(float v) {
    return fmaxf(v, as_float(__builtin_amdgcn_update_dpp(as_uint(v), as_uint(v), kCtrl, kRows, 0xF, false)));
}
// Largest over the wave, as a scalar.
__device__ __forceinline__ float wave_max(float v) {
    v = dpp_max<0xB1>(v);
    v = dpp_max<0x4E>(v);
    v = dpp_max<0x141>(v);
    v = dpp_max<0x140>(v);
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    return as_float(__builtin_amdgcn_readlane(as_uint(v), 63));
}

// Fills r (LDS) from the logits, by one workgroup of kThr threads.  A wave chooses for a token: its lanes hold the
// logits of experts lane, lane + 64, ..., and each choice is the wave's maximum, at the lowest index that has it.
// (Counting for every logit how many are larger needs no rounds, but E comparisons a logit: 16 tokens, top 8 of 256
// experts of 256 x 64, 71 us for the layer against 20; of 64 experts 18.9 against 19.1.)  The loops stay rolled: the code
// runs once, and fetching it is much of its time.
template <int kThr>
__device__ __forceinline__ void route(const RouteArgs& a, RouteScratch& s, Routes& r) {
    constexpr int kPer = kMaxE / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid < kMaxE) s.mask[tid] = 0;
    __syncthreads();
#pragma unroll 1
    for (int t = __builtin_amdgcn_readfirstlane(wave); t < a.T; t += kThr / 64) {
        float v[kPer], left[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 64 * i;
            v[i] = e < a.E ? load_logit(a.logits, a.dtype, t * a.E + e) : -INFINITY;
            left[i] = v[i];
        }
        float mine = 0.0f, top = 0.0f;                   // lane k: the logit of choice k
        int who = 0, chosen = 0;
#pragma unroll 1
        while (chosen < a.top_k) {
            const float m = wave_max(fmaxf(fmaxf(left[0], left[1]), fmaxf(left[2], left[3])));
            if (m == -INFINITY) break;
            int e = 0;
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i) {
                const uint64_t at = __ballot(left[i] == m);
                if (at) e = 64 * i + __builtin_ctzll(at);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 64 * i == e) left[i] = -INFINITY;
            if (lane == chosen) {
                mine = m;
                who = e;
            }
            if (chosen == 0) top = m;
            ++chosen;
        }
        const float p = lane < chosen ? expf(mine - top) : 0.0f;
        float den = row_sum(p);
        if (!a.renorm) {                                 // the sum over every expert instead
            float all = 0.0f;
#pragma unroll 1
            for (int i = 0; i < kPer; ++i) {
                const float x = v[0];
                v[0] = v[1];
                v[1] = v[2];
                v[2] = v[3];
                all += x != -INFINITY ? expf(x - top) : 0.0f;
            }
            all = row_sum(all);
            den = (as_float(__builtin_amdgcn_readlane(as_uint(all), 0)) + as_float(__builtin_amdgcn_readlane(as_uint(all), 16))) +
                  (as_float(__builtin_amdgcn_readlane(as_uint(all), 32)) + as_float(__builtin_amdgcn_readlane(as_uint(all), 48)));
        }
        if (lane == 0) r.chosen[t] = chosen;
        if (lane < chosen) {
            s.who[t][lane] = who;
            s.w[t][lane] = p / den;
            atomicOr(&s.mask[who], 1u << t);
        }
    }
    __syncthreads();
    uint32_t mk = 0;
    int scan = 0;                                        // tokens of the experts up to here, and listings << 16
    if (tid < kMaxE) {
        mk = s.mask[tid];
        scan = wave_scan(__popc(mk) + ((__popc(mk) + a.most - 1) / a.most << 16));
        if (lane == 63) s.total[wave] = scan;
    }
    __syncthreads();
    if (tid < kMaxE) {
        const int tokens = __popc(mk), listings = (tokens + a.most - 1) / a.most;
        int before = scan - tokens - (listings << 16), all = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) before += s.total[w];
            all += s.total[w];
        }
        const int first = before & 0xFFFF, slot = before >> 16;
        s.first[tid] = first;
#pragma unroll 1
        for (int i = 0; i < listings; ++i) {
            r.expert[slot + i] = tid;
            r.start[slot + i] = first + i * a.most;
        }
        if (tid == 0) {
            r.listed = all >> 16;
            r.start[all >> 16] = all & 0xFFFF;
        }
    }
    __syncthreads();
    const int t = tid / kMaxK, k = tid % kMaxK;          // choice k of token t
    if (t < a.T && k < r.chosen[t]) {
        const int e = s.who[t][k], at = s.first[e] + __popc(s.mask[e] & ((1u << t) - 1));
        r.tok[at] = (uint8_t)t;
        r.pair[at] = (uint8_t)(t * a.top_k + k);
        r.w[at] = s.w[t][k];
    }
    __syncthreads();
}

// A weight view of either form.
template <int F>
struct View {
    typedef Int4View type;
};
template <>
struct View<kLevels> {
    typedef LevelsView type;
};

template <int F>
struct ExpertArgs {
    const void* x;           // up: x [T, H], 16-bit; down: h [T * top_k, Ipad], fp32
    typename View<F>::type w;
    const Routes* routes;
    float* out;              // up: h; down: the parts [T * top_k, H]
    int32_t H;
    int32_t I;
    int32_t Ipad;            // I rounded up to 8 values
    uint32_t grid;           // workgroups
    int32_t x_rows;
    int32_t x_aligned;
    int32_t kwl;
};

// Workgroups per CU, at most: the level table takes 64 KB of its LDS.
template <int F>
constexpr int kPerCu = F == kLevels ? 1 : 2;
template <int F>
int64_t workgroups(int64_t items, size_t lds) {
    return std::min<int64_t>(items, (lds > kLdsBytes / 2 ? 1 : kPerCu<F>) * device_cu_count());
}
// LDS of the activations; those of a whole row stay there where all of them fit.
template <int F, int MI>
size_t x_lds(int tokens, bool split, int64_t K, bool resident) {
    constexpr int kw = 1 << w4_most_kwl((Form)F, MI);
    return w4_x_bytes((Form)F, kw, split ? 2 * tokens : tokens, MI, split, K, resident);
}
template <int F, int NG, int RT, int MI>
bool fits(int tokens, bool split, int64_t K) {
    return (F == kLevels ? kTabBytes : 0) + sizeof(Routes) + w4_fixed_bytes((Form)F, NG, RT, MI, true) +
               x_lds<F, MI>(tokens, split, K, true) <= kLdsBytes;
}
// Tokens that a pass over an expert's rows takes; the down product needs two operand rows for one.
template <int MI, bool kSplit>
constexpr int kTokens = kSplit ? 2 * MI : 4 * MI;

template <int F, int NG, int MI, bool kResident>
__global__ __launch_bounds__(kThreads<F>, 4) void moe_up_kernel(ExpertArgs<F> p, RouteArgs ra, Routes* keep) {
    extern __shared__ __align__(16) uint8_t lds[];
    typedef RowTiles<F, NG, 2, MI, kResident, false> Tiles;
    uint8_t* work = lds + (F == kLevels ? kTabBytes : 0) + sizeof(Routes);
    static_assert(sizeof(RouteScratch) <= Tiles::kFixedBytes);
    // Every workgroup routes for itself (a launch of its own would cost more); the first one keeps the result.
    Routes& routes = *reinterpret_cast<Routes*>(lds + (F == kLevels ? kTabBytes : 0));
    route<kThreads<F>>(ra, *reinterpret_cast<RouteScratch*>(work), routes);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < (int)(sizeof(Routes) / 4); i += kThreads<F>)
            reinterpret_cast<uint32_t*>(keep)[i] = reinterpret_cast<const uint32_t*>(&routes)[i];
    if constexpr (F == kLevels) build_table(lds, p.w.levels, threadIdx.x, kThreads<F>);
    // an item: per row group 16 rows of gate and the same of up of one listed expert; equal shares of the items
    const int step = (16 * Tiles::W) >> p.kwl;
    const uint32_t tiles = (uint32_t)(p.Ipad + step - 1) / step, all = tiles * (uint32_t)routes.listed;
    const uint32_t share = all / p.grid, more = all % p.grid, b = blockIdx.x;
    uint32_t lo = b * share + (b < more ? b : more);
    const uint32_t hi = lo + share + (b < more);
    while (lo < hi) {
        const int a = (int)(lo / tiles);
        const int i0 = (int)(lo - a * tiles), i1 = (int)(hi - a * tiles < tiles ? hi - a * tiles : tiles);
        lo += i1 - i0;
        const int first = routes.start[a], count = routes.start[a + 1] - first;
        const int64_t e = routes.expert[a];
        Rows<2> r;
        r.base[0] = e * 2 * p.I;
        r.base[1] = r.base[0] + p.I;
        r.off[0] = r.off[1] = 0;
        r.step = step;
        r.group_step = 16;
        r.count = p.I;
        r.x = p.x;
        r.K = r.x_pitch = p.H;
        r.x_rows = p.x_rows;
        r.x_aligned = p.x_aligned;
        r.kwl = p.kwl;
        r.xrow = routes.tok + first;
        r.M = count;
        Tiles::run(p.w, r, i0, i1, work, [&](int item, int q, const float* put) {
#pragma unroll
            for (int s = threadIdx.x & 63; s < 64 * MI; s += 64) {
                const int m = Tiles::act_of(s);
                const int i = item * step + 16 * q + (s & 15);
                if (m < count && i < p.Ipad) {
                    const float gate = Tiles::sum(put, p.kwl, q, 0, s), up = Tiles::sum(put, p.kwl, q, 1, s);
                    const float v = gate / (1.0f + expf(-gate)) * up;
                    p.out[(int64_t)routes.pair[first + m] * p.Ipad + i] = i < p.I ? v : 0.0f;
                }
            }
        });
    }
}

template <int F, int NG, int RT, int MI, bool kResident>
__global__ __launch_bounds__(kThreads<F>, 4) void moe_down_kernel(ExpertArgs<F> p) {
    extern __shared__ __align__(16) uint8_t lds[];
    typedef RowTiles<F, NG, RT, MI, kResident, true> Tiles;
    uint8_t* work = lds + (F == kLevels ? kTabBytes : 0);
    if constexpr (F == kLevels) build_table(lds, p.w.levels, threadIdx.x, kThreads<F>);
    const int step = (16 * RT * Tiles::W) >> p.kwl;
    const uint32_t tiles = (uint32_t)(p.H + step - 1) / step, all = tiles * (uint32_t)p.routes->listed;
    const uint32_t share = all / p.grid, more = all % p.grid, b = blockIdx.x;
    uint32_t lo = b * share + (b < more ? b : more);
    const uint32_t hi = lo + share + (b < more);
    while (lo < hi) {
        const int a = (int)(lo / tiles);
        const int i0 = (int)(lo - a * tiles), i1 = (int)(hi - a * tiles < tiles ? hi - a * tiles : tiles);
        lo += i1 - i0;
        const int first = p.routes->start[a], count = p.routes->start[a + 1] - first;
        Rows<RT> r;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            r.base[t] = (int64_t)p.routes->expert[a] * p.H;
            r.off[t] = 16 * t;
        }
        r.step = step;
        r.group_step = 16 * RT;
        r.count = p.H;
        r.x = p.x;
        r.K = p.I;
        r.x_pitch = p.Ipad;
        r.x_rows = p.x_rows;
        r.x_aligned = 1;
        r.kwl = p.kwl;
        constexpr int kTok = kTokens<MI, true>;
        for (int m0 = 0; m0 < count; m0 += kTok) {
            const int M = count - m0 < kTok ? count - m0 : kTok;
            r.xrow = p.routes->pair + first + m0;
            r.M = M;
            Tiles::run(p.w, r, i0, i1, work, [&](int item, int q, const float* put) {
                for (int o = threadIdx.x & 63; o < M * (16 * RT); o += 64) {
                    const int m = o / (16 * RT), row = o % (16 * RT), t = row / 16;
                    const int n = item * step + q * (16 * RT) + row;
                    // two operand rows a token
                    const float v = Tiles::sum(put, p.kwl, q, t, Tiles::place_of(row & 15, 2 * m)) +
                                    Tiles::sum(put, p.kwl, q, t, Tiles::place_of(row & 15, 2 * m + 1));
                    if (n < p.H) p.out[(int64_t)p.routes->pair[first + m0 + m] * p.H + n] = v * p.routes->w[first + m0 + m];
                }
            });
        }
    }
}

__global__ __launch_bounds__(256) void moe_combine_kernel(const float* parts, const Routes* routes, uint16_t* y,
                                                          int64_t H, int32_t top_k, int32_t f16) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int t = blockIdx.y;
    if (n >= H) return;
    const int chosen = routes->chosen[t];
    const float* src = parts + (int64_t)t * top_k * H + n;
    float v = 0.0f;
    // eight loads on their way at a time, beside that of `chosen` (what lies behind it is stale and not added)
    for (int k0 = 0; k0 < top_k; k0 += 8) {
        float part[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) part[k] = src[(k0 + k < top_k ? k0 + k : k0) * H];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < chosen) v += part[k];
    }
    y[t * H + n] = float_to_bits16(v, f16);
}

// tokens: that a pass stages at most; listed: the most listings that there can be
template <int F, int NG, int MI, bool kResident>
hipError_t launch_up_one(ExpertArgs<F> p, const RouteArgs& ra, Routes* keep, int tokens, int32_t listed, hipStream_t s) {
    typedef RowTiles<F, NG, 2, MI, kResident, false> Tiles;
    p.kwl = w4_kwl((Form)F, p.H, (int64_t)p.Ipad * listed, 16, kResident ? 3 : w4_most_kwl((Form)F, MI));
    const size_t lds = (F == kLevels ? kTabBytes : 0) + sizeof(Routes) + Tiles::kFixedBytes +
                       x_lds<F, MI>(tokens, false, p.H, kResident);
    const hipError_t e = allow_lds<&moe_up_kernel<F, NG, MI, kResident>>(lds);
    if (e != hipSuccess) return e;
    const int step = (16 * Tiles::W) >> p.kwl;
    const int64_t items = (int64_t)(p.Ipad + step - 1) / step * listed;
    p.grid = (uint32_t)workgroups<F>(items, lds);
    moe_up_kernel<F, NG, MI, kResident><<<dim3(p.grid), dim3(kThreads<F>), lds, s>>>(p, ra, keep);
    return hipGetLastError();
}

template <int F, int NG, int MI>
hipError_t launch_up_mi(const ExpertArgs<F>& p, RouteArgs ra, Routes* keep, int32_t* listed, hipStream_t s) {
    const int tokens = std::min(ra.T, kTokens<MI, false>);
    ra.most = kTokens<MI, false>;
    *listed = std::min(ra.E * ((ra.T + ra.most - 1) / ra.most), ra.T * ra.top_k);
    if (fits<F, NG, 2, MI>(tokens, false, p.H)) return launch_up_one<F, NG, MI, true>(p, ra, keep, tokens, *listed, s);
    return launch_up_one<F, NG, MI, false>(p, ra, keep, tokens, *listed, s);
}

// Tokens of a listing, four or eight, by how many an expert has on average: eight read the weights of crowded experts
// less often, four take less LDS and half the registers.  Weights from memory, four / eight (the down product likewise):
// 16 tokens, top 2 of 8 experts, H = I = 4096 (4 an expert), int4 95 / 66 us, levels 110 / 84; 12 tokens (3 an expert),
// int4 79 / 64, levels 100 / 82; top 8 of 64, 2048 x 1024 (2 an expert), int4 63 / 75, levels 69 / 85.  Sixteen gained 2 %
// where every expert has 16 and lost 10 % at 6.
// listed: set to the most listings that there can be
template <int F, int NG>
hipError_t launch_up(const ExpertArgs<F>& p, const MoeItem& m, Routes* keep, int32_t* listed, hipStream_t s) {
    const RouteArgs ra{m.logits, m.logits_dtype, m.T, m.E, m.top_k, m.renorm, 0};
    if (m.T <= 4 || m.T * m.top_k < 3 * m.E) return launch_up_mi<F, NG, 1>(p, ra, keep, listed, s);
    return launch_up_mi<F, NG, 2>(p, ra, keep, listed, s);
}

template <int F, int NG, int RT, int MI, bool kResident>
hipError_t launch_down_one(ExpertArgs<F> p, int tokens, int32_t listed, hipStream_t s) {
    typedef RowTiles<F, NG, RT, MI, kResident, true> Tiles;
    p.kwl = w4_kwl((Form)F, p.I, (int64_t)p.H * listed, 16 * RT, kResident ? 3 : w4_most_kwl((Form)F, MI));
    const size_t lds = (F == kLevels ? kTabBytes : 0) + Tiles::kFixedBytes + x_lds<F, MI>(tokens, true, p.I, kResident);
    const hipError_t e = allow_lds<&moe_down_kernel<F, NG, RT, MI, kResident>>(lds);
    if (e != hipSuccess) return e;
    const int64_t step = (16 * RT * Tiles::W) >> p.kwl, items = (p.H + step - 1) / step * listed;
    p.grid = (uint32_t)workgroups<F>(items, lds);
    moe_down_kernel<F, NG, RT, MI, kResident><<<dim3(p.grid), dim3(kThreads<F>), lds, s>>>(p);
    return hipGetLastError();
}

template <int F, int NG, int MI>
hipError_t launch_down_mi(const ExpertArgs<F>& p, int32_t T, int32_t listed, hipStream_t s) {
    const int tokens = std::min(T, kTokens<MI, true>);
    constexpr int RT = MI == 4 ? 1 : 2;                  // (eight tokens beside two tiles do not fit the registers)
    if (!fits<F, NG, RT, MI>(tokens, true, p.I)) return launch_down_one<F, NG, RT, MI, false>(p, tokens, listed, s);
    return launch_down_one<F, NG, RT, MI, true>(p, tokens, listed, s);
}

// Tokens of a pass of the down product, two or four, in int4 eight where experts are crowded (see above).  Two at a time,
// weights from memory: four tokens of top 8 of 64 experts int4 35.9 us instead of 35.0, levels 43.4 instead of 42.2; four
// at a time, two tokens of one expert, 4096 x 4096: int4 equal, levels 37 us instead of 29.
template <int F, int NG>
hipError_t launch_down(const ExpertArgs<F>& p, const MoeItem& m, int32_t listed, hipStream_t s) {
    if (m.T <= 2) return launch_down_mi<F, NG, 1>(p, m.T, listed, s);
    if constexpr (F != kLevels)
        if (m.T > 4 && m.T * m.top_k >= 3 * m.E) return launch_down_mi<F, NG, 4>(p, m.T, listed, s);
    return launch_down_mi<F, NG, 2>(p, m.T, listed, s);
}

// The bf16 copy of a level, as qk_gemv_nf4 reads it.
float bf16_copy(float v) {
    uint32_t u;
    std::memcpy(&u, &v, 4);
    u = (u + 0x7FFFu + (u >> 16 & 1)) & 0xFFFF0000u;
    std::memcpy(&v, &u, 4);
    return v;
}

LevelsView levels_view(const MatArgs& w) {
    LevelsView v;
    v.codes = w.w.codes;
    v.absmax = w.w.absmax;
    v.q8 = w.w.q8;
    v.dq_scale = w.w.dq_scale;
    v.dq_mean = w.w.dq_mean;
    v.stride = w.K / 2;
    v.bshift = w.w.blocksize_log2;
    v.nested = w.w.nested;
    float most = 0.0f;
    for (int i = 0; i < 16; ++i) most = std::max(most, std::fabs(bf16_copy(w.w.levels[i])));
    int k = 0;
    if (most > 0.0f && std::isfinite(most)) k = 14 - std::ilogb(most);
    for (int i = 0; i < 16; ++i) v.levels[i] = std::ldexp(bf16_copy(w.w.levels[i]), k);
    v.unit = std::ldexp(1.0f, -k);
    return v;
}

// The workspace: routes, h, parts.
constexpr size_t kRoutesBytes = (sizeof(Routes) + 255) / 256 * 256;
size_t h_bytes(int32_t T, int32_t top_k, int64_t I) {
    return ((size_t)T * (size_t)top_k * (size_t)((I + 7) / 8 * 8) * 4 + 255) / 256 * 256;
}

struct Buffers {
    Routes* routes;
    float* h;
    float* parts;
};
Buffers buffers(const MoeItem& m, void* workspace) {
    uint8_t* b = static_cast<uint8_t*>(workspace);
    return {reinterpret_cast<Routes*>(b), reinterpret_cast<float*>(b + kRoutesBytes),
            reinterpret_cast<float*>(b + kRoutesBytes + h_bytes(m.T, m.top_k, m.I))};
}

template <int F>
ExpertArgs<F> expert_args(const MoeItem& m, const Buffers& b, bool up) {
    ExpertArgs<F> p;
    p.x = up ? m.x : b.h;
    p.routes = b.routes;
    p.out = up ? b.h : b.parts;
    p.H = (int32_t)m.H;
    p.I = (int32_t)m.I;
    p.Ipad = (int32_t)((m.I + 7) / 8 * 8);
    p.grid = 0;
    p.x_rows = up ? m.T : m.T * m.top_k;
    p.x_aligned = !up || (m.H % 8 == 0 && reinterpret_cast<uintptr_t>(m.x) % 4 == 0);
    p.kwl = 0;
    return p;
}

template <int F>
hipError_t launch_up_int4(const MoeItem& m, const Buffers& b, const qk_int4_state* w, int32_t* listed, hipStream_t s) {
    ExpertArgs<F> p = expert_args<F>(m, b, true);
    p.w = int4_view(w);
    const int ng = int4_groups_per_chunk(w->group);
    if (ng == 4) return launch_up<F, 4>(p, m, b.routes, listed, s);
    if (ng == 2) return launch_up<F, 2>(p, m, b.routes, listed, s);
    return launch_up<F, 1>(p, m, b.routes, listed, s);
}

hipError_t launch_combine(const MoeItem& m, const Buffers& b, hipStream_t s) {
    moe_combine_kernel<<<dim3((unsigned)((m.H + 255) / 256), (unsigned)m.T), dim3(256), 0, s>>>(
        b.parts, b.routes, static_cast<uint16_t*>(m.y), m.H, m.top_k, m.f16);
    return hipGetLastError();
}

}  // namespace

size_t moe_workspace_bytes(int32_t T, int32_t top_k, int64_t H, int64_t I) {
    return kRoutesBytes + h_bytes(T, top_k, I) + (size_t)T * (size_t)top_k * (size_t)H * 4;
}

hipError_t launch_moe_int4(const MoeItem& m, const qk_int4_state* gate_up, const qk_int4_state* down, void* workspace,
                           hipStream_t s) {
    const Buffers b = buffers(m, workspace);
    int32_t listed = 0;
    hipError_t e = m.f16 ? launch_up_int4<kInt4F16>(m, b, gate_up, &listed, s) : launch_up_int4<kInt4Bf16>(m, b, gate_up, &listed, s);
    if (e != hipSuccess) return e;
    ExpertArgs<kInt4Bf16> p = expert_args<kInt4Bf16>(m, b, false);
    p.w = int4_view(down);
    const int ng = int4_groups_per_chunk(down->group);
    e = ng == 4 ? launch_down<kInt4Bf16, 4>(p, m, listed, s)
        : ng == 2 ? launch_down<kInt4Bf16, 2>(p, m, listed, s) : launch_down<kInt4Bf16, 1>(p, m, listed, s);
    if (e != hipSuccess) return e;
    return launch_combine(m, b, s);
}

hipError_t launch_moe_levels(const MoeItem& m, const MatArgs& gate_up, const MatArgs& down, void* workspace,
                             hipStream_t s) {
    const Buffers b = buffers(m, workspace);
    int32_t listed = 0;
    ExpertArgs<kLevels> u = expert_args<kLevels>(m, b, true);
    u.w = levels_view(gate_up);
    hipError_t e = launch_up<kLevels, 2>(u, m, b.routes, &listed, s);
    if (e != hipSuccess) return e;
    ExpertArgs<kLevels> d = expert_args<kLevels>(m, b, false);
    d.w = levels_view(down);
    e = launch_down<kLevels, 2>(d, m, listed, s);
    if (e != hipSuccess) return e;
    return launch_combine(m, b, s);
}

}  // namespace qk
