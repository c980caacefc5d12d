// Decode product with an int4 weight of group scales and zero points, for gfx950:
//     y[m, n] = sum_k x[m, k] s[n, k / g] (q[n, k] - z[n, k / g]),   m < M <= 16
// for one weight or for up to 16 of a grouped call in one launch.
//
// A workgroup of 8 waves owns 16 RT consecutive rows of one weight; its waves take the row's
// 128-k chunks in turn (chunk w, w + 8, ...) and their partial outputs are added through LDS
// in wave order, so the result does not depend on timing.  The activations of a window of 8 U
// chunks are staged in LDS once for the 8 waves (in the order the decoded codes have, zero past
// K), while the codes of the next window are already being loaded.
// Bound by the bytes of the codes at every M (64 flops a byte at M = 16).
#include <algorithm>

#include "qk_device.h"
#include "qk_internal.h"
#include "w4_tile.h"

namespace qk {
namespace {

using namespace w4;

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;

struct Int4Task {
    const uint16_t* x;       // [M, K]
    uint16_t* y;             // [M, N]
    Int4View w;
    int64_t N;
    int64_t K;
    int64_t item0;           // first workgroup of the task
    int32_t x_aligned;       // rows of x start at 16-byte boundaries
    int32_t pad;
};

struct Int4Group {
    Int4Task t[kMaxGemvTasks];
    int32_t ntasks;
    int32_t M;
};

// bytes of a staged activation row: the window and 16 more, so that the rows of a fragment
// read fall in different banks
template <int U>
constexpr int kPitch = kWaves * U * kChunk * 2 + 16;

template <int F, int NG, int RT, int U>
__global__ __launch_bounds__(kThreads) void int4_gemv_kernel(Int4Group g) {
    extern __shared__ __align__(16) uint8_t lds[];
    constexpr int kWin = kWaves * U * kChunk;          // k per window
    constexpr int kWinUnits = kWin / 8;                // 16-byte units of a row in a window
    constexpr int kGroupChunks = 4 / NG;               // MFMAs per scale
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, h = lane >> 4;
    int ti = 0;
    while (ti + 1 < g.ntasks && (int64_t)blockIdx.x >= g.t[ti + 1].item0) ++ti;
    const Int4Task& t = g.t[ti];
    const int M = g.M;
    const int64_t row0 = ((int64_t)blockIdx.x - t.item0) * (16 * RT);
    const int64_t K = t.K, N = t.N;
    int64_t row[RT];
    const uint8_t* codes[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        row[r] = row0 + 16 * r + n < N ? row0 + 16 * r + n : N - 1;
        codes[r] = t.w.codes + row[r] * t.w.stride;
    }
    const int nchunk = (int)((K + kChunk - 1) / kChunk);
    const int nwin = (nchunk + kWaves * U - 1) / (kWaves * U);

    floatx4_t y[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) y[r] = (floatx4_t){0, 0, 0, 0};
    u32x4_t cw[2][U][RT];
    GroupScales<NG> sc[2][U][RT];

    auto fetch = [&](int buf, int win) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int c = (win * U + u) * kWaves + wave;
            c = c < nchunk ? c : nchunk - 1;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                cw[buf][u][r] = load_codes(codes[r], t.w.stride, c, h);
                sc[buf][u][r].load(t.w, row[r], c);
            }
        }
    };
    auto stage = [&](int win) {
        for (int i = tid; i < M * kWinUnits; i += kThreads) {
            const int m = i / kWinUnits, u = i % kWinUnits;
            const u32x4_t v = load_x8(t.x + m * K, (int64_t)win * kWin + 8 * u, K, t.x_aligned);
            *reinterpret_cast<u32x4_t*>(lds + m * kPitch<U> + 16 * u) = int4_order(v);
        }
    };
    const uint8_t* arow = lds + (n < M ? n : M - 1) * kPitch<U> + 16 * h;
    auto compute = [&](int buf, int win) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if ((win * U + u) * kWaves + wave >= nchunk) break;
            u32x4_t w[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                w[r] = cw[buf][u][r];
                transpose_groups(w[r]);
            }
#pragma unroll
            for (int q = 0; q < NG; ++q) {
                floatx4_t acc[RT], xs = {0, 0, 0, 0};
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[r] = (floatx4_t){0, 0, 0, 0};
#pragma unroll
                for (int j = q * kGroupChunks; j < (q + 1) * kGroupChunks; ++j) {
                    const u32x4_t a =
                        *reinterpret_cast<const u32x4_t*>(arow + (u * kWaves + wave) * (kChunk * 2) + 64 * j);
                    xs = mfma<F>(a, ones<F>(), xs);
#pragma unroll
                    for (int r = 0; r < RT; ++r) acc[r] = mfma<F>(a, decode8<F>(w[r][j]), acc[r]);
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float s = sc[buf][u][r].scale(t.w, q);
                    const float zb = (float)sc[buf][u][r].z[q] + kCodeBias<F>;
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

    // the 8 partial sums of every output, in wave order
    floatx4_t* red = reinterpret_cast<floatx4_t*>(lds);
#pragma unroll
    for (int r = 0; r < RT; ++r) red[(wave * RT + r) * 64 + lane] = y[r];
    __syncthreads();
    const float* redf = reinterpret_cast<const float*>(lds);
    for (int o = tid; o < RT * 256; o += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += redf[w * RT * 256 + o];
        const int r = o >> 8, l = (o >> 2) & 63, m = 4 * (l >> 4) + (o & 3);
        const int64_t nn = row0 + 16 * r + (l & 15);
        if (m < M && nn < N) t.y[m * N + nn] = float_to_bits16(v, F == kInt4F16);
    }
}

template <int F, int NG, int RT, int U>
hipError_t launch_one(const Int4Group& g, int64_t items, hipStream_t s) {
    const size_t lds = std::max<size_t>((size_t)g.M * kPitch<U>, (size_t)kWaves * RT * 64 * 16);
    int4_gemv_kernel<F, NG, RT, U><<<dim3((unsigned)items), dim3(kThreads), lds, s>>>(g);
    return hipGetLastError();
}

template <int F, int NG>
hipError_t launch_m(const Int4Group& g, int64_t items, int rt, hipStream_t s) {
    if (g.M <= 4) return launch_one<F, NG, 1, 2>(g, items, s);
    (void)rt;
    return launch_one<F, NG, 1, 1>(g, items, s);
}

template <int F>
hipError_t launch_ng(const Int4Group& g, int64_t items, int ng, int rt, hipStream_t s) {
    if (ng == 4) return launch_m<F, 4>(g, items, rt, s);
    if (ng == 2) return launch_m<F, 2>(g, items, rt, s);
    return launch_m<F, 1>(g, items, rt, s);
}

}  // namespace

Int4View int4_view(const qk_int4_state* st) {
    Int4View v;
    v.codes = st->codes;
    v.scales = static_cast<const uint16_t*>(st->scales);
    v.zeros = st->zeros;
    v.stride = st->code_stride;
    v.G = st->group ? (int32_t)((st->cols + st->group - 1) / st->group) : 1;
    v.gshift = st->group ? __builtin_ctz((unsigned)st->group) : 30;
    v.scale_f16 = st->scale_dtype == QK_F16;
    v.pad = 0;
    return v;
}

// groups per chunk of 128 k that the kernels tell apart: 4, 2 or 1
int int4_groups_per_chunk(int32_t group) { return group == 32 ? 4 : group == 64 ? 2 : 1; }

hipError_t launch_int4_gemv_group(const Int4Item* items, int32_t count, int32_t M, bool f16, hipStream_t s) {
    // One launch per run of up to kMaxGemvTasks weights of one scale granularity, in task order.
    bool done[256] = {false};
    for (int32_t first = 0; first < count; ++first) {
        if (done[first]) continue;
        const int ng = int4_groups_per_chunk(items[first].st->group);
        Int4Group g;
        g.ntasks = 0;
        g.M = M;
        int64_t item0 = 0;
        for (int32_t i = first; i < count && g.ntasks < kMaxGemvTasks; ++i) {
            if (done[i] || int4_groups_per_chunk(items[i].st->group) != ng) continue;
            const qk_int4_state* st = items[i].st;
            const int64_t tiles = (st->rows + 15) / 16;
            if (g.ntasks > 0 && item0 + tiles > (1 << 24)) break;
            done[i] = true;
            Int4Task& t = g.t[g.ntasks++];
            t.x = static_cast<const uint16_t*>(items[i].x);
            t.y = static_cast<uint16_t*>(items[i].y);
            t.w = int4_view(st);
            t.N = st->rows;
            t.K = st->cols;
            t.item0 = item0;
            t.x_aligned = st->cols % 8 == 0 && reinterpret_cast<uintptr_t>(items[i].x) % 16 == 0;
            t.pad = 0;
            item0 += tiles;
        }
        const hipError_t e = f16 ? launch_ng<kInt4F16>(g, item0, ng, 1, s) : launch_ng<kInt4Bf16>(g, item0, ng, 1, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qk
