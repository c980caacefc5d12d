// Decode product with an int4 weight of group scales and zero points, for gfx950:
//     y[m, n] = sum_k x[m, k] s[n, k / g] (q[n, k] - z[n, k / g]),   m < M <= 16
// for one weight or for up to 16 of a grouped call in one launch.
//
// The rows of all weights of a launch are cut into items of 16 RT rows, and the items, in order,
// into equal shares of work, one per workgroup of 8 waves; a workgroup walks its items with
// RowTiles (w4_tile.h), the next item's codes being loaded while one is multiplied.
// Bound by the bytes of the codes at every M (64 flops a byte at M = 16).
#include <algorithm>

#include "qk_device.h"
#include "qk_internal.h"
#include "w4_tile.h"

namespace qk {
namespace {

using namespace w4;

constexpr int kThreads = 512;

struct Int4Task {
    const uint16_t* x;       // [M, K]
    uint16_t* y;             // [M, N]
    Int4View w;
    int64_t N;
    int64_t K;
    int32_t x_aligned;       // rows of x start at 16-byte boundaries
    int32_t kwl;             // log2 of the waves that split a row
};

struct Int4Group {
    Int4Task t[kMaxGemvTasks];
    int64_t cost0[kMaxGemvTasks + 1];    // work before the task's first item, in chunks of an item
    int32_t chunks[kMaxGemvTasks];       // work of one item
    int32_t ntasks;
    int32_t M;
    int32_t x_bufs;
    int32_t pad;
};

template <int F, int NG, int RT, int NS, int MI, bool kResident>
__global__ __launch_bounds__(kThreads, 2) void int4_gemv_kernel(Int4Group g) {
    extern __shared__ __align__(16) uint8_t lds[];
    typedef RowTiles<F, NG, RT, NS, MI, kResident, false> Tiles;
    // this workgroup's share: the items that start in [lo, hi) of the work
    const int64_t all = g.cost0[g.ntasks];
    const int64_t lo = all * blockIdx.x / gridDim.x, hi = all * (blockIdx.x + 1) / gridDim.x;
    for (int ti = 0; ti < g.ntasks; ++ti) {
        const int64_t c0 = g.cost0[ti], c1 = g.cost0[ti + 1];
        if (c1 <= lo || c0 >= hi) continue;
        const int64_t ch = g.chunks[ti];
        const int64_t i0 = lo > c0 ? (lo - c0 + ch - 1) / ch : 0;
        const int64_t i1 = ((hi < c1 ? hi : c1) - c0 + ch - 1) / ch;
        if (i0 >= i1) continue;
        const Int4Task& t = g.t[ti];
        Rows<RT> p;
        p.kwl = t.kwl;
        p.group_step = 16 * RT;
        p.step = (16 * RT * 8) >> t.kwl;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            p.base[r] = 0;
            p.off[r] = 16 * r;
        }
        p.count = t.N;
        p.x = t.x;
        p.xrow = nullptr;
        p.K = t.K;
        p.x_pitch = t.K;
        p.x_rows = g.M;
        p.x_aligned = t.x_aligned;
        p.M = g.M;
        p.x_bufs = g.x_bufs;
        Tiles::run(t.w, p, i0, i1, nullptr, lds, [&](int64_t item, const float* put) {
            for (int o = threadIdx.x; o < (RT * 64 * MI * 8) >> t.kwl; o += kThreads) {
                const int q = o / (RT * 64 * MI), r = o / (64 * MI) % RT, e = o % (64 * MI), m = Tiles::act_of(e);
                const int64_t n = item * p.step + q * (16 * RT) + 16 * r + (e & 15);
                const float v = Tiles::sum(put, t.kwl, q, r, e);
                if (m < g.M && n < t.N) t.y[m * t.N + n] = float_to_bits16(v, F == kInt4F16);
            }
        });
    }
}

// How a weight of K inputs is cut for M activation rows: tiles per item and row group, lines per wave and
// window, waves that split a row, and whether the activations of a whole row stay in LDS.
struct Shape {
    int rt;
    int ns;
    int kwl;
    bool resident;
};

constexpr size_t kMaxResident = 72 * 1024;

Shape shape_for(int M, int64_t K) {
    if (w4_x_bytes(8, 2, M, K, true, 1) <= kMaxResident) return {2, 2, w4_kwl(2, K), true};
    return {4, 1, 2, false};
}

template <int F, int NG, int RT, int NS, int MI, bool kResident>
hipError_t launch_one(Int4Group& g, int64_t items, int64_t kmax, hipStream_t s) {
    typedef RowTiles<F, NG, RT, NS, MI, kResident, false> Tiles;
    g.x_bufs = 2;
    const size_t lds = Tiles::kFixedBytes + w4_x_bytes(4, NS, g.M, kmax, kResident, 2);
    if (lds > 65536) {
        const hipError_t e =
            hipFuncSetAttribute(reinterpret_cast<const void*>(&int4_gemv_kernel<F, NG, RT, NS, MI, kResident>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    const int64_t grid = std::min<int64_t>(items, device_cu_count());
    int4_gemv_kernel<F, NG, RT, NS, MI, kResident><<<dim3((unsigned)grid), dim3(kThreads), lds, s>>>(g);
    return hipGetLastError();
}

template <int F, int NG, int MI>
hipError_t launch_shape(Int4Group& g, int64_t items, bool resident, int64_t kmax, hipStream_t s) {
    if (resident) return launch_one<F, NG, 2, 2, MI, true>(g, items, kmax, s);
    return launch_one<F, NG, 4, 1, MI, false>(g, items, kmax, s);
}

template <int F, int NG>
hipError_t launch_mi(Int4Group& g, int64_t items, bool resident, int64_t kmax, hipStream_t s) {
    if (g.M <= 4) return launch_shape<F, NG, 1>(g, items, resident, kmax, s);
    if (g.M <= 8) return launch_shape<F, NG, 2>(g, items, resident, kmax, s);
    return launch_shape<F, NG, 4>(g, items, resident, kmax, s);
}

template <int F>
hipError_t launch_ng(Int4Group& g, int64_t items, int ng, bool resident, int64_t kmax, hipStream_t s) {
    if (ng == 4) return launch_mi<F, 4>(g, items, resident, kmax, s);
    if (ng == 2) return launch_mi<F, 2>(g, items, resident, kmax, s);
    return launch_mi<F, 1>(g, items, resident, kmax, s);
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
        // the weights of the launch: one scale granularity, activations that all fit, or all do not
        const bool resident = shape_for(M, items[first].st->cols).resident;
        Int4Group g;
        g.ntasks = 0;
        g.M = M;
        g.cost0[0] = 0;
        int64_t total = 0, kmax = 0;
        for (int32_t i = first; i < count && g.ntasks < kMaxGemvTasks; ++i) {
            const qk_int4_state* st = items[i].st;
            const Shape sh = shape_for(M, st->cols);
            if (done[i] || int4_groups_per_chunk(st->group) != ng || sh.resident != resident) continue;
            done[i] = true;
            const int64_t rows = (16 * sh.rt * 8) >> sh.kwl;
            const int64_t tiles = (st->rows + rows - 1) / rows;
            Int4Task& t = g.t[g.ntasks];
            t.x = static_cast<const uint16_t*>(items[i].x);
            t.y = static_cast<uint16_t*>(items[i].y);
            t.w = int4_view(st);
            t.N = st->rows;
            t.K = st->cols;
            t.x_aligned = st->cols % 8 == 0 && reinterpret_cast<uintptr_t>(items[i].x) % 16 == 0;
            t.kwl = sh.kwl;
            g.chunks[g.ntasks] = (int32_t)((st->cols + kChunk - 1) / kChunk * (8 >> sh.kwl));
            total += tiles;
            kmax = std::max(kmax, st->cols);
            g.cost0[g.ntasks + 1] = g.cost0[g.ntasks] + tiles * g.chunks[g.ntasks];
            ++g.ntasks;
        }
        const hipError_t e = f16 ? launch_ng<kInt4F16>(g, total, ng, resident, kmax, s)
                                 : launch_ng<kInt4Bf16>(g, total, ng, resident, kmax, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qk
