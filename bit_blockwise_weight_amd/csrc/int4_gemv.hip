// Decode product with an int4 weight of group scales and zero points, for gfx950:
//     y[m, n] = sum_k x[m, k] s[n, k / g] (q[n, k] - z[n, k / g]),   m < M <= 16
// for one weight or for up to 16 of a grouped call in one launch.
//
// The host deals the workgroups (8 waves each, two per CU) to the weights of a launch so that the longest
// is as short as can be; a workgroup owns a run of rows of one weight and walks it with RowTiles (w4_tile.h), the
// codes of the next rows being loaded while some are multiplied.
//
// Bound by the bytes of the codes, at 6 TB/s, where few rows of activations meet large weights: the seven weights of a
// layer (4096 wide, 11008 inside, groups of 128, 106 MB) at M = 1 23.9 us, 4.4 TB/s; 28672 x 8192, M = 4, 27.6 us.  In
// groups of 32 at M = 16 the layer takes 53 us, more than half of it instructions: decoding, scales, and every
// workgroup's turning of x into fp16.  1024 x 1024 at M = 1: a kernel of 4.2 us, a launch and two rounds of loads.
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
    int32_t x_aligned;       // rows of x start at 4-byte boundaries and K % 8 == 0
    int32_t kwl;             // log2 of the waves that split a row
    int32_t share, more;     // items per workgroup; the first `more` workgroups take one more
};

// A launch of one weight has arguments of its own: finding a task in the longer list costs two
// dependent reads of the arguments, about a microsecond.
template <int kTasks>
struct Int4Group {
    int32_t wg0[kTasks];     // first workgroup of each task (past the last one: never reached)
    int32_t M;
    int32_t pad;
    Int4Task t[kTasks];
};

template <int F, int NG, int RT, int MI, bool kResident, int kTasks>
__global__ __launch_bounds__(kThreads, 4) void int4_gemv_kernel(Int4Group<kTasks> g) {
    extern __shared__ __align__(16) uint8_t lds[];
    typedef RowTiles<F, NG, RT, MI, kResident, false> Tiles;
    int ti = 0;
#pragma unroll
    for (int i = 1; i < kTasks; ++i) ti += (int)blockIdx.x >= g.wg0[i];
    const Int4Task& t = g.t[ti];
    // this workgroup's rows
    const int b = (int)blockIdx.x - g.wg0[ti];
    Rows<RT> p;
    p.kwl = t.kwl;
    p.group_step = 16 * RT;
    p.step = (16 * RT * 8) >> t.kwl;
    const int64_t row0 = (int64_t)p.step * ((int64_t)b * t.share + (b < t.more ? b : t.more));
    const int items = t.share + (b < t.more);
    const int64_t row1 = row0 + (int64_t)p.step * items;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        p.base[r] = row0;
        p.off[r] = 16 * r;
    }
    p.count = (int32_t)((row1 < t.N ? row1 : t.N) - row0);
    p.x = t.x;
    p.xrow = nullptr;
    p.K = (int32_t)t.K;
    p.x_pitch = (int32_t)t.K;
    p.x_rows = g.M;
    p.x_aligned = t.x_aligned;
    p.M = g.M;
    Tiles::run(t.w, p, 0, items, lds, [&](int item, int q, const float* put) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int o = 64 * i + (threadIdx.x & 63), m = Tiles::act_of(o);
                const int j = item * p.step + q * (16 * RT) + 16 * r + (o & 15);
                const float v = Tiles::sum(put, t.kwl, q, r, o);
                if (m < g.M && j < p.count) t.y[m * t.N + row0 + j] = float_to_bits16(v, F == kInt4F16);
            }
    });
}

// Registers of a product that carry activations: the least that hold M rows (weights from memory: the layer at M = 8 38 us,
// in the form of sixteen 46).
constexpr int mi_for(int M) { return M <= 4 ? 1 : M <= 8 ? 2 : 4; }

size_t lds_bytes(int M, bool f16, int ng, int rt, int64_t K, bool resident) {
    const int mi = mi_for(M), kw = 1 << w4_most_kwl(kInt4Bf16, mi);
    return w4_fixed_bytes(kInt4Bf16, ng, rt, mi, resident) +
           w4_x_bytes(f16 ? kInt4F16 : kInt4Bf16, kw, M, mi, false, K, resident);
}
// The activations of a whole row stay in LDS where they fit; above four rows where they leave room for a second
// workgroup on the CU (weights from memory, 28672 x 8192 at M = 8: 38.2 us streaming with two, 38.9 resident with one; at
// M = 3 and 4, resident at any size is faster, 29.2 us against 30.8 for the layer at M = 3).
bool resident_for(int M, bool f16, int ng, int rt, int64_t K) {
    return lds_bytes(M, f16, ng, rt, K, true) <= (M > 4 ? kLdsBytes / 2 : kLdsBytes);
}

constexpr int32_t kNever = 0x7FFFFFFF;

template <int F, int NG, int RT, int MI, bool kResident, int kTasks>
hipError_t launch_tasks(const Int4Group<kTasks>& g, int64_t grid, size_t lds, hipStream_t s) {
    constexpr auto kernel = &int4_gemv_kernel<F, NG, RT, MI, kResident, kTasks>;
    const hipError_t e = allow_lds<kernel>(lds);
    if (e != hipSuccess) return e;
    kernel<<<dim3((unsigned)grid), dim3(kThreads), lds, s>>>(g);
    return hipGetLastError();
}

// How a launch is made.
struct Launch {
    int64_t grid;
    size_t lds;
    int ng, rt;
    bool resident;
};

template <int F, int NG, int RT, int MI, bool kResident>
hipError_t launch_one(Int4Group<kMaxGemvTasks>& g, const Launch& l, hipStream_t s) {
    if (g.wg0[1] == kNever) {
        Int4Group<1> one;
        one.wg0[0] = 0;
        one.M = g.M;
        one.pad = 0;
        one.t[0] = g.t[0];
        return launch_tasks<F, NG, RT, MI, kResident, 1>(one, l.grid, l.lds, s);
    }
    return launch_tasks<F, NG, RT, MI, kResident, kMaxGemvTasks>(g, l.grid, l.lds, s);
}

template <int F, int NG, int RT, int MI>
hipError_t launch_shape(Int4Group<kMaxGemvTasks>& g, const Launch& l, hipStream_t s) {
    return l.resident ? launch_one<F, NG, RT, MI, true>(g, l, s) : launch_one<F, NG, RT, MI, false>(g, l, s);
}

template <int F, int NG>
hipError_t launch_mi(Int4Group<kMaxGemvTasks>& g, const Launch& l, hipStream_t s) {
    if (mi_for(g.M) == 4) return launch_shape<F, NG, 1, 4>(g, l, s);
    if (mi_for(g.M) == 2) return launch_shape<F, NG, 1, 2>(g, l, s);
    return l.rt == 1 ? launch_shape<F, NG, 1, 1>(g, l, s) : launch_shape<F, NG, 2, 1>(g, l, s);
}

template <int F>
hipError_t launch_ng(Int4Group<kMaxGemvTasks>& g, const Launch& l, hipStream_t s) {
    if (l.ng == 4) return launch_mi<F, 4>(g, l, s);
    if (l.ng == 2) return launch_mi<F, 2>(g, l, s);
    return launch_mi<F, 1>(g, l, s);
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
    const int most_kwl = w4_most_kwl(kInt4Bf16, mi_for(M));
    // One launch per run of up to kMaxGemvTasks weights of one scale granularity, in task order.
    bool done[256] = {false};
    for (int32_t first = 0; first < count; ++first) {
        if (done[first]) continue;
        Launch l;
        l.ng = int4_groups_per_chunk(items[first].st->group);
        Int4Group<kMaxGemvTasks> g;
        int32_t n = 0;
        int64_t items_of[kMaxGemvTasks], windows[kMaxGemvTasks], kmax = 0, pairs = 0;
        for (int32_t i = first; i < count && n < kMaxGemvTasks; ++i) {
            const qk_int4_state* st = items[i].st;
            if (done[i] || int4_groups_per_chunk(st->group) != l.ng) continue;
            done[i] = true;
            Int4Task& t = g.t[n];
            t.x = static_cast<const uint16_t*>(items[i].x);
            t.y = static_cast<uint16_t*>(items[i].y);
            t.w = int4_view(st);
            t.N = st->rows;
            t.K = st->cols;
            t.x_aligned = st->cols % 8 == 0 && reinterpret_cast<uintptr_t>(items[i].x) % 4 == 0;
            // how many waves split a row decides the order of its sum: by the weight alone, not by its launch
            t.kwl = w4_kwl(kInt4Bf16, st->cols, st->rows, 16, most_kwl);
            while (t.kwl < most_kwl && (256 >> t.kwl) * st->code_stride > 1 << 30) ++t.kwl;
            const int64_t window = (int64_t)kLineK << t.kwl;
            windows[n] = (st->cols + window - 1) / window;
            pairs += (st->rows + (256 >> t.kwl) - 1) / (256 >> t.kwl);
            kmax = std::max(kmax, st->cols);
            ++n;
        }
        const int per_cu_most = 2;
        // Tiles of 16 rows per item and row group: two, which bring more codes on their way at a time, where every
        // workgroup has an item of two (weights from memory, M = 1: the layer 26.4 us, with one 28.8), one where not
        // (4096 x 4096 5.4 us, with two 6.2) and above four rows, whose sums and scales leave no room for two workgroups on
        // a CU (M = 16, groups of 32: the layer 56 us, with two 61; M = 8, groups of 128, 38 and 43).
        l.rt = mi_for(M) == 1 && pairs > (int64_t)per_cu_most * device_cu_count() ? 2 : 1;
        // (an output's bits do not depend on whether the activations stay)
        l.resident = resident_for(M, f16, l.ng, l.rt, kmax);
        l.lds = lds_bytes(M, f16, l.ng, l.rt, kmax, l.resident);
        const int per_cu = l.lds > kLdsBytes / 2 ? 1 : per_cu_most;
        for (int32_t i = 0; i < n; ++i) {
            const int64_t step = (128 * l.rt) >> g.t[i].kwl;
            items_of[i] = (g.t[i].N + step - 1) / step;
        }
        // The workgroups that the CUs hold at a time are dealt so that the longest one is as short as can be: with at
        // most `most` windows each, a task needs ceil(items / floor(most / windows of an item)) of them.
        const int64_t slots = (int64_t)per_cu * device_cu_count();
        auto wgs_for = [&](int32_t i, int64_t most) {
            const int64_t per = most / windows[i];
            return (items_of[i] + per - 1) / per;
        };
        int64_t lo = 1, hi = 1;
        for (int32_t i = 0; i < n; ++i) {
            lo = std::max(lo, windows[i]);
            hi = std::max(hi, windows[i] * items_of[i]);
        }
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            int64_t need = 0;
            for (int32_t i = 0; i < n; ++i) need += wgs_for(i, mid);
            if (need <= slots) hi = mid;
            else lo = mid + 1;
        }
        l.grid = 0;
        for (int32_t i = 0; i < n; ++i) {
            Int4Task& t = g.t[i];
            int64_t wgs = wgs_for(i, lo);
            // A workgroup's rows stay under 2^29 bytes of codes and one item more, of 2^30 bytes at most: offsets of
            // 32 bits reach them (and the scales: at most two bytes for 16 of codes).
            const int64_t bytes = ((128 * l.rt) >> t.kwl) * t.w.stride;
            wgs = std::max(wgs, std::min(items_of[i], (int64_t)((double)items_of[i] * (double)bytes / (1 << 29)) + 1));
            t.share = (int32_t)(items_of[i] / wgs);
            t.more = (int32_t)(items_of[i] % wgs);
            g.wg0[i] = (int32_t)l.grid;
            l.grid += wgs;
        }
        for (int32_t i = n; i < kMaxGemvTasks; ++i) g.wg0[i] = kNever;
        g.M = M;
        g.pad = 0;
        const hipError_t e = f16 ? launch_ng<kInt4F16>(g, l, s) : launch_ng<kInt4Bf16>(g, l, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qk
