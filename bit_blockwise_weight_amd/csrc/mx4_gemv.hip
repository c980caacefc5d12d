// Decode product of 16-bit activations with a microscaled 4-bit weight, for gfx950:
//     y[m, n] = sum_k x[m, k] value(code[n, k]) 2^(e[n, k / 32] - 127),   m < M <= 16
// A workgroup (8 waves, two per CU) owns a run of rows and walks it with RowTiles (w4_tile.h), the codes and scales of the
// next rows being loaded while some are multiplied.  Bound by the bytes of the codes and
// by decoding them: 28672 x 8192 fp16 at M = 4 29 us, 4.3 TB/s, VALU busy 36 %, bf16 26; 1024 x 1024 bf16 at M = 1 3.0 us, latency.
#include <algorithm>

#include "qk_device.h"
#include "qk_internal.h"
#include "w4_tile.h"

namespace qk {
namespace {

using namespace w4;

constexpr int kThreads = 512;

struct GemvArgs {
    const uint16_t* x;       // [M, K]
    uint16_t* y;             // [M, N]
    Mx4View w;
    int64_t N;
    int32_t K;
    int32_t M;
    int32_t x_aligned;       // rows of x start at 4-byte boundaries and K % 8 == 0
    int32_t kwl;             // log2 of the waves that split a row
    int32_t share, more;     // items per workgroup; the first `more` workgroups take one more
};

constexpr int groups_for(int f) { return f == kMx4F16 ? 4 : 1; }

// First row of workgroup b and the row behind its last one.
template <int RT>
__device__ __forceinline__ int step_of(const GemvArgs& a) { return (16 * RT * 8) >> a.kwl; }
template <int RT>
__device__ __forceinline__ void rows_of(const GemvArgs& a, int b, int64_t& row0, int64_t& row1) {
    row0 = (int64_t)step_of<RT>(a) * ((int64_t)b * a.share + (b < a.more ? b : a.more));
    row1 = row0 + (int64_t)step_of<RT>(a) * (a.share + (b < a.more));
    row1 = row1 < a.N ? row1 : a.N;
}

// Weights of the two largest scales may pass bf16, though their products with small activations are numbers: an infinity among
// them, or a NaN where it meets a 0, stays in the sum.  The outputs of row group q of an item for which that may be so, stored as no
// numbers and with such a scale in their row, are made again, each group's scale applied to its sum: one after the other, the
// lanes taking groups.  (Quantization gives no scale over 252.  Looking for them where scales land costs every call 1 to 3 %.  This
// code stands behind the kernel's end, and reads its arguments anew: between the loops, or with registers kept for it, it costs as much.)
template <int RT, int MI, class Tiles>
__device__ __forceinline__ void make_again(int item, int q) {
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    auto args = (const __attribute__((address_space(4))) GemvArgs*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(args));
    const GemvArgs& a = *(const GemvArgs*)args;
    const int lane = threadIdx.x & 63;
    int64_t row0, row1;
    rows_of<RT>(a, (int)blockIdx.x, row0, row1);
#pragma unroll 1
    for (int t = 0; t < RT * MI; ++t) {
        const int r = t / MI, o = 64 * (t % MI) + lane;
        const int64_t first = row0 + item * step_of<RT>(a) + q * (16 * RT) + 16 * r;
        // the rows with such a scale, lane l looking through a quarter of row l % 16's
        bool large = false;
        if (first + (lane & 15) < row1) {
            const uint32_t* scales = reinterpret_cast<const uint32_t*>(a.w.scales + (first + (lane & 15)) * a.w.scale_stride);
#pragma unroll 4
            for (int d = lane >> 4; 4 * d < a.w.G; d += 4) {        // (bytes behind the last scale may be anything, and 255 is)
                const uint32_t v = scales[d];
                large |= (((v & 0x7F7F7F7Fu) + 0x03030303u) & v & 0x80808080u) != 0;
            }
        }
        uint64_t rows = __ballot(large);
        rows |= rows >> 32 | rows << 32;
        rows |= rows >> 16 | rows << 48;
        const bool mine = Tiles::act_of(o) < a.M && first + (lane & 15) < row1;
        const uint16_t y = mine ? a.y[Tiles::act_of(o) * a.N + first + (lane & 15)] : 0;
        uint64_t bad = rows & __ballot((y & 0x7F80) == 0x7F80);
        for (; bad; bad &= bad - 1) {
            const int l = (int)__builtin_ctzll(bad), m = Tiles::act_of(o - lane + l);
            const int64_t row = first + (l & 15);
            const uint8_t* scales = a.w.scales + row * a.w.scale_stride;
            float sum = 0.0f;
            for (int g = lane; g < a.w.G; g += 64) {
                // a group of 32: its codes, padded, and its activations, or what there are of them
                const uint8_t* codes = a.w.codes + row * a.w.stride + 16 * g;
                const uint16_t* x = a.x + (int64_t)m * a.K + 32 * g;
                uint32_t c[4];
                __builtin_memcpy(c, codes, 16);
                float part = 0.0f;
#pragma unroll 1
                for (int d = 0; d < 4; ++d) {
                    uint16_t v[8];
                    if (32 * g + 8 * d + 8 <= a.K) {
                        __builtin_memcpy(v, x + 8 * d, 16);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = 32 * g + 8 * d + i < a.K ? x[8 * d + i] : 0;
                    }
                    const uint32_t w = d == 0 ? c[0] : d == 1 ? c[1] : d == 2 ? c[2] : c[3];
                    f32x2_t f[4];
                    f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
                    f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
                    f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
                    f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
#pragma unroll
                    for (int i = 0; i < 8; ++i) part = fmaf(bf16_bits_to_float(v[i]), f[i / 2][i % 2], part);
                }
                const uint32_t e = scales[g];
                sum = fmaf(part, as_float(e == 0 ? 0x00400000u : e == 255u ? 0x7FC00000u : e << 23), sum);
            }
#pragma unroll 1
            for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
            if (lane == 0) a.y[m * a.N + row] = float_to_bits16(sum, false);
        }
    }
}

template <int F, int RT, int MI, bool kResident>
__global__ __launch_bounds__(kThreads, 4) void mx4_gemv_kernel(GemvArgs a) {
    extern __shared__ __align__(16) uint8_t lds[];
    typedef RowTiles<F, groups_for(F), RT, MI, kResident, false> Tiles;
    Rows<RT> p;
    p.kwl = a.kwl;
    p.group_step = 16 * RT;
    p.step = step_of<RT>(a);
    int64_t row0, row1;
    rows_of<RT>(a, (int)blockIdx.x, row0, row1);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        p.base[r] = row0;
        p.off[r] = 16 * r;
    }
    p.count = (int32_t)(row1 - row0);
    p.x = a.x;
    p.xrow = nullptr;
    p.K = a.K;
    p.x_pitch = a.K;
    p.x_rows = a.M;
    p.x_aligned = a.x_aligned;
    p.M = a.M;
    const int items = a.share + ((int)blockIdx.x < a.more);
    uint64_t again = 0;                                             // the items (modulo 64) of this wave with outputs that are no numbers
    Tiles::run(a.w, p, 0, items, lds, [&](int item, int q, const float* put) {
        bool all = true;                                            // numbers
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int o = 64 * i + (threadIdx.x & 63), m = Tiles::act_of(o);
                const int j = item * p.step + q * (16 * RT) + 16 * r + (o & 15);
                const float v = Tiles::sum(put, a.kwl, q, r, o);
                all &= fabsf(v) < INFINITY;
                if (m < a.M && j < p.count) a.y[m * a.N + row0 + j] = float_to_bits16(v, F == kMx4F16);
            }
        if (F == kMx4Bf16 && __ballot(!all)) again |= 1ull << (item & 63);
    });
    if constexpr (F == kMx4Bf16) {
        if (__builtin_expect(again != 0, 0)) {
            const int q = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) >> p.kwl;   // the row group that this wave sums
#pragma unroll 1
            for (int item = 0; item < items; ++item)
                if (again >> (item & 63) & 1) make_again<RT, MI, Tiles>(item, q);
        }
    }
}

// Registers of a product that carry activations: the least that hold M rows.
constexpr int mi_for(int M) { return M <= 4 ? 1 : M <= 8 ? 2 : 4; }

size_t lds_bytes(Form f, int M, int rt, int64_t K, bool resident) {
    const int mi = mi_for(M), kw = 1 << w4_most_kwl(f, mi);
    return w4_fixed_bytes(f, groups_for(f), rt, mi, resident) + w4_x_bytes(f, kw, M, mi, false, K, resident);
}

template <int F, int RT, int MI, bool kResident>
hipError_t launch(const GemvArgs& a, int64_t grid, size_t lds, hipStream_t s) {
    constexpr auto kernel = &mx4_gemv_kernel<F, RT, MI, kResident>;
    const hipError_t e = allow_lds<kernel>(lds);
    if (e != hipSuccess) return e;
    kernel<<<dim3((unsigned)grid), dim3(kThreads), lds, s>>>(a);
    return hipGetLastError();
}

template <int F, int RT, int MI>
hipError_t launch(const GemvArgs& a, int64_t grid, size_t lds, bool resident, hipStream_t s) {
    return resident ? launch<F, RT, MI, true>(a, grid, lds, s) : launch<F, RT, MI, false>(a, grid, lds, s);
}

template <int F>
hipError_t launch_form(GemvArgs& a, hipStream_t s) {
    const int mi = mi_for(a.M), most_kwl = w4_most_kwl((Form)F, mi);
    // offsets of 32 bits: the bytes of a row's codes or scales, whichever are more
    const int64_t pitch = std::max<int64_t>(a.w.stride, a.w.scale_stride);
    a.kwl = w4_kwl((Form)F, a.K, a.N, 16, most_kwl);
    while (a.kwl < most_kwl && (256 >> a.kwl) * pitch > 1 << 30) ++a.kwl;
    const int64_t pairs = (a.N + (256 >> a.kwl) - 1) / (256 >> a.kwl);
    // Two tiles of 16 rows per item, which bring more codes on their way at a time, where every workgroup has an item of
    // two, and one where not and above four rows, as for int4.
    const int rt = mi == 1 && pairs > 2 * (int64_t)device_cu_count() ? 2 : 1;
    // the activations of a whole row stay in LDS where they fit, above four rows where they leave room for a second
    // workgroup (an output's bits do not depend on it)
    const bool resident = lds_bytes((Form)F, a.M, rt, a.K, true) <= (a.M > 4 ? kLdsBytes / 2 : kLdsBytes);
    const size_t lds = lds_bytes((Form)F, a.M, rt, a.K, resident);
    const int64_t slots = (lds > kLdsBytes / 2 ? 1 : 2) * (int64_t)device_cu_count();
    const int64_t step = (128 * rt) >> a.kwl, items = (a.N + step - 1) / step;
    const int64_t per = (items + slots - 1) / slots;
    int64_t wgs = (items + per - 1) / per;
    // a workgroup's rows stay under 2^29 bytes and one item more, of 2^30 at most
    wgs = std::max(wgs, std::min(items, (int64_t)((double)items * (double)(step * pitch) / (1 << 29)) + 1));
    a.share = (int32_t)(items / wgs);
    a.more = (int32_t)(items % wgs);
    if (mi == 4) return launch<F, 1, 4>(a, wgs, lds, resident, s);
    if (mi == 2) return launch<F, 1, 2>(a, wgs, lds, resident, s);
    return rt == 1 ? launch<F, 1, 1>(a, wgs, lds, resident, s) : launch<F, 2, 1>(a, wgs, lds, resident, s);
}

}  // namespace

hipError_t launch_mx4_gemv(const void* x, int32_t M, const qk_mx4_state* w, void* y, bool f16, hipStream_t s) {
    GemvArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.y = static_cast<uint16_t*>(y);
    a.w.codes = w->codes;
    a.w.scales = w->scales;
    a.w.stride = w->code_stride;
    a.w.scale_stride = (int32_t)w->scale_stride;
    a.w.G = (int32_t)((w->cols + 31) / 32);
    a.N = w->rows;
    a.K = (int32_t)w->cols;
    a.M = M;
    a.x_aligned = w->cols % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 4 == 0;
    return f16 ? launch_form<kMx4F16>(a, s) : launch_form<kMx4Bf16>(a, s);
}

}  // namespace qk
