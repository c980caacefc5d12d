// Quantization of rows to microscaled 4-bit groups and back, for gfx950.
//
// Per group of 32 consecutive inputs of a row, with top = max |x|:
//     e    = max(floor(log2 top) - 2 + 127, 0)       the exponent bits of top, less 2
//     code = e2m1 value nearest to x / 2^(e - 127), ties to the even code, at most 6
// Everything is exact: the maximum on the bits of |x| as integers, the exponent taken from them, the division (by a
// power of two) and the rounding in v_cvt_scalef32_pk_fp4_*.  An infinity or a NaN makes e = 255 and every code 0.
//
// A lane takes 8 inputs, 4 lanes a group: the maximum crosses two DPP steps, the codes leave as a dword a lane
// (256 contiguous bytes a wave), the scales of four groups as a dword from every 16th lane.  16 lanes take a run of 128
// inputs of one row, so short rows leave no more than that idle.  Bound by memory: 2 bytes in, 0.53 out (28672 x 8192
// bf16 126 us, 4.7 TB/s, and back 86 us, 6.9 TB/s of codes partly cached; one row of 4096 1.7 us, a launch).
#include "mx4.h"

namespace qk {
namespace {

using namespace mx4;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kRun = 128;                  // inputs that 16 lanes take
constexpr int kRuns = 2;                   // runs per 16 lanes, loaded together

struct QuantArgs {
    const void* x;
    uint8_t* codes;
    uint8_t* scales;
    int64_t pitch;             // of x, in elements
    int64_t code_stride, scale_stride;
    int32_t cols;
    int32_t groups;
    uint32_t per_row;          // runs of a row
    uint32_t total;            // runs of this launch
};

// 8 inputs as loaded: 16-bit pairs, or fp32.
template <int DT>
struct Raw {
    u32x4_t v[DT == QK_F32 ? 2 : 1];
};

// Inputs k..k+7 of a row that starts at element `row`, zero from cols on.  The hardware takes any alignment.
template <int DT>
__device__ __forceinline__ void load(Raw<DT>& r, const void* x, int64_t row, int32_t k, int32_t cols) {
    if constexpr (DT == QK_F32) {
        const float* p = static_cast<const float*>(x) + row + k;
        if (k + 8 <= cols) {
            __builtin_memcpy(&r, p, 32);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r.v[i >> 2][i & 3] = k + i < cols ? as_uint(p[i]) : 0u;
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(x) + row + k;
        if (k + 8 <= cols) {
            __builtin_memcpy(&r, p, 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r.v[0][i] = (k + 2 * i < cols ? (uint32_t)p[2 * i] : 0u) |
                            (k + 2 * i + 1 < cols ? (uint32_t)p[2 * i + 1] << 16 : 0u);
        }
    }
}

// The bits of the largest |x| of the eight as fp32.
template <int DT>
__device__ __forceinline__ uint32_t top_bits(const Raw<DT>& r) {
    if constexpr (DT == QK_F32) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, r.v[i >> 2][i & 3] & 0x7FFFFFFFu);
        return top;
    } else {
        u16x2_t m = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, r.v[0][i] & 0x7FFF7FFFu));
        const uint16_t top = max(m[0], m[1]);
        if constexpr (DT == QK_BF16) return (uint32_t)top << 16;
        return as_uint((float)__builtin_bit_cast(_Float16, top));
    }
}

// (the pairs go through plain locals: a bit cast of a vector element lvalue reads the vector's first element)
template <int DT>
__device__ __forceinline__ uint32_t encode(const Raw<DT>& r, float scale) {
    const uint32_t d0 = r.v[0][0], d1 = r.v[0][1], d2 = r.v[0][2], d3 = r.v[0][3];
    uint32_t c = 0;
    if constexpr (DT == QK_F32) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_float(d0), as_float(d1), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_float(d2), as_float(d3), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_float(r.v[1][0]), as_float(r.v[1][1]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_float(r.v[1][2]), as_float(r.v[1][3]), scale, 3);
    } else if constexpr (DT == QK_BF16) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, d0), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, d1), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, d2), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, d3), scale, 3);
    } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, d0), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, d1), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, d2), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, d3), scale, 3);
    }
    return c;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(QuantArgs a) {
    const int lane16 = threadIdx.x & 15;
    const uint32_t first = (blockIdx.x * (uint32_t)(kThreads / 16) + threadIdx.x / 16) * kRuns;
    Raw<DT> r[kRuns];
    uint32_t row[kRuns];
    int32_t k[kRuns];
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
        const uint32_t run = first + i;
        row[i] = run / a.per_row;
        k[i] = (int32_t)(run - row[i] * a.per_row) * kRun + 8 * lane16;
        if (run >= a.total) k[i] = a.cols;
        if (run < a.total && k[i] < a.cols) load<DT>(r[i], a.x, (int64_t)row[i] * a.pitch, k[i], a.cols);
        else r[i] = Raw<DT>{};
    }
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
        const uint32_t top = group_max_u32<4>(top_bits<DT>(r[i])) >> 23;
        const uint32_t e = top == 255 ? kScaleNan : max(top, 2u) - 2u;
        const uint32_t c = top == 255 ? 0u : encode<DT>(r[i], scale_bits(e));
        const int32_t g = k[i] / kGroup;               // the lane's group: four lanes share one
        if (first + i < a.total && g < a.groups)
            *reinterpret_cast<uint32_t*>(a.codes + (int64_t)row[i] * a.code_stride + k[i] / 2) = c;
        // the bytes of four groups in the first lane of 16 (those behind the last group are zero)
        uint32_t s = g < a.groups ? e << (8 * (g & 3)) : 0u;
        s |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x141, 0xF, 0xF, true);   // lane i with 7 - i
        s |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x140, 0xF, 0xF, true);   // lane i with 15 - i
        if (lane16 == 0 && first + i < a.total && g < a.groups)
            *reinterpret_cast<uint32_t*>(a.scales + (int64_t)row[i] * a.scale_stride + g) = s;
    }
}

struct DequantArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    void* out;
    int64_t code_stride, scale_stride;
    int32_t cols;
    uint32_t per_row;
    uint32_t total;
};

typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Eight values of a dword of codes.
template <int DT>
__device__ __forceinline__ Raw<DT> decode(uint32_t c, float scale) {
    Raw<DT> r;
    f32x2_t f[4];
    f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
    f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
    f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2);
    f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == QK_F32) {
            r.v[i >> 1][2 * (i & 1)] = as_uint(f[i][0]);
            r.v[i >> 1][2 * (i & 1) + 1] = as_uint(f[i][1]);
        } else if constexpr (DT == QK_BF16) {
            r.v[0][i] = pack_bf16x2(f[i][0], f[i][1]);
        } else {
            r.v[0][i] = __builtin_bit_cast(uint32_t, (f16x2_t){(_Float16)f[i][0], (_Float16)f[i][1]});
        }
    }
    return r;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(DequantArgs a) {
    const int lane16 = threadIdx.x & 15;
    const uint32_t first = (blockIdx.x * (uint32_t)(kThreads / 16) + threadIdx.x / 16) * kRuns;
    uint32_t c[kRuns], e[kRuns], row[kRuns];
    int32_t k[kRuns];
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
        const uint32_t run = first + i;
        row[i] = run / a.per_row;
        k[i] = (int32_t)(run - row[i] * a.per_row) * kRun + 8 * lane16;
        if (run >= a.total) k[i] = a.cols;
        c[i] = e[i] = 0;
        if (k[i] < a.cols) {
            c[i] = *reinterpret_cast<const uint32_t*>(a.codes + (int64_t)row[i] * a.code_stride + k[i] / 2);
            e[i] = a.scales[(int64_t)row[i] * a.scale_stride + k[i] / kGroup];
        }
    }
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
        if (k[i] >= a.cols) continue;
        const Raw<DT> r = decode<DT>(c[i], scale_bits(e[i]));
        const int64_t at = (int64_t)row[i] * a.cols + k[i];
        if constexpr (DT == QK_F32) {
            float* p = static_cast<float*>(a.out) + at;
            if (k[i] + 8 <= a.cols) {
                __builtin_memcpy(p, &r, 32);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k[i] + j < a.cols) p[j] = as_float(r.v[j >> 2][j & 3]);
            }
        } else {
            uint16_t* p = static_cast<uint16_t*>(a.out) + at;
            if (k[i] + 8 <= a.cols) {
                __builtin_memcpy(p, &r, 16);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k[i] + j < a.cols) p[j] = (uint16_t)(r.v[0][j >> 1] >> (16 * (j & 1)));
            }
        }
    }
}

// Launches over rows in pieces of at most 2^28 runs (a launch has fewer than 2^32 threads): launch(first row, rows).
template <class Launch>
hipError_t by_rows(int64_t rows, int64_t per_row, Launch&& launch) {
    const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 28) / per_row);
    for (int64_t r = 0; r < rows; r += most) {
        launch(r, std::min(most, rows - r));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

unsigned grid_for(uint32_t total) { return (total + kThreads / 16 * kRuns - 1) / (kThreads / 16 * kRuns); }

}  // namespace

hipError_t launch_mx4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t pitch, uint8_t* codes,
                               int64_t code_stride, uint8_t* scales, int64_t scale_stride, hipStream_t s) {
    QuantArgs a;
    a.pitch = pitch;
    a.code_stride = code_stride;
    a.scale_stride = scale_stride;
    a.cols = (int32_t)cols;
    a.groups = (int32_t)((cols + kGroup - 1) / kGroup);
    a.per_row = (uint32_t)((cols + kRun - 1) / kRun);
    return by_rows(rows, a.per_row, [&](int64_t r, int64_t n) {
        a.x = static_cast<const uint8_t*>(x) + r * pitch * (x_dtype == QK_F32 ? 4 : 2);
        a.codes = codes + r * code_stride;
        a.scales = scales + r * scale_stride;
        a.total = (uint32_t)(n * a.per_row);
        const dim3 grid(grid_for(a.total));
        if (x_dtype == QK_F32) mx4_quantize_kernel<QK_F32><<<grid, kThreads, 0, s>>>(a);
        else if (x_dtype == QK_BF16) mx4_quantize_kernel<QK_BF16><<<grid, kThreads, 0, s>>>(a);
        else mx4_quantize_kernel<QK_F16><<<grid, kThreads, 0, s>>>(a);
    });
}

hipError_t launch_mx4_dequantize(const qk_mx4_state* st, void* out, int32_t out_dtype, hipStream_t s) {
    DequantArgs a;
    a.code_stride = st->code_stride;
    a.scale_stride = st->scale_stride;
    a.cols = (int32_t)st->cols;
    a.per_row = (uint32_t)((st->cols + kRun - 1) / kRun);
    return by_rows(st->rows, a.per_row, [&](int64_t r, int64_t n) {
        a.codes = st->codes + r * st->code_stride;
        a.scales = st->scales + r * st->scale_stride;
        a.out = static_cast<uint8_t*>(out) + r * st->cols * (out_dtype == QK_F32 ? 4 : 2);
        a.total = (uint32_t)(n * a.per_row);
        const dim3 grid(grid_for(a.total));
        if (out_dtype == QK_F32) mx4_dequantize_kernel<QK_F32><<<grid, kThreads, 0, s>>>(a);
        else if (out_dtype == QK_BF16) mx4_dequantize_kernel<QK_BF16><<<grid, kThreads, 0, s>>>(a);
        else mx4_dequantize_kernel<QK_F16><<<grid, kThreads, 0, s>>>(a);
    });
}

}  // namespace qk
