// Device code shared by the kernels that multiply a few activation rows with 4-bit
// weights straight from memory (int4 with group scales; NF4 and other 16-level tables
// in the mixture-of-experts layer), for gfx950.
//
// One step of a wave is a "chunk": 16 weight rows x 128 k.  Lane l holds row n = l % 16
// and, with h = l / 16, the 16 bytes of k = 128 c + 32 h + [0, 32): one 16-byte load, 64
// contiguous bytes of a row per instruction.  The four dwords of a lane are transposed
// over the four lane groups in registers (four lane swaps), after which dword j holds
// k = 128 c + 32 j + 8 h + [0, 8): MFMA j (16x16x32) then covers the 32 consecutive k of
// [128 c + 32 j, +32), so a scale group of 32 or more never splits an MFMA.
//
//   A = activations (row m = l % 16, k = 8 (l / 16) + i), B = W^T (column n = l % 16, the
//   same k), D: column n = l % 16, rows m = 4 (l / 16) + r.  A scale of row n is then one
//   value per lane, applied to the fp32 partial product of its group.
//
// int4 decoding, two weights an instruction pair: (dword >> 4 i) & 0x000F000F leaves two
// codes in the low bits of the two halves; OR-ing an exponent whose last mantissa bits they
// become gives 128 + q in bf16 (0x4300) or 1024 + q in fp16 (0x6400), both exact.  The halves
// hold elements (1, 5), (0, 4), (3, 7), (2, 6) of the dword's eight (the first of a pair
// sits in the high nibble), so the activations are stored in that order too.  The product
// with W is then
//     sum x (q - z) = sum x (128 + q) - (128 + z) sum x,
// where sum x comes from one more MFMA against a matrix of ones, in the layout of D.  fp16
// subtracts 1032 from each pair first (exact: q - 8), which leaves (z - 8) sum x.  In bf16
// the subtraction happens in fp32 after the sums: its rounding error is 2^-24 of terms up to
// 143 |x|, about 2^-19 of the group's result, far under the 2^-9 of the rounded output.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qk_device.h"
#include "qk_internal.h"

namespace qk {
namespace w4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Weight forms of the kernels: int4 times bf16 or fp16 activations, 16 levels times bf16.
enum Form { kInt4Bf16 = 0, kInt4F16 = 1, kLevels = 2 };

constexpr int kChunk = 128;               // k per step of a wave

__device__ __forceinline__ float f16_bits_to_float(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
__device__ __forceinline__ float bf16_bits_to_float(uint16_t b) { return as_float((uint32_t)b << 16); }

__device__ __forceinline__ uint16_t float_to_bits16(float v, bool f16) {
    if (f16) return __builtin_bit_cast(uint16_t, (_Float16)v);
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// d[j] of lane group h  ->  d[h] of lane group j (see the top of the file)
__device__ __forceinline__ void transpose_groups(u32x4_t& d) {
    auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d[0] = lo[0];
    d[1] = lo[1];
    d[2] = hi[0];
    d[3] = hi[1];
}

// Eight codes of a dword as an MFMA fragment (int4 forms).
template <int F>
__device__ __forceinline__ u32x4_t decode8(uint32_t w) {
    static_assert(F == kInt4Bf16 || F == kInt4F16, "levels are decoded through their table");
    constexpr uint32_t kMagic = F == kInt4Bf16 ? 0x43004300u : 0x64006400u;
    u32x4_t f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | kMagic;
        if constexpr (F == kInt4F16)
            v = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, v) - (f16x2_t){1032, 1032});
        f[i] = v;
    }
    return f;
}

// Activations of eight consecutive k in the order decode8 gives the weights.
__device__ __forceinline__ u32x4_t int4_order(u32x4_t v) {
    u32x4_t r;
    r[0] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302);   // (1, 5)
    r[1] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100);   // (0, 4)
    r[2] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302);   // (3, 7)
    r[3] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100);   // (2, 6)
    return r;
}
// Position inside its eight that element k of a row takes in that order.
__device__ __forceinline__ int int4_slot(int k) {
    const int e = k & 7;                                    // 1 5 0 4 3 7 2 6
    return 4 * ((e >> 1) & 1) + 2 * (1 - (e & 1)) + (e >> 2);
}

template <int F>
__device__ __forceinline__ floatx4_t mfma(u32x4_t a, u32x4_t b, floatx4_t c) {
    if constexpr (F == kInt4F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// A fragment of ones, and what the stored codes exceed q by.
template <int F>
__device__ __forceinline__ u32x4_t ones() {
    constexpr uint32_t k = F == kInt4F16 ? 0x3C003C00u : 0x3F803F80u;
    return (u32x4_t){k, k, k, k};
}
template <int F>
constexpr float kCodeBias = F == kInt4Bf16 ? 128.0f : -8.0f;


// One int4 weight as the kernels see it.
struct Int4View {
    const uint8_t* codes;     // [rows, stride], 16-byte aligned
    const uint16_t* scales;   // [rows, G], fp16 or bf16 bits
    const uint8_t* zeros;     // [rows, G], or NULL: every zero point is 8
    int64_t stride;           // bytes of a row of codes, a multiple of 16
    int32_t G;                // groups of a row
    int32_t gshift;           // log2 of the group size (>= 5); 30: one group
    int32_t scale_f16;        // 1: fp16 scales, 0: bf16
    int32_t pad;
};

// Codes of one chunk of a row: bytes past the row's end are never read (what is read in
// their place meets activations that are zero).
__device__ __forceinline__ u32x4_t load_codes(const uint8_t* row, int64_t stride, int c, int h) {
    int64_t off = (int64_t)c * (kChunk / 2) + 16 * h;
    off = off < stride - 16 ? off : stride - 16;
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(row + off));
}

// Scales and zero points of one row in one chunk: NG groups of 128 / NG k.  Groups past the
// row's end (they only meet zero activations) repeat the last one.
template <int NG>
struct GroupScales {
    uint16_t s[NG];
    uint8_t z[NG];
    __device__ __forceinline__ void load(const Int4View& w, int64_t row, int c) {
        const int64_t base = row * w.G;
        const int g0 = (c * kChunk) >> w.gshift;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int g = g0 + i < w.G ? g0 + i : w.G - 1;
            s[i] = w.scales[base + g];
            z[i] = w.zeros ? w.zeros[base + g] : (uint8_t)8;
        }
    }
    __device__ __forceinline__ float scale(const Int4View& w, int i) const {
        return w.scale_f16 ? f16_bits_to_float(s[i]) : bf16_bits_to_float(s[i]);
    }
};

// Eight consecutive activations of a row from k on, zero past the row's end (cols).
__device__ __forceinline__ u32x4_t load_x8(const uint16_t* row, int64_t k, int64_t cols, bool aligned16) {
    if (aligned16 && k + 8 <= cols) return *reinterpret_cast<const u32x4_t*>(row + k);
    u32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = k + 2 * i < cols ? row[k + 2 * i] : 0u;
        const uint32_t hi = k + 2 * i + 1 < cols ? row[k + 2 * i + 1] : 0u;
        v[i] = lo | (hi << 16);
    }
    return v;
}

// A 16-level weight (NF4 and the like) as the kernels see it: rows of K elements, K a multiple
// of 64, so that every run of 64 k of a row lies in one quantization block.
struct LevelsView {
    const uint8_t* codes;
    const float* absmax;      // plain
    const int8_t* q8;         // nested
    const float* dq_scale;
    const float* dq_mean;
    int64_t stride;           // K / 2
    int64_t last_block;       // number of blocks - 1
    int32_t bshift;           // log2(block size)
    int32_t nested;
    float levels[16];
};

// Block scales of one row in one chunk (two runs of 64 k; a run past the row's end meets zero
// activations, its index is only kept in range).
struct LevelScales {
    float a[2];
    int8_t q[2];
    __device__ __forceinline__ void load(const LevelsView& w, int64_t row, int c) {
        const int64_t e = row * (2 * w.stride) + (int64_t)c * kChunk;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int64_t b = (e + 64 * i) >> w.bshift;
            b = b < w.last_block ? b : w.last_block;
            if (w.nested) {
                q[i] = w.q8[b];
                a[i] = w.dq_scale[b / QK_DQ_BLOCK];
            } else {
                q[i] = 0;
                a[i] = w.absmax[b];
            }
        }
    }
    __device__ __forceinline__ float scale(const LevelsView& w, float mean, int i) const {
        return w.nested ? __fadd_rn(__fmul_rn((float)q[i], a[i]), mean) : a[i];
    }
};

// Table of the 256 code bytes as (bf16 level of the high nibble, bf16 level of the low nibble),
// 64 copies so that a lane reads its own bank: entry b of copy l at b * 256 + 4 l.
constexpr int kTabBytes = 256 * 64 * 4;

__device__ __forceinline__ void build_table(uint8_t* tab, const float* levels, int tid, int threads) {
    for (int i = tid; i < 256 * 16; i += threads) {
        const int b = i >> 4;
        const uint32_t v = pack_bf16x2(levels[b >> 4], levels[b & 15]);
        *reinterpret_cast<u32x4_t*>(tab + b * 256 + (i & 15) * 16) = (u32x4_t){v, v, v, v};
    }
}

__device__ __forceinline__ u32x4_t decode8_table(const uint8_t* tab, uint32_t w, uint32_t lane4) {
    u32x4_t f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t off = __builtin_amdgcn_perm(w, lane4, 0x0C0C0000u | ((4u + i) << 8));
        f[i] = *reinterpret_cast<const uint32_t*>(tab + off);
    }
    return f;
}

}  // namespace w4
}  // namespace qk
