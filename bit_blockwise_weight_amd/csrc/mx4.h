// Microscaled 4-bit matrices on gfx950: what the kernels that read or write them share.
//
// A row is cut into groups of 32 inputs.  A group holds 32 e2m1 codes (sign, two bits of exponent, one of mantissa:
// 0, 1/2, 1, 3/2, 2, 3, 4, 6) in 16 bytes, the first of a pair in the low bits, and one scale byte e that stands for
// 2^(e - 127), 255 for NaN.  That is the form in which the scaled matrix instructions and the scaled conversions of
// gfx950 take both: 16 bytes and a byte are one lane's share of a 16 x 128 operand.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qk_device.h"
#include "qk_internal.h"

namespace qk {
namespace mx4 {

constexpr int kGroup = 32;                  // inputs of a scale
constexpr uint32_t kScaleNan = 255;

// A matrix as the kernels see it.
struct View {
    const uint8_t* codes;     // [rows, code_stride], 16-byte aligned, code_stride % 16 == 0
    const uint8_t* scales;    // [rows, scale_stride], 4-byte aligned, scale_stride % 4 == 0
    int64_t rows;
    int32_t cols;
    int32_t code_stride;
    int32_t scale_stride;
};

inline View view(const qk_mx4_state* st) {
    View v;
    v.codes = st->codes;
    v.scales = st->scales;
    v.rows = st->rows;
    v.cols = (int32_t)st->cols;
    v.code_stride = (int32_t)st->code_stride;
    v.scale_stride = (int32_t)st->scale_stride;
    return v;
}

// The scale operand of the conversions: the float whose exponent bits are the byte (0 counts as 2^-127, 255 as NaN).
__device__ __forceinline__ float scale_bits(uint32_t e) { return as_float(e << 23); }

}  // namespace mx4
}  // namespace qk
