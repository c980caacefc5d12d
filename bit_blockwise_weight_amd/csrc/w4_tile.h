// Device code shared by the kernels that multiply a few activation rows with 4-bit
// weights straight from memory (int4 with group scales; NF4 and other 16-level tables
// in the mixture-of-experts layer), for gfx950.
//
// One step of a wave is a "chunk": 16 weight rows x 128 k.  For its matrix instructions lane l holds
// row n = l % 16 and, with h = l / 16, the 16 bytes of k = 128 c + 32 h + [0, 32).  Where a scale
// group covers the whole chunk the four dwords are taken as they are, in any k order; for groups of
// 64 two lane swaps, for groups of 32 four, exchange dwords between the lane groups, so that a
// product of 64 k, or of 32, stays inside a group.
//
// From memory the codes come in whole 128-byte lines, 8 rows x 128 bytes per load instruction,
// and change to the layout above through a wave's own piece of LDS.  Loading them in that
// layout directly (16 rows x 64 bytes an instruction) streams 105 MB in 23 us against 18 us.
//
//   A = activations (row m = l % 16), B = W^T (column n = l % 16, the same k), D: column
//   n = l % 16, rows m = 4 (l / 16) + r.  A scale of row n is then one value per lane, applied to
//   the fp32 partial product of its group.
//
// The products are fp16 (16x16x32).  int4, two weights an instruction pair: (dword >> 4 i) & 0x000F000F leaves two codes in
// the low bits of the two halves; OR-ing 0x6400, an exponent whose last mantissa bits they become, gives 1024 + q, and
// 1024 + z taken off in fp16 leaves q - z, all of it exact.  The halves hold elements (1, 5), (0, 4), (3, 7), (2, 6)
// of the dword's eight (the first of a pair sits in the high nibble), so the activations are stored in that order
// too.  The zero point goes before the product, not after the sum: a sum of x (128 + q) less (128 + z) times that of x, the
// bf16 way, loses the neighbours of a large x whose q - z is 0.
//
// Activations other than fp16 ones are scaled by a power of two for each run of 128 (a chunk), 2^(14 - e) with e the
// exponent of the largest |x|, and become fp16 values: bf16 exactly down to 2^-31 of the largest, below to 2^-38 of it;
// fp32 (h of the expert layer) as a pair hi + lo, to 2^-24 of themselves, or 2^-38 of the largest.  Each chunk's sums are
// multiplied by 2^(e - 14) in fp32.
//
// 16 levels: codes become levels by a table in LDS of all 256 bytes.  A level is its bf16 copy times the power of two that
// brings the largest of the table to 2^14, as fp16: exact down to 2^-31 of the largest.
//
// Microscaled e2m1 (mx4.h): times bf16, the scaled conversion makes a weight with its scale, exact in bf16, and nothing is
// left to do after the product; activations are taken as they are, k in any order (a lane holds 32 k of one group).  Times
// fp16, whose range does not hold the scales, the bare e2m1 values are converted and a group's sum is scaled, as for int4
// in groups of 32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "qk_device.h"
#include "qk_internal.h"

namespace qk {
namespace w4 {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x3_t __attribute__((ext_vector_type(3)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Weight forms of the kernels: int4 times bf16 or fp16 activations, 16 levels times bf16, microscaled e2m1 times bf16 or
// fp16.
enum Form { kInt4Bf16 = 0, kInt4F16 = 1, kLevels = 2, kMx4Bf16 = 3, kMx4F16 = 4 };
constexpr bool is_int4(int f) { return f == kInt4Bf16 || f == kInt4F16; }
constexpr bool is_mx4(int f) { return f == kMx4Bf16 || f == kMx4F16; }

constexpr int kChunk = 128;               // k per step of a wave

__device__ __forceinline__ float f16_bits_to_float(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
__device__ __forceinline__ float bf16_bits_to_float(uint16_t b) { return as_float((uint32_t)b << 16); }

__device__ __forceinline__ uint16_t float_to_bits16(float v, bool f16) {
    if (f16) return __builtin_bit_cast(uint16_t, (_Float16)v);
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Brings the four dwords of the lane groups into the order in which no MFMA crosses a scale
// group, for NG groups in the chunk (see the top of the file).
template <int NG>
__device__ __forceinline__ void order_chunk(u32x4_t& d) {
    if constexpr (NG == 1) return;
    auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    if constexpr (NG == 2) {
        d[0] = a[0];
        d[1] = b[0];
        d[2] = a[1];
        d[3] = b[1];
        return;
    }
    auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d[0] = lo[0];
    d[1] = lo[1];
    d[2] = hi[0];
    d[3] = hi[1];
}
// First k, inside the chunk, of the eight that MFMA j takes from lane group h after order_chunk.
template <int NG>
__device__ __forceinline__ constexpr int chunk_k(int j, int h) {
    if (NG == 1) return 32 * h + 8 * j;
    if (NG == 2) return 64 * (j >> 1) + 32 * (h & 1) + 16 * (h >> 1) + 8 * (j & 1);
    return 32 * j + 8 * h;
}

// Constants that the compiler must keep in registers (as literals it cannot use v_and_or_b32,
// which may read one scalar register and no literal).
struct Magic {
    uint32_t m0, m4, e;          // masks of the low nibbles, of the next ones; exponent
    __device__ __forceinline__ Magic() : m0(0x000F000Fu), m4(0x00F000F0u), e(0x64006400u) {
        asm("" : "+s"(m0));
        asm("" : "+s"(m4));
        asm("" : "+v"(e));
    }
};

// Eight codes of a dword, less the zero point, as an MFMA fragment: 9 instructions.  zero: -(1024 + z) twice, zero4:
// -(64 + z).
__device__ __forceinline__ u32x4_t decode8(uint32_t w, f16x2_t zero, f16x2_t zero4, const Magic& k) {
    // 1024 + q less 1024 + z, or (1024 + 16 q) / 16 less 64 + z
    const uint32_t v = w >> 8;
    const f16x2_t sc = {0.0625f, 0.0625f};
    const uint32_t a0 = (w & k.m0) | k.e, a1 = (w & k.m4) | k.e, a2 = (v & k.m0) | k.e, a3 = (v & k.m4) | k.e;
    u32x4_t f;
    f[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, a0) + zero);
    f[1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, a1), sc, zero4));
    f[2] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, a2) + zero);
    f[3] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, a3), sc, zero4));
    return f;
}

// Activations of eight consecutive k in the order decode8 gives the weights: dword q holds int4_first(q) and the fourth
// after it.
__device__ __forceinline__ constexpr int int4_first(int q) { return q ^ 1; }
__device__ __forceinline__ u32x4_t int4_order(u32x4_t v) {
    u32x4_t r;
    r[0] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302);   // (1, 5)
    r[1] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100);   // (0, 4)
    r[2] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302);   // (3, 7)
    r[3] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100);   // (2, 6)
    return r;
}
__device__ __forceinline__ floatx4_t mfma(u32x4_t a, u32x4_t b, floatx4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
__device__ __forceinline__ floatx4_t mfma_bf16(u32x4_t a, u32x4_t b, floatx4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
// Eight e2m1 codes of a dword in their order: times a scale as bf16, or by themselves as fp16.
__device__ __forceinline__ u32x4_t decode8_mx4(uint32_t w, float scale) {
    u32x4_t f;
    f[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    f[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    f[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    f[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    return f;
}
__device__ __forceinline__ u32x4_t decode8_mx4(uint32_t w) {
    u32x4_t f;
    f[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
    f[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
    f[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
    f[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
    return f;
}

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

// A microscaled weight as the kernels see it.
struct Mx4View {
    const uint8_t* codes;     // [rows, stride], 16-byte aligned
    const uint8_t* scales;    // [rows, scale_stride], 4-byte aligned, scale_stride % 4 == 0
    int64_t stride;
    int32_t scale_stride;
    int32_t G;                // groups of a row
};

// A 16-level weight (NF4 and the like) as the kernels see it: rows of K elements, K a multiple
// of 64, so that every run of 64 k of a row lies in one quantization block.
struct LevelsView {
    const uint8_t* codes;
    const float* absmax;      // plain
    const int8_t* q8;         // nested
    const float* dq_scale;
    const float* dq_mean;
    int64_t stride;           // K / 2
    int32_t bshift;           // log2(block size)
    int32_t nested;
    float levels[16];         // their bf16 copies times 2^k, the largest magnitude in [2^14, 2^15)
    float unit;               // 2^-k
};

// Table of the 256 code bytes as (fp16 level of the high nibble, fp16 level of the low nibble),
// 32 copies so that each lane of the 32 that are served at a time reads a bank of its own: entry b of copy l at
// b * 256 + 4 l of LDS itself (the kernels have no other LDS than the dynamic part, which starts at 0), so that a
// v_perm makes the address.  The other half of the 256 bytes holds rows of codes (RowTiles).
constexpr int kTabBytes = 256 * 256;

__device__ __forceinline__ void build_table(uint8_t* tab, const float* levels, int tid, int threads) {
    for (int i = tid; i < 256 * 8; i += threads) {
        const int b = i >> 3;
        const uint32_t v = __builtin_bit_cast(uint32_t, (f16x2_t){(_Float16)levels[b >> 4], (_Float16)levels[b & 15]});
        *reinterpret_cast<u32x4_t*>(tab + b * 256 + (i & 7) * 16) = (u32x4_t){v, v, v, v};
    }
}

typedef const __attribute__((address_space(3))) uint32_t* lds_u32_t;

__device__ __forceinline__ u32x4_t decode8_table(uint32_t w, uint32_t lane4) {
    u32x4_t f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t off = __builtin_amdgcn_perm(w, lane4, 0x0C0C0000u | ((4u + i) << 8));
        f[i] = *reinterpret_cast<lds_u32_t>(off);
    }
    return f;
}

// ---------------------------------------------------------------------------
// Items of RT tiles of 16 weight rows (per row group) times M activation rows, one after the
// other by one workgroup of W waves: run() takes a run of items that share their activations.
//
// kw of the waves split k, W / kw groups of them take different rows.  A row is cut into windows
// of kw * 256 k; a wave takes one line (128 bytes, 256 k) of each row per window, and the
// partial outputs of the kw waves meet in LDS once per item, where the last wave to arrive adds
// them in wave order (the same bits every time).  No wave waits for another except every kSlots
// items, and per window of these where the activations do not stay.  While a wave works on one
// window the codes and scales of the next one (of the same item or the next) are already on their
// way into registers: 16 waves of a CU have 64 KB of codes in flight with RT = 2, 32 KB with RT = 1.
//
// The code is kept small (5 to 8 KB a kernel; the loops over chunks stay rolled): a launch fetches it
// anew, at 0.3 us a KB, and the smallest calls take 4 us.
//
// Activations live in LDS, zero past K, 16 bytes more than a row apart, so that a fragment read of 16
// rows falls in different banks: all of K for the whole run (kResident), or the current window,
// loaded one window ahead and used for kSlots items; sums are made in the same order either way.
// They are 16-bit values, for int4 in the order of its decoded codes, with a factor for each chunk and row behind them
// where they are scaled.  With kSplit they are fp32 and become two rows, hi and lo (activation m: rows 2 m and
// 2 m + 1).
// Scales go to LDS as well, per row and group the pair (scale, -(1024 + zero point)) for int4, the scale alone for
// levels; a wave writes and reads only its own, an odd number of entries apart.
//
// Codes are read by buffer loads whose range check returns 0 without a memory access: rows past
// the last one and lines past K cost no traffic and no branch.
// ---------------------------------------------------------------------------

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
    const int32_t n = (int32_t)(bytes < 0x7FFF0000 ? bytes : 0x7FFF0000);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, n, 0x00020000);
}
constexpr int32_t kOutside = 0x7FFF0000;  // an offset that no range reaches
constexpr int kNontemporal = 2;           // cache policy: each code byte is read once

// What a run of items reads.  Tile r of row group q in item i holds the rows base[r] + j,
// j = i * step + q * group_step + off[r] + [0, 16), as far as j < count.
template <int RT>
struct Rows {
    int64_t base[RT];
    int32_t off[RT];
    int32_t step, group_step;
    int32_t count;           // (count + 16) rows of codes stay under 2^31 - 2^16 bytes
    const void* x;           // 16-bit values, or fp32 (kSplit)
    const uint8_t* xrow;     // activation m is row xrow[m] of x; NULL: row m
    int32_t K;
    int32_t x_pitch;         // values from a row of x to the next
    int32_t x_rows;          // rows of x
    int32_t x_aligned;       // rows of x start at multiples of 4 bytes and K % 8 == 0
    int32_t M;               // activations
    int32_t kwl;             // log2(kw); at most w4_most_kwl() where x is not resident
};

// The product's row 4 h + i lands in register i of lane group h.  With few activation rows only the
// first MI registers of a group carry any: row m sits at 4 (m / MI) + m % MI.
template <int MI>
__device__ __forceinline__ constexpr int act_of_row(int row) { return MI * (row >> 2) + (row & (MI - 1)); }

constexpr int kLineK = 256;               // k of a 128-byte line of codes

// bytes of LDS beside the activations: scales, codes, partial sums of a few items and their counters
// With a table one workgroup of 16 waves fills a CU (two of 8 have no room for two tables): 16 tokens, top 8 of 64
// experts of 2048 x 1024, 66 us against 98 with 8 waves; one token 24 against 23.
constexpr int w4_waves(Form f) { return f == kLevels ? 16 : 8; }
constexpr int w4_put_bytes(Form f, int RT, int MI) { return w4_waves(f) * RT * 64 * MI * 4; }
// items that a window of activations serves, or (resident) whose sums wait for their last wave without a barrier.  One
// tile a wave above four activations: four, 38 us for the seven weights of a layer at M = 8, with two 45; for more
// than eight there is room for two.
constexpr int w4_slots(Form f, int RT, int MI, bool resident) {
    return resident || f == kLevels ? 2 : RT == 2 ? 3 : MI == 4 ? 2 : 4;
}
constexpr int w4_scale_bytes(Form f, int NG, int RT) { return w4_waves(f) * RT * 16 * ((2 * NG) | 1) * (is_int4(f) ? 8 : 4); }
// log2 of the waves that split a row, at most: a window of the activations has to fit where these do not stay
constexpr int w4_most_kwl(Form f, int MI) { return f == kLevels || MI == 4 ? 2 : 3; }
constexpr int w4_code_bytes(int RT) { return 8 * RT * 16 * 128; }       // of 8 waves; 8 more have theirs beside the table
constexpr int w4_fixed_bytes(Form f, int NG, int RT, int MI, bool resident) {
    return w4_scale_bytes(f, NG, RT) + w4_code_bytes(RT) + w4_slots(f, RT, MI, resident) * (w4_put_bytes(f, RT, MI) + w4_waves(f) * 4);
}
constexpr size_t kLdsBytes = 160 * 1024;  // of a CU

// Lets a kernel use more than 64 KB of LDS: once per device.
template <auto kKernel>
hipError_t allow_lds(size_t lds) {
    if (lds <= 65536) return hipSuccess;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return hipSuccess;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kKernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)kLdsBytes);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Whether activations are scaled chunk by chunk: not where they are what the product takes.
constexpr bool w4_scaled(Form f, bool split) { return split || f == kInt4Bf16 || f == kLevels; }
// bytes of LDS that the activations take: rows of 16-bit values (two an activation with kSplit), and the factors of the
// chunks for the 4 mi rows of the operand
inline size_t w4_x_bytes(Form f, int kw, int rows, int mi, bool split, int64_t K, bool resident) {
    const size_t k = resident ? (size_t)((K + kLineK - 1) / kLineK) * kLineK : (size_t)kw * kLineK;
    return (size_t)rows * (k * 2 + 16) + (w4_scaled(f, split) ? k / kChunk * (size_t)(16 * mi) : 0);
}
// log2 of the waves that split a row of K: as many as it has lines, up to 8; more (some then have nothing to do) as
// long as there are fewer items than CUs.  rows: of all items, in pieces of `piece` rows that a wave takes
inline int w4_kwl(Form f, int64_t K, int64_t rows, int piece, int most) {
    const int64_t n = (K + kLineK - 1) / kLineK, pieces = (rows + piece - 1) / piece;
    int kwl = n > 4 ? 3 : n > 2 ? 2 : n > 1 ? 1 : 0;
    if (kwl > most) kwl = most;
    while (kwl < most && pieces * ((int64_t)1 << kwl) < (int64_t)w4_waves(f) * device_cu_count()) ++kwl;
    return kwl;
}

template <int F, int NG, int RT, int MI, bool kResident, bool kSplit>
struct RowTiles {
    static constexpr Form kForm = (Form)F;
    static constexpr int W = w4_waves(kForm);
    static constexpr int kThreads = W * 64;
    static constexpr bool kScaled = w4_scaled(kForm, kSplit);
    static constexpr int kOpRows = 4 * MI;                      // rows of the operand that carry activations, at most
    static constexpr int U = 2;                                 // chunks of a wave in a window
    static constexpr int kMfmas = 4 / NG;                       // MFMAs per scale group
    static constexpr int kEntries = U * NG;                     // scale groups of a wave's chunks in a window
    static constexpr int kSPitch = kEntries | 1;
    static constexpr int kScaleBytes = w4_scale_bytes(kForm, NG, RT);
    static constexpr int kCodeBytes = w4_code_bytes(RT);        // a window's codes changing layout
    static constexpr int kCodePitch = F == kLevels ? 256 : 128; // from row to row there
    static constexpr int kPutBytes = w4_put_bytes(kForm, RT, MI);
    static constexpr int kSlots = w4_slots(kForm, RT, MI, kResident);
    // units of x per thread and batch; a window's fit one batch
    static constexpr int kMaxM = kSplit ? 2 * MI : 4 * MI;
    static constexpr int kXUnits = kResident ? (MI == 1 && F != kLevels ? 1 : 2) : ((kMaxM * 32 << w4_most_kwl(kForm, MI)) + kThreads - 1) / kThreads;
    static constexpr int kFixedBytes = w4_fixed_bytes(kForm, NG, RT, MI, kResident);

    static_assert(RT == 1 || RT == 2);
    // The scales of a window come by one load per kind, in lane 16 r + n for row n of tile r (a load instruction that
    // touches many lines costs as much as one that brings a kilobyte of codes): as dwords from an address rounded
    // down to 4 bytes, put right when they land.
    struct alignas(4 * MI) Factors {
        float v[MI];
        __device__ __forceinline__ float operator[](int i) const { return v[i]; }
    };
    struct ScaleZero {
        float s;
        uint32_t zero;       // -(1024 + z) in fp16, twice
    };
    // (kMx4Bf16: the scale bytes of a chunk's four groups)
    typedef std::conditional_t<is_int4(F), ScaleZero, std::conditional_t<F == kMx4Bf16, uint32_t, float>> Scale;
    struct Fetched {
        u32x4_t c[RT][2];
        u32x4_t s;           // int4: 2 NG scales; levels: four block scales of a plain weight; mx4: eight scales
        uint32_t s4;         // int4 with NG = 4: the fifth dword
        u32x3_t z;           // int4: 2 NG zero points; levels: q8 of four blocks
        u32x2_t d;           // levels: double-quantization scales of the first block and of the next 256
    };

    // lds (behind the level table, for kLevels): kFixedBytes + w4_x_bytes(), 16-byte aligned.
    // out(item, q, put), called by one wave, stores the outputs of row group q of an item from the partial sums.
    template <class V, class Out>
    static __device__ __forceinline__ void run(const V& w, const Rows<RT>& p, int item0, int item1,
                                               uint8_t* lds, Out&& out) {
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int n = lane & 15, h = lane >> 4;
        const int kw = 1 << p.kwl, wk = wave & (kw - 1), wr = wave >> p.kwl;
        Scale* slds = reinterpret_cast<Scale*>(lds) + wave * (RT * 16 * kSPitch);
        // With a table the rows of codes are 256 bytes apart: eight waves' lie behind the table's entries (in front of
        // lds, see there), those of eight more share a piece of their own, four and four.
        uint8_t* clds = lds + kScaleBytes + wave * (RT * 16 * 128);
        if constexpr (F == kLevels) {
            extern __shared__ __align__(16) uint8_t lds0[];
            clds = wave < 8 ? lds0 + 128 + wave * (RT * 16 * 256)
                            : lds + kScaleBytes + (wave & 3) * (RT * 16 * 256) + (wave >> 2 & 1) * 128;
        }
        float* put = reinterpret_cast<float*>(lds + kScaleBytes + kCodeBytes);
        int* arrived = reinterpret_cast<int*>(lds + kScaleBytes + kCodeBytes + kSlots * kPutBytes);
        uint8_t* xlds = lds + kFixedBytes;
        const int nchunk = (p.K + kChunk - 1) / kChunk;
        const int wchunks = kw * U;
        const int xchunks = kResident ? (nchunk + U - 1) / U * U : wchunks;   // chunks of x that LDS holds
        const int xpitch = xchunks * (2 * kChunk) + 16;
        const int xrows = kSplit ? 2 * p.M : p.M;
        const Magic magic;
        float mean = 0.0f;
        uint32_t zbase = 0;                                      // -1024 in fp16, and the zero point where there is no array
        if constexpr (F == kLevels) mean = w.nested ? *w.dq_mean : 0.0f;
        if constexpr (is_int4(F)) zbase = 0xE400u + (w.zeros ? 0u : 8u);
        // Staging of activations, thread by thread, rows as if they had 2^ush units of 8 values.  A unit is read
        // as four dwords from an address rounded down to 4 bytes, and one dword more where rows may start
        // between dwords, and put right (and zero past K) when it is stored.
        const uint64_t xa = reinterpret_cast<uint64_t>(p.x);
        const uint32_t xodd = (uint32_t)(xa & 2);
        const __amdgpu_buffer_rsrc_t xbuf = buffer(reinterpret_cast<const void*>(xa & ~3ull),
                                                   ((int64_t)p.x_rows * p.x_pitch * (kSplit ? 4 : 2) + xodd + 3) / 4 * 4);
        const int units = xchunks * (kChunk / 8);
        const int ush = 32 - __builtin_clz(units - 1);
        const int total = p.M << ush;
        u32x4_t xr[kXUnits][kSplit ? 2 : 1];
        uint32_t xe[kXUnits];
        auto x_load = [&](int base, int k0) {
#pragma unroll
            for (int b = 0; b < kXUnits; ++b) {
                const int i = base + b * kThreads + tid, m = i >> ush, u = i & ((1 << ush) - 1), k = k0 + 8 * u;
                const bool in = i < total && u < units && k < p.K;
                const int row = in && p.xrow ? p.xrow[m] : m;
                if constexpr (kSplit) {
                    const int32_t off = in ? (row * p.x_pitch + k) * 4 : kOutside;
                    xr[b][0] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, off, 0, 0);
                    xr[b][1] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, off, 16, 0);
                } else {
                    const int32_t off = in ? ((row * p.x_pitch + k) * 2 + xodd) & ~3 : kOutside;
                    xr[b][0] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, off, 0, 0);
                    xe[b] = __builtin_amdgcn_raw_buffer_load_b32(xbuf, off, p.x_aligned ? kOutside : 16, 0);
                }
            }
        };
        // Unit b of a batch as 8 16-bit values: from the dwords it was read in, zero past K.
        auto x_unit = [&](int b, int m, int k) -> u32x4_t {
            u32x4_t v = xr[b][0];
            if (!p.x_aligned) {
                const int row = p.xrow ? p.xrow[m < p.M ? m : 0] : m;
                const uint32_t sh = 8 * (((row * p.x_pitch + k) * 2 + xodd) & 2);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t d = __builtin_amdgcn_alignbit(q < 3 ? xr[b][0][q + 1] : xe[b], xr[b][0][q], sh);
                    v[q] = k + 2 * q + 1 < p.K ? d : k + 2 * q < p.K ? d & 0xFFFFu : 0u;
                }
            }
            return v;
        };
        // Stores unit b of a batch, unit i of all.  Every thread stores (what lies outside, to the 16 bytes behind row 0,
        // which nobody reads): under a condition the compiler would move the loads down to it, behind those of the codes.
        auto x_store_unit = [&](uint8_t* dst, int b, int i, int k0) {
            const int m = i >> ush, u = i & ((1 << ush) - 1);
            const bool in = i < total && u < units;
            u32x4_t hi, lo;
            if constexpr (!kSplit) hi = x_unit(b, m, k0 + 8 * u);
            if constexpr (kScaled) {
                float v[8];
                uint32_t big;
                if constexpr (kSplit) {
                    big = 0;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        v[q] = as_float(xr[b][q >> 2][q & 3]);
                        big = max(big, as_uint(v[q]) & 0x7FFFFFFFu);
                    }
                } else {
                    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
                    u16x2_t most = {0, 0};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        v[2 * q] = bf16_lo(hi[q]);
                        v[2 * q + 1] = bf16_hi(hi[q]);
                        most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2_t, hi[q] & 0x7FFF7FFFu));
                    }
                    big = (uint32_t)max(most[0], most[1]) << 16;
                }
                // (16 lanes hold a chunk; below 2^-112, where 2^(e - 14) ends, by the factor of 2^-112; an infinity
                // or a NaN stays one)
                const uint32_t e = max(group_max_u32<16>(big) >> 23, 15u);
                const float up = as_float((268u - e) << 23);                    // 2^(14 - (e - 127))
                if (in && (lane & 15) == 0) {
                    float* f = reinterpret_cast<float*>(dst + xrows * xpitch) + (u >> 4) * kOpRows + (kSplit ? 2 * m : m);
                    f[0] = as_float((e - 14u) << 23);
                    if constexpr (kSplit) f[1] = f[0];
                }
                // in the order in which they are stored
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i0 = F == kLevels ? 2 * q : int4_first(q), i1 = F == kLevels ? 2 * q + 1 : int4_first(q) + 4;
                    const float a = v[i0] * up, c = v[i1] * up;
                    const f16x2_t near = {(_Float16)a, (_Float16)c};
                    hi[q] = __builtin_bit_cast(uint32_t, near);
                    if constexpr (kSplit)
                        lo[q] = __builtin_bit_cast(uint32_t, (f16x2_t){(_Float16)(a - (float)near[0]), (_Float16)(c - (float)near[1])});
                }
            } else if constexpr (is_int4(F)) {
                hi = int4_order(hi);
            }
            const int at = in ? (kSplit ? 2 * m : m) * xpitch + 16 * u : xpitch - 16;
            *reinterpret_cast<u32x4_t*>(dst + at) = hi;
            if constexpr (kSplit) *reinterpret_cast<u32x4_t*>(dst + (in ? at + xpitch : at)) = lo;
        };
        auto x_store = [&](uint8_t* dst, int base, int k0) {
            // (with two tiles and two sums a lane the registers do not hold several units' intermediates: there the units
            // come one after the other, each moved to the front)
            if constexpr (!kResident && RT == 2 && MI > 1) {
                const int batch = base + kXUnits * kThreads;
#pragma unroll 1
                for (; base < batch; base += kThreads) {
                    x_store_unit(dst, 0, base + tid, k0);
#pragma unroll
                    for (int b = 0; b + 1 < kXUnits; ++b) {
                        xr[b][0] = xr[b + 1][0];
                        if constexpr (kSplit) xr[b][1] = xr[b + 1][1];
                        else xe[b] = xe[b + 1];
                    }
                }
            } else {
#pragma unroll
                for (int b = 0; b < kXUnits; ++b) x_store_unit(dst, b, base + b * kThreads + tid, k0);
            }
        };

        // Codes and scales of the wave's line in the window that starts at chunk c0 of the item whose tile 0
        // of this wave's row group starts at row j.  One descriptor per tile covers the whole run of rows (under
        // 2 GB, see the callers), so a window costs a few scalar instructions; j < 0: nothing.
        __amdgpu_buffer_rsrc_t cbuf[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) cbuf[r] = buffer(w.codes + p.base[r] * w.stride, (int64_t)p.count * w.stride);
        const int32_t stride = (int32_t)w.stride;
        const int32_t voff = (lane >> 3) * stride + 16 * (lane & 7);
        // scales: row of the lane relative to base[0]; lanes 32..63 and what is past the end read nothing
        const int32_t apart = (int32_t)(p.base[RT - 1] - p.base[0]) + p.off[RT - 1];
        const int32_t srow = n + (lane & 16 ? apart : p.off[0]);
        const int64_t srows = p.base[RT - 1] - p.base[0] + p.count;
        __amdgpu_buffer_rsrc_t sbuf, zbuf, dbuf;
        uint32_t sfirst = 0, zfirst = 0, dfirst = 0;             // of base[0], from the rounded-down address, in its unit
        if constexpr (F == kLevels) {
            const int64_t e0 = p.base[0] * p.K, b0 = e0 >> w.bshift;
            const int64_t blocks = ((srows * p.K + (e0 - (b0 << w.bshift)) - 1) >> w.bshift) + 1;
            sbuf = buffer(w.absmax + b0, w.nested ? 0 : blocks * 4);
            const uint64_t qa = reinterpret_cast<uint64_t>(w.q8 + b0);
            zbuf = buffer(reinterpret_cast<const void*>(qa & ~3ull), w.nested ? (blocks + (int64_t)(qa & 3) + 3) / 4 * 4 : 0);
            const int64_t dlast = (b0 + blocks - 1) / QK_DQ_BLOCK, d0 = b0 / QK_DQ_BLOCK;
            dbuf = buffer(w.dq_scale + d0, w.nested ? (dlast - d0 + 1) * 4 : 0);
            sfirst = (uint32_t)(e0 - (b0 << w.bshift));          // elements of the first block before base[0]
            zfirst = (uint32_t)(qa & 3);
            dfirst = (uint32_t)(b0 % QK_DQ_BLOCK);
        } else if constexpr (is_mx4(F)) {
            sbuf = buffer(w.scales + p.base[0] * w.scale_stride, srows * w.scale_stride);
        } else {
            const uint64_t sa = reinterpret_cast<uint64_t>(w.scales + p.base[0] * w.G);
            sbuf = buffer(reinterpret_cast<const void*>(sa & ~3ull), (srows * w.G * 2 + (int64_t)(sa & 3) + 3) / 4 * 4);
            const uint64_t za = reinterpret_cast<uint64_t>(w.zeros + p.base[0] * w.G);
            zbuf = buffer(reinterpret_cast<const void*>(za & ~3ull), w.zeros ? (srows * w.G + (int64_t)(za & 3) + 3) / 4 * 4 : 0);
            sfirst = (uint32_t)(sa & 3);
            zfirst = (uint32_t)(za & 3);
        }
        // Where the lane's scales of a window start: int4, the index of the first group from base[0]; levels, the
        // block of the first 64 values, from the first block (and in `run` which 64 values of it).
        auto scale_at = [&](int j, int c) -> uint32_t {
            if constexpr (F == kLevels) return (uint32_t)(j + srow) * (uint32_t)p.K + (uint32_t)c * kChunk + sfirst;
            else if constexpr (is_mx4(F)) return (uint32_t)(j + srow) * (uint32_t)w.scale_stride + (uint32_t)c * 4;
            else return (uint32_t)(j + srow) * (uint32_t)w.G + (uint32_t)((c * kChunk) >> w.gshift);
        };
        uint32_t at = 0;                                         // of the window in flight
        int left = 0;                                            // and the scale groups (runs of 64) from there to the row's end
        auto fetch = [&](Fetched& f, int j, int c0) {
            const int c = c0 + wk * U;
            const bool in = j >= 0 && c < nchunk, lane_in = in && lane < 16 * RT;
            at = scale_at(j, c);
            if constexpr (F == kLevels) left = (p.K >> 6) - 2 * c;
            else if constexpr (is_mx4(F)) left = w.G - 4 * c;
            else left = w.G - ((c * kChunk) >> w.gshift);
            if constexpr (F == kLevels) {
                const uint32_t blk = at >> w.bshift;
                f.s = __builtin_amdgcn_raw_buffer_load_b128(sbuf, lane_in ? 4 * blk : kOutside, 0, 0);
                const u32x2_t t = __builtin_amdgcn_raw_buffer_load_b64(zbuf, lane_in ? (blk + zfirst) & ~3u : kOutside, 0, 0);
                f.z[0] = t[0];
                f.z[1] = t[1];
                f.d = __builtin_amdgcn_raw_buffer_load_b64(dbuf, lane_in ? (blk + dfirst) / QK_DQ_BLOCK * 4 : kOutside, 0, 0);
            } else if constexpr (is_mx4(F)) {
                const u32x2_t t = __builtin_amdgcn_raw_buffer_load_b64(sbuf, lane_in ? at : kOutside, 0, 0);
                f.s[0] = t[0];
                f.s[1] = t[1];
            } else {
                const uint32_t so = lane_in ? (2 * at + sfirst) & ~3u : kOutside;
                const uint32_t zo = lane_in ? (at + zfirst) & ~3u : kOutside;
                if constexpr (NG == 4) {
                    f.s = __builtin_amdgcn_raw_buffer_load_b128(sbuf, so, 0, 0);
                    f.s4 = __builtin_amdgcn_raw_buffer_load_b32(sbuf, so, 16, 0);
                    f.z = __builtin_amdgcn_raw_buffer_load_b96(zbuf, zo, 0, 0);
                } else {
                    if constexpr (NG == 2) {
                        const u32x3_t t = __builtin_amdgcn_raw_buffer_load_b96(sbuf, so, 0, 0);
                        f.s[0] = t[0];
                        f.s[1] = t[1];
                        f.s[2] = t[2];
                    } else {
                        const u32x2_t t = __builtin_amdgcn_raw_buffer_load_b64(sbuf, so, 0, 0);
                        f.s[0] = t[0];
                        f.s[1] = t[1];
                    }
                    const u32x2_t t = __builtin_amdgcn_raw_buffer_load_b64(zbuf, zo, 0, 0);
                    f.z[0] = t[0];
                    f.z[1] = t[1];
                }
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                // tiles behind the last row, too, are outside: no offset of theirs is formed
                const bool in_tile = in && j + p.off[r] < p.count;
                const int32_t coff = in_tile ? (j + p.off[r]) * stride + c * (kChunk / 2) : kOutside;
#pragma unroll
                for (int q = 0; q < 2; ++q)                      // rows 8 q + lane / 8
                    f.c[r][q] = __builtin_amdgcn_raw_buffer_load_b128(cbuf[r], voff, in_tile ? coff + 8 * q * stride : kOutside,
                                                                      kNontemporal);
            }
        };

        // The lanes of a wave exchange codes and scales through LDS.  Nothing waits (a wave's LDS accesses keep their
        // order), but the compiler must not move one lane's reads across another's writes.
        auto exchanged = [] {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        // What was fetched goes to the wave's own LDS: codes from lines to fragments (16-byte unit u of row r
        // sits in unit u ^ (r % 8) of its row), scales converted.
        auto land = [&](const Fetched& f) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    *reinterpret_cast<u32x4_t*>(clds + (16 * r + 8 * q + (lane >> 3)) * kCodePitch +
                                                16 * ((lane & 7) ^ (lane >> 3))) = f.c[r][q];
            }
            if (lane >= 16 * RT) return;
            if constexpr (F == kLevels) {
                // the four runs of 64: their blocks follow the first one's
                const uint32_t blk = at >> w.bshift, run = at >> 6, shift = w.bshift - 6;
                const uint32_t q = __builtin_amdgcn_alignbyte(f.z[1], f.z[0], blk + zfirst);
#pragma unroll
                for (int e = 0; e < kEntries; ++e) {
                    const uint32_t o = ((run + e) >> shift) - blk;
                    float v;
                    if (w.nested) {
                        const uint32_t dq = (blk + o + dfirst) / QK_DQ_BLOCK - (blk + dfirst) / QK_DQ_BLOCK;
                        v = __fadd_rn(__fmul_rn((float)(int8_t)(q >> (8 * o)), as_float(dq ? f.d[1] : f.d[0])), mean);
                    } else {
                        v = as_float(o == 0 ? f.s[0] : o == 1 ? f.s[1] : o == 2 ? f.s[2] : f.s[3]);
                    }
                    slds[lane * kSPitch + e] = e < left ? v * w.unit : 0.0f;
                }
            } else if constexpr (is_mx4(F)) {
                // what lies behind the row's last scale meets activations of 0, but may be a NaN: 0, 2^-127, instead
                uint32_t sv[2] = {f.s[0], f.s[1]};
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int n4 = left - 4 * u;
                    sv[u] = n4 >= 4 ? sv[u] : n4 <= 0 ? 0u : sv[u] & ((1u << (8 * n4)) - 1u);
                }
#pragma unroll
                for (int e = 0; e < kEntries; ++e) {
                    if constexpr (F == kMx4Bf16) {
                        slds[lane * kSPitch + e] = sv[e];
                    } else {
                        const uint32_t b = (sv[e >> 2] >> (8 * (e & 3))) & 255u;
                        slds[lane * kSPitch + e] = as_float(b == 0 ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23);
                    }
                }
            } else {
                const uint32_t sh = 8 * ((2 * at + sfirst) & 2);
                uint32_t sv[NG], zv[NG == 4 ? 2 : 1];
                sv[0] = __builtin_amdgcn_alignbit(f.s[1], f.s[0], sh);
                if constexpr (NG >= 2) sv[1] = __builtin_amdgcn_alignbit(f.s[2], f.s[1], sh);
                if constexpr (NG == 4) {
                    sv[2] = __builtin_amdgcn_alignbit(f.s[3], f.s[2], sh);
                    sv[3] = __builtin_amdgcn_alignbit(f.s4, f.s[3], sh);
                }
                zv[0] = __builtin_amdgcn_alignbyte(f.z[1], f.z[0], at + zfirst);
                if constexpr (NG == 4) zv[1] = __builtin_amdgcn_alignbyte(f.z[2], f.z[1], at + zfirst);
                // What lies behind the row's last group (the next row's, or memory of somebody else) meets activations
                // of 0, but may be an infinity or a NaN: a scale of 0 instead.
#pragma unroll
                for (int i = 0; i < NG; ++i) sv[i] &= left >= 2 * i + 2 ? 0xFFFFFFFFu : left == 2 * i + 1 ? 0xFFFFu : 0u;
                if constexpr (NG == 1) {                         // groups of 256 and more: both chunks in one
                    if (w.gshift > 7) {
                        sv[0] = (sv[0] & 0xFFFFu) | (sv[0] << 16);
                        zv[0] = (zv[0] & 0xFFu) | (zv[0] << 8);
                    }
                }
#pragma unroll
                for (int e = 0; e < kEntries; ++e) {
                    const uint16_t bits = (uint16_t)(sv[e >> 1] >> (16 * (e & 1)));
                    const uint32_t z = ((zv[e >> 2] >> (8 * (e & 3))) & 255u) + zbase;
                    slds[lane * kSPitch + e] = Scale{w.scale_f16 ? f16_bits_to_float(bits) : bf16_bits_to_float(bits), z | z << 16};
                }
            }
        };
        // the lane's row of the activation operand, and where the factors of its rows of the product start
        const int am = act_of_row<MI>(n);
        const int arow = (am < xrows ? am : xrows - 1) * xpitch;
        const int xfac = xrows * xpitch + 4 * MI * h;
        float y[RT][MI];
        // The products of one window.  Rolled: a workgroup runs this code a few times at most, and fetching an
        // instruction for the first time costs more than looping.
        auto compute = [&](int c0, const uint8_t* xwin) {
            const int first = kResident ? c0 + wk * U : wk * U;  // the wave's first chunk in LDS
            const uint8_t* ax = xwin + arow + first * (2 * kChunk);
            const Scale* sp = slds + n * kSPitch;
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                u32x4_t c[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    c[r] = *reinterpret_cast<const u32x4_t*>(clds + (16 * r + n) * kCodePitch + 16 * ((4 * u + h) ^ (n & 7)));
                u32x4_t a[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a[j] = *reinterpret_cast<const u32x4_t*>(ax + 2 * (u * kChunk + chunk_k<NG>(j, h)));
#pragma unroll
                for (int r = 0; r < RT; ++r) order_chunk<NG>(c[r]);
                // A chunk's sums, scale group by scale group; its factor at the end.
                float t[RT][MI];
                Factors x;
                if constexpr (kScaled) x = *reinterpret_cast<const Factors*>(xwin + xfac + (first + u) * (4 * kOpRows));
#pragma unroll
                for (int q = 0; q < NG; ++q) {
                    Scale s[RT];
                    floatx4_t acc[RT];
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        s[r] = sp[16 * r * kSPitch + u * NG + q];
                        acc[r] = (floatx4_t){0, 0, 0, 0};
                    }
#pragma unroll
                    for (int j = q * kMfmas; j < (q + 1) * kMfmas; ++j) {
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            if constexpr (F == kMx4Bf16) {
                                acc[r] = mfma_bf16(a[j], decode8_mx4(c[r][j], as_float((s[r] >> (8 * h) & 255u) << 23)), acc[r]);
                            } else if constexpr (F == kMx4F16) {
                                acc[r] = mfma(a[j], decode8_mx4(c[r][j]), acc[r]);
                            } else if constexpr (F == kLevels) {
                                acc[r] = mfma(a[j], decode8_table(c[r][j], 4 * (lane & 31)), acc[r]);
                            } else {
                                const f16x2_t zero = __builtin_bit_cast(f16x2_t, s[r].zero), zero4 = zero + (f16x2_t){960, 960};
                                acc[r] = mfma(a[j], decode8(c[r][j], zero, zero4, magic), acc[r]);
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        float sr = 1.0f;
                        if constexpr (is_int4(F)) sr = s[r].s;
                        else if constexpr (F != kMx4Bf16) sr = s[r];
#pragma unroll
                        for (int i = 0; i < MI; ++i) {
                            if constexpr (F == kMx4Bf16) y[r][i] += acc[r][i];
                            else if constexpr (!kScaled) y[r][i] = fmaf(sr, acc[r][i], y[r][i]);
                            else t[r][i] = q == 0 ? sr * acc[r][i] : fmaf(sr, acc[r][i], t[r][i]);
                        }
                    }
                }
                if constexpr (kScaled) {
#pragma unroll
                    for (int i = 0; i < MI; ++i) {
#pragma unroll
                        for (int r = 0; r < RT; ++r) y[r][i] = fmaf(x[i], t[r][i], y[r][i]);
                    }
                }
            }
        };

        Fetched f;
        float* mine = put + wave * (RT * 64 * MI) + lane;        // this wave's sums of an item, slot by slot
        auto save = [&](int slot) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < MI; ++i) mine[slot * (kPutBytes / 4) + (r * MI + i) * 64] = y[r][i];
        };
        auto clear = [&] {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < MI; ++i) y[r][i] = 0.0f;
        };
        // The wave's sums of an item are saved: the last wave of the row group to say so adds them up.
        auto finish = [&](int item, int slot) {
            int before = 0;
            if (lane == 0)
                before = __hip_atomic_fetch_add(&arrived[slot * W + wr], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_WORKGROUP);
            if (__builtin_amdgcn_readfirstlane(before) == kw - 1) out(item, wr, put + slot * (kPutBytes / 4));
        };
        // after the last item of the slots: no sum may be overwritten before it is added
        auto recycle = [&] {
            __syncthreads();
            if (tid < kSlots * W) arrived[tid] = 0;
            __syncthreads();
        };
        int j = item0 * p.step + wr * p.group_step;              // row of the next window to fetch
        x_load(0, 0);
        fetch(f, j, 0);
        if (tid < kSlots * W) arrived[tid] = 0;
        clear();
        // Every step: what was fetched goes to LDS, the next window's loads are issued (without a condition: a
        // branch around them would make later waits cover them; past the end every offset is outside and nothing is
        // read), the products are made.
        if constexpr (kResident) {
            // item by item, window by window
            x_store(xlds, 0, 0);
#pragma unroll 1
            for (int base = kXUnits * kThreads; base < total; base += kXUnits * kThreads) {
                x_load(base, 0);
                x_store(xlds, base, 0);
            }
            __syncthreads();
            int item = item0, c0 = 0, slot = 0;
            while (true) {
                exchanged();
                land(f);
                exchanged();
                const bool last = c0 + wchunks >= nchunk;        // last window of the item
                const bool end = last && item + 1 >= item1;
                const int nc = last ? 0 : c0 + wchunks;
                if (last) j += p.step;
                fetch(f, end ? -1 : j, nc);
                if (c0 + wk * U < nchunk) compute(c0, xlds);
                c0 = nc;
                if (!last) continue;
                save(slot);
                clear();
                finish(item, slot);
                if (end) break;
                ++item;
                if (++slot == kSlots) {
                    slot = 0;
                    recycle();
                }
            }
        } else {
            // kSlots items at a time, so that a window of activations serves all of them; their sums stay in LDS
            // from window to window
            for (int first = item0; first < item1; first += kSlots) {
                const int items = item1 - first < kSlots ? item1 - first : kSlots;
                const int j0 = j;
#pragma unroll 1
                for (int c0 = 0; c0 < nchunk; c0 += wchunks) {
                    const bool last = c0 + wchunks >= nchunk;
                    const int nc = last ? 0 : c0 + wchunks;
                    __syncthreads();                             // the last window's reads
                    x_store(xlds, 0, c0 * kChunk);
                    x_load(0, nc * kChunk);
                    __syncthreads();
#pragma unroll 1
                    for (int slot = 0; slot < items; ++slot) {
                        exchanged();
                        land(f);
                        exchanged();
                        const bool turn = slot + 1 == items;     // on to the next window, or to the next items
                        const bool end = turn && last && first + items >= item1;
                        j = turn && !last ? j0 : j + p.step;
                        fetch(f, end ? -1 : j, turn ? nc : c0);
                        if (c0 > 0)
#pragma unroll
                            for (int r = 0; r < RT; ++r)
#pragma unroll
                                for (int i = 0; i < MI; ++i) y[r][i] = mine[slot * (kPutBytes / 4) + (r * MI + i) * 64];
                        else
                            clear();
                        if (c0 + wk * U < nchunk) compute(c0, xlds);
                        save(slot);
                        if (last) finish(first + slot, slot);
                    }
                }
                if (first + items < item1) recycle();
            }
        }
        __syncthreads();
    }

    // From the partial sums: output o (o < 64 MI) of tile r of row group q, the waves added in their
    // order.  Its row in the tile is o % 16, its activation row act_of(o).
    static __device__ __forceinline__ float sum(const float* put, int kwl, int q, int r, int o) {
        const float* first = put + ((q << kwl) * RT + r) * (64 * MI) + o;
        constexpr int kMost = 8;                                 // waves that split a row
        float p[kMost], v = 0.0f;                                // all reads first, then the sum
#pragma unroll
        for (int w = 0; w < kMost; ++w) p[w] = first[(w < (1 << kwl) ? w : 0) * (RT * 64 * MI)];
#pragma unroll
        for (int w = 0; w < kMost; ++w) v += w < (1 << kwl) ? p[w] : 0.0f;
        return v;
    }
    static __device__ __forceinline__ int act_of(int o) { return MI * ((o & 63) >> 4) + (o >> 6); }
    // Where that output of activation row m sits.
    static __device__ __forceinline__ int place_of(int row, int m) {
        return 64 * (m & (MI - 1)) + 16 * (m / MI) + row;
    }
};

}  // namespace w4
}  // namespace qk
