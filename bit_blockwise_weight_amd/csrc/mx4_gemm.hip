// Products of microscaled 4-bit matrices on the scaled matrix cores of gfx950: Y = X W^T, and the gate / up and down
// products of a mixture of experts over a routing.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes, of each operand, a row's 32 codes (16 bytes) and their scale byte from every
// lane: row l % 16, group l / 16 of the four.  Which four groups those are does not matter as long as both operands
// agree.  A stage is 256 inputs, a 128-byte line of a row; its two instructions s = 0, 1 take group 2 (l / 16) + s, so
// that a lane's two scale bytes are neighbours and the instruction picks one by its byte select.  W is the first operand: a
// lane then ends up with 4 consecutive columns of one row of Y.
//
// Codes and scales go from memory straight to LDS.  A row of a stage keeps its 128 bytes, the pieces of 16 in an order
// turned by the row: what lanes read at a time then falls in all banks (slot_of).
//
// What lies past the last input of a row (the row's padding, the next row, nothing) is in the last line too: before that
// line is used its groups past the end get the scale 1 in both operands and its codes past the end become 0 in X.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "mx4.h"

namespace qk {
namespace {

using namespace mx4;

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef int v4i_t __attribute__((ext_vector_type(4)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kLineK = 256;                // inputs of a stage: 128 bytes of codes, 8 of scales
constexpr int kXcds = 8;

enum Mode { kDense, kUp, kDown };

struct GemmArgs {
    View x, w;
    void* y;                   // dense: [M, N]; up: h [slots, I]; down: the weighted parts [slots, H], fp32
    const int32_t* list;       // of the plan: the slots by expert
    const int32_t* tiles;      // of the plan: how many tiles, and from the 4th number on each one's rows
    const float* weights;      // down: of the slots
    int64_t M;                 // dense: rows of x
    int64_t N;                 // outputs of a row: N, I or H
    int64_t w_rows;            // rows of an expert's weights: 2 I or H
    int32_t y_dtype;
    int32_t E;
    int32_t slots;
    uint32_t per_token;        // ceil(2^32 / top_k): the token of a slot is the upper half of slot * per_token; 0: the slot
};

// The part of the product that a workgroup makes: rows of X by position 0..count-1, columns n0 on, of one expert.
struct Tile {
    int64_t m0;                // dense: first row of X and Y; otherwise the first place in the list of slots
    int64_t n0;
    int32_t count;
    int32_t expert;            // E: slots without one
};

// Numbers of the plan, which no kernel here writes: through the scalar cache.
__device__ __forceinline__ int32_t plan_number(const int32_t* p) {
    return *(const __attribute__((address_space(4))) int32_t*)(uintptr_t)p;
}

// Rows and number of the tiles of a launch.
template <bool kExperts, int BM, int BN>
struct Tiling {
    uint32_t rows, cols;
    __device__ __forceinline__ explicit Tiling(const GemmArgs& a) {
        rows = kExperts ? (uint32_t)plan_number(a.tiles) : (uint32_t)((a.M + BM - 1) / BM);
        cols = (uint32_t)((a.N + BN - 1) / BN);
    }
    __device__ __forceinline__ uint32_t count() const { return rows * cols; }

    // Tile `id`, made on XCD id % 8: each XCD gets a run of tiles, 8 rows of them at a time going through all columns, so that
    // the tiles of an XCD share operands in its L2.  The experts' tiles have their rows from the plan, one after the other in
    // one list: those of an expert are neighbours.
    __device__ __forceinline__ Tile at(const GemmArgs& a, uint32_t id) const {
        const uint32_t nt = count(), xcd = id % kXcds, q = nt / kXcds, rem = nt % kXcds;
        const uint32_t lid = xcd * q + (xcd < rem ? xcd : rem) + id / kXcds;
        const uint32_t band = lid / (kXcds * cols), in = lid - band * (kXcds * cols);
        const uint32_t high = rows - band * kXcds < kXcds ? rows - band * kXcds : kXcds;
        const uint32_t m = band * kXcds + in % high;
        Tile t;
        t.n0 = (int64_t)(in / high) * BN;
        if constexpr (kExperts) {
            const int32_t expert_count = plan_number(a.tiles + 4 + 2 * m + 1);
            t.m0 = plan_number(a.tiles + 4 + 2 * m);
            t.expert = expert_count & 0xFFFF;
            t.count = expert_count >> 16;
        } else {
            t.m0 = (int64_t)m * BM;
            t.expert = 0;
            t.count = (int32_t)(a.M - t.m0 < BM ? a.M - t.m0 : BM);
        }
        return t;
    }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p, int64_t bytes) {
    const uint32_t n = (uint32_t)(bytes < 0xFFFF0000ll ? bytes : 0xFFFF0000ll);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), (short)0, (int)n, 0x00020000);
}

// Row i of a tile (clamped to its last one): its slot (dense: itself).
template <Mode MODE>
__device__ __forceinline__ uint32_t slot_at(const GemmArgs& a, const Tile& t, int i) {
    i = min(i, t.count - 1);
    return MODE == kDense ? (uint32_t)i : (uint32_t)a.list[t.m0 + i];
}

// Where the rows of a tile's operands are.  Rows of X and of W (clamped to the last one there is) as rows of their buffers.
template <Mode MODE>
struct Operands {
    __amdgpu_buffer_rsrc_t xc, xs, wc, ws;
    int32_t w_rows;            // of a kind, from n0 on
    int32_t up;                // rows from a gate row to its up row
    uint32_t per_token;

    __device__ __forceinline__ Operands(const GemmArgs& a, const Tile& t) {
        per_token = a.per_token;
        up = (int32_t)a.N;
        const int64_t left = a.N - t.n0;
        w_rows = (int32_t)(left < 1024 ? left : 1024);
        const uint8_t *cx = a.x.codes, *sx = a.x.scales;
        int64_t xr = a.x.rows;
        if constexpr (MODE == kDense) {
            cx += t.m0 * a.x.code_stride;
            sx += t.m0 * a.x.scale_stride;
            xr = t.count;
        }
        xc = buffer(cx, xr * a.x.code_stride);
        xs = buffer(sx, xr * a.x.scale_stride);
        const int64_t row0 = (MODE == kDense ? 0 : t.expert * a.w_rows) + t.n0;
        const int64_t rows = MODE == kUp ? a.w_rows - t.n0 : w_rows;
        wc = buffer(a.w.codes + row0 * a.w.code_stride, rows * a.w.code_stride);
        ws = buffer(a.w.scales + row0 * a.w.scale_stride, rows * a.w.scale_stride);
    }
    // the row of X of a slot
    __device__ __forceinline__ uint32_t row_of(uint32_t slot) const {
        return MODE == kUp && per_token ? __umulhi(slot, per_token) : slot;
    }
    // column c of the tile, of the gate or the up rows
    __device__ __forceinline__ uint32_t w_row(int c, bool second) const {
        c = min(c, w_rows - 1);
        return (uint32_t)(MODE == kUp && second ? c + up : c);
    }
};

__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)dst, 16, (int)voff, (int)soff, 0, 0);
}
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)dst, 4, (int)voff, (int)soff, 0, 0);
}

// f(0), f(1), ... f(N - 1), each with its number as a constant (a loop this long is not unrolled).
template <class F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
    each_of(f, std::make_integer_sequence<int, N>{});
}

// Slot of a 16-byte piece in its row of 128 bytes, and the piece in a slot.  The pieces of one instruction, 2 h + s, come to
// lie in neighbouring slots, turned by the row: 4.1 cycles a 16-byte read of a wave; the pieces in their own order take 5.8.
__device__ __forceinline__ int slot_of(int row, int piece) { return ((piece >> 1) | ((piece & 1) << 2)) ^ ((row >> 1) & 7); }
__device__ __forceinline__ int piece_in(int row, int slot) {
    const int t = slot ^ ((row >> 1) & 7);
    return ((t & 3) << 1) | (t >> 2);
}

// The last line of a row, in LDS: groups past the end of scale 1, codes past the end 0 (X).  valid: inputs of the line.
__device__ __forceinline__ void end_scales(uint8_t* s, int valid) {
    const int groups = (valid + kGroup - 1) / kGroup;
#pragma unroll
    for (int b = 0; b < 8; ++b)
        if (b >= groups) s[b] = 127;
}
__device__ __forceinline__ void end_codes(uint8_t* line, int row, int valid) {
    for (int p = valid / kGroup; p < 8; ++p) {
        v4i_t* at = reinterpret_cast<v4i_t*>(line + 16 * slot_of(row, p));
        v4i_t v = *at;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int left = valid - kGroup * p - 8 * d;             // codes of this dword that count
            v[d] = left >= 8 ? v[d] : left <= 0 ? 0 : (int)((uint32_t)v[d] & ((1u << (4 * left)) - 1u));
        }
        *at = v;
    }
}

__device__ __forceinline__ v8i_t wide(v4i_t v) { return (v8i_t){v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

template <int S>
__device__ __forceinline__ floatx4_t mfma(v4i_t w, int ws, v4i_t x, int xs, floatx4_t c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(w), wide(x), c, 4, 4, S, ws, S, xs);
}

// The same in place.  The compiler's own form may write its sum elsewhere, and with 256 of them there is no elsewhere: it
// then moves sums about between the instructions.  What reads the sums has to wait for the last instruction by itself
// (settle).  A vector instruction that writes an operand has to be two instructions away, which the compiler does not see to
// here: operands are whole dwords as they come from LDS, whose waits the compiler sets for any reader (of a 16-bit read it
// clears the upper half first; two idle cycles before every product would cost 5%).  That nothing stands too close in the code
// that comes of it is checked in the built library (tests/test_mfma_operands.py).
template <int S>
__device__ __forceinline__ void mfma_in_place(floatx4_t& c, v4i_t w, int ws, v4i_t x, int xs) {
#define QK_MFMA(SEL, SEL_HI)                                                                                                 \
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:" SEL " op_sel_hi:" SEL_HI          \
                 " cbsz:4 blgp:4"                                                                                            \
                 : "+a"(c) : "v"(w), "v"(x), "v"(ws), "v"(xs))
    if constexpr (S == 0) QK_MFMA("[0,0,0]", "[0,0,0]");
    else if constexpr (S == 1) QK_MFMA("[1,1,0]", "[0,0,0]");
    else if constexpr (S == 2) QK_MFMA("[0,0,0]", "[1,1,0]");
    else QK_MFMA("[1,1,0]", "[1,1,0]");
#undef QK_MFMA
}
// 32 idle cycles, more than an instruction of 8 passes needs before its result may be read; the sums count as written behind them.
template <int MT, int RT>
__device__ __forceinline__ void settle(floatx4_t (&acc)[MT][RT]) {
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) asm volatile("" : "+a"(acc[i][j]));
}

// N consecutive outputs (4 or 8), those of them below `left`.
template <int DT, int N>
__device__ __forceinline__ void store_row(void* y, int64_t at, const float (&v)[N], int64_t left) {
    if constexpr (DT == QK_F32) {
        float* p = static_cast<float*>(y) + at;
        if (left >= N) {
            __builtin_memcpy(p, v, 4 * N);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < left) p[i] = v[i];
        }
    } else {
        typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
        uint32_t d[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            d[i] = DT == QK_BF16 ? pack_bf16x2(v[2 * i], v[2 * i + 1])
                                 : __builtin_bit_cast(uint32_t, (f16x2_t){(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
        uint16_t* p = static_cast<uint16_t*>(y) + at;
        if (left >= N) {
            __builtin_memcpy(p, d, 2 * N);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < left) p[i] = (uint16_t)(d[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// g / (1 + exp(-g)) by e = exp(-|g|) <= 1.  For outputs of 16 bits: e to |g| 2^-24 of itself, the rounding of its exponent, 2^-17
// where it matters.  For fp32 to a few of its steps: the exponent of 2 in two parts, a reciprocal improved once; e is 0 from
// |g| = 104 on, and the parts of a larger one would pass the largest number.  (The library's exponential and a full division
// took a third of a tile's time.)
template <int DT>
__device__ __forceinline__ float silu(float g) {
    const float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;
    const float a = DT == QK_F32 ? fmaxf(-fabsf(g), -256.0f) : -fabsf(g), t = a * kLog2e, p = __builtin_amdgcn_exp2f(t);
    if constexpr (DT != QK_F32) return g * (g >= 0.0f ? 1.0f : p) * __builtin_amdgcn_rcpf(1.0f + p);
    const float low = fmaf(a, kLog2eLow, fmaf(a, kLog2e, -t));
    const float e = fmaf(p, low * kLn2, p), d = 1.0f + e;
    const float r = __builtin_amdgcn_rcpf(d), q = fmaf(fmaf(-d, r, 1.0f), r, r);
    return g * (g >= 0.0f ? q : e * q);
}

// Which of a wave's columns line q of its W lines is.  Of every two neighbouring blocks of 16 the lines alternate by fours,
// so that a lane's 4 outputs of the one and 4 of the other are neighbours: 8 of a row.
// (A wave with one block of gate and one of up rows keeps them apart.)
template <Mode MODE, int RT>
__device__ __forceinline__ int column_of(int q) {
    if constexpr (MODE == kUp && RT == 2) return q;
    return (q & ~31) | ((q >> 2 & 3) << 3) | ((q >> 4 & 1) << 2) | (q & 3);
}

// Outputs of one wave: acc[i][j], rows 16 i + lane % 16 of the wave's rows m, columns 4 (lane / 16) + q of block j of its n (up:
// the second half of the blocks are the up products of the first).  slots, weights: of the tile's rows.
template <Mode MODE, int DT, bool kWhole, int MT, int RT>
__device__ __forceinline__ void store_outputs(const GemmArgs& a, const Tile& t, const int32_t* slots, const float* weights, int m,
                                              int n, const floatx4_t (&acc)[MT][RT]) {
    const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
    constexpr int kCols = MODE == kUp ? RT / 2 : RT, kPair = kCols % 2 == 0 ? 2 : 1, kN = 4 * kPair;
    const int64_t col0 = t.n0 + n + kN * h;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int pos = m + 16 * i + r;
        if (!kWhole && pos >= t.count) continue;
        int64_t row;
        float wt = 1.0f;
        if constexpr (MODE == kDense) {
            row = t.m0 + pos;
        } else {
            row = slots[pos];
            if constexpr (MODE == kDown) wt = weights[pos];
        }
#pragma unroll
        for (int j = 0; j < kCols; j += kPair) {
            const int64_t col = col0 + 16 * j;
            if (!kWhole && col >= a.N) continue;
            float v[kN];
#pragma unroll
            for (int q = 0; q < kN; ++q) {
                const int b = j + q / 4;
                v[q] = acc[i][b][q % 4];
                if constexpr (MODE == kUp) v[q] = silu<DT>(v[q]) * acc[i][b + RT / 2][q % 4];
                if constexpr (MODE == kDown) v[q] *= wt;
            }
            store_row<DT, kN>(a.y, row * a.N + col, v, kWhole ? kN : a.N - col);
        }
    }
}

template <Mode MODE, int MT, int RT>
__device__ __forceinline__ void store_wave(const GemmArgs& a, const Tile& t, const int32_t* slots, const float* weights, int m, int n,
                                           const floatx4_t (&acc)[MT][RT]) {
    const bool whole = m + 16 * MT <= t.count && t.n0 + n + 16 * (MODE == kUp ? RT / 2 : RT) <= a.N;
    auto typed = [&](auto Whole) {
        constexpr bool w = decltype(Whole)::value;
        if (MODE == kDown || a.y_dtype == QK_F32) store_outputs<MODE, QK_F32, w>(a, t, slots, weights, m, n, acc);
        else if (a.y_dtype == QK_BF16) store_outputs<MODE, QK_BF16, w>(a, t, slots, weights, m, n, acc);
        else store_outputs<MODE, QK_F16, w>(a, t, slots, weights, m, n, acc);
    };
    if (whole) typed(std::true_type{});
    else typed(std::false_type{});
}

// ---------------------------------------------------------------------------
// Many rows: tiles of BM x BN, waves of WM x WN, two stages of LDS.  Up: columns [0, WN / 2) of a wave are gate rows,
// the others their up rows.
//
// A stage is two halves of WM / 16 x WN / 16 instructions.  While a half is multiplied, row of fragments by row, the X
// fragments of the row after next and the W fragments of the next half are read from LDS, in the order written here (the
// scheduling barriers keep it).  Between the halves, when the W lines of the stage have been read, all waves meet, and the W
// lines of the stage after next start on their way to the same place; two rows before the stage ends they meet again: the
// next stage has landed, and the X lines of the stage after next follow.
//
// Copies of W set out a stage and a half before they are read, those of X one stage, in a ring of three stages (kRing) one
// stage earlier.
//
// A workgroup makes one tile after the other (kTurns; a launch has as many as are on the CUs at a time): while a tile is
// multiplied the slots of the next one's rows come from the plan, and its first copies are on their way while outputs are
// stored.  4096 tokens of 64 experts, up: 126 us where every tile has a workgroup of its own, 111 so.  Not in the largest tiles, whose
// sums leave no registers for it.
// ---------------------------------------------------------------------------
constexpr bool takes_turns(int BM, int BN) { return BM * BN < 256 * 256; }

template <Mode MODE, int BM, int BN, int WM, int WN, int kRing>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void mx4_tile_kernel(GemmArgs a) {
    constexpr int kWaves = (BM / WM) * (BN / WN), kThreads = kWaves * 64;
    constexpr int MT = WM / 16, RT = WN / 16;
    static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 && BM % 64 == 0 && BN % 64 == 0);
    constexpr int kBNo = MODE == kUp ? BN / 2 : BN;
    constexpr bool kTurns = takes_turns(BM, BN);
    // codes of X and of W by the parity of the stage, 128 bytes a line (objects of their own: the compiler waits for copies on
    // their way to the object that it reads from); scales of two stages, 16 bytes a line, by the parity of the pair
    __shared__ __align__(16) uint8_t x0[BM * 128];
    __shared__ __align__(16) uint8_t w0[BN * 128];
    __shared__ __align__(16) uint8_t x1[BM * 128];
    __shared__ __align__(16) uint8_t w1[BN * 128];
    __shared__ __align__(16) uint8_t x2[kRing > 2 ? BM * 128 : 16];
    __shared__ __align__(16) uint8_t w2[kRing > 2 ? BN * 128 : 16];
    __shared__ __align__(16) uint8_t sc[2 * (BM + BN) * 16];
    // slots of the tile's rows and their weights, by the parity of the tile
    __shared__ int32_t slots[MODE == kDense ? 1 : 2 * BM];
    __shared__ float weights[MODE == kDown ? 2 * BM : 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / (BN / WN), wn = wave % (BN / WN);
    const int r = lane & 15, h = lane >> 4;
    const Tiling<MODE != kDense, BM, kBNo> tiling(a);
    uint32_t id = blockIdx.x;
    if (id >= tiling.count()) return;
    Tile t = tiling.at(a, id);
    const int nst = (a.x.cols + kLineK - 1) / kLineK;
    const int valid = a.x.cols - (nst - 1) * kLineK;                  // inputs of the last line
    Operands<MODE> op(a, t);
    auto w_row = [&](int b) {                           // row b of the tile's W lines
        const int q = column_of<MODE, RT>(b % WN);
        return MODE == kUp ? op.w_row(b / WN * (WN / 2) + q % (WN / 2), q >= WN / 2) : op.w_row(b / WN * WN + q, false);
    };
    // what this lane copies: line l / 8 of 8, slot l % 8; and the lines whose scales it loads
    constexpr int kXCopies = BM / 8 / kWaves, kWCopies = BN / 8 / kWaves, kSLoads = (BM + BN + kThreads - 1) / kThreads;
    uint32_t xslot[kXCopies], sslot[kSLoads], xoff[kXCopies], woff[kWCopies], soff[kSLoads];
    auto look_up = [&](const Tile& u) {
#pragma unroll
        for (int k = 0; k < kXCopies; ++k) xslot[k] = slot_at<MODE>(a, u, 8 * (wave + kWaves * k) + (lane >> 3));
#pragma unroll
        for (int k = 0; k < kSLoads; ++k)
            if (64 * wave + kThreads * k < BM) sslot[k] = slot_at<MODE>(a, u, tid + kThreads * k);
    };
    // Copy k of stage st, which is line `line`; past the last stage every offset is outside its buffer, and zeros are written.
    auto copy_x = [&](uint8_t* dst, int st, int line, int k) {
        to_lds(op.xc, dst + (wave + kWaves * k) * 1024, xoff[k] | (st < nst ? 0u : 0xFFFF0000u), st < nst ? 128u * line : 0u);
    };
    auto copy_w = [&](uint8_t* dst, int st, int line, int k) {
        to_lds(op.wc, dst + (wave + kWaves * k) * 1024, woff[k] | (st < nst ? 0u : 0xFFFF0000u), st < nst ? 128u * line : 0u);
    };
    // Scales come 16 bytes a line at a time, those of two stages, through registers: a line of memory that is brought for
    // 8 of its bytes costs as much as one of codes.  In LDS dword h of a line holds groups 2 h and 2 h + 1 of the first stage,
    // then of the second: what a lane needs.
    u32x4_t sv[kSLoads], sl[kSLoads];
    auto scale_load = [&](int k, uint32_t at) {
        const bool x = 64 * wave + kThreads * k < BM;
        return __builtin_amdgcn_raw_buffer_load_b128(x ? op.xs : op.ws, (int)soff[k], (int)at, 0);
    };
    auto scale_store = [&](int pair, int k) {
        if (64 * wave + kThreads * k >= BM + BN) return;
        const u32x4_t v = sv[k];
        *reinterpret_cast<u32x4_t*>(sc + (pair & 1) * ((BM + BN) * 16) + (tid + kThreads * k) * 16) =
            (u32x4_t){__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                      __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
    };
    const int xline = (wm * WM + r) * 128, wline = (wn * WN + r) * 128;
    const int xsc = (wm * WM + r) * 16 + 4 * h, wsc = (BM + wn * WN + r) * 16 + 4 * h;
    const int at0 = 16 * slot_of(r, 2 * h), at1 = 16 * slot_of(r, 2 * h + 1);
    // fragments of W by half; those of X, of which four are enough; scales by the parity of the stage
    v4i_t wf[2][RT], xf[4];
    int ws[2][RT], xs[2][MT];
    auto read_x = [&](const uint8_t* src, int s, int i) {
        xf[i % 4] = *reinterpret_cast<const v4i_t*>(src + xline + (s ? at1 : at0) + 2048 * i);
    };
    auto read_w = [&](const uint8_t* src, int s, int j) {
        wf[s][j] = *reinterpret_cast<const v4i_t*>(src + wline + (s ? at1 : at0) + 2048 * j);
    };
    auto read_scale = [&](int st, int p, int n) {
        const uint8_t* src = sc + (st >> 1 & 1) * ((BM + BN) * 16);
        if (n < RT) ws[p][n] = *reinterpret_cast<const int*>(src + wsc + 256 * n);
        else xs[p][n - RT] = *reinterpret_cast<const int*>(src + xsc + 256 * (n - RT));
    };
    static_assert(MT % 4 == 0);
    constexpr int kOps = MT * RT, kTail = 2 * RT;                 // instructions of a half; of it behind the meeting
    // Items 0..n-1 spread over instructions [from, to): those behind instruction o.
    auto spread = [](auto O, auto From, auto To, auto N, auto&& item) {
        constexpr int o = decltype(O)::value - decltype(From)::value, ops = decltype(To)::value - decltype(From)::value;
        constexpr int n = decltype(N)::value;
        static_assert(ops > 0);
        if constexpr (o >= 0 && o < ops) {
            constexpr int k0 = (o * n + ops - 1) / ops, k1 = ((o + 1) * n + ops - 1) / ops;
            each<k1 - k0>([&](auto K) { item(k0 + decltype(K)::value); });
        }
    };
    // Waves meet once all but the last `flying` copies of each have landed and its reads are done.
    auto meet = [&](auto Flying) {
        constexpr int n = decltype(Flying)::value;
        __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | 0x70);   // vmcnt(n) expcnt(7) lgkmcnt(0)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int kXEarly = kXCopies / 4;                             // of the copies of X before the next stage begins
    typedef std::integral_constant<int, kXEarly> XEarly;
    typedef std::integral_constant<int, kWCopies> WCopies;
    // copies that are sent off later than those of the next stage: W's of the last one to come, in a ring of three all of the one before
    typedef std::integral_constant<int, kWCopies + (kRing - 2) * (kWCopies + kXCopies)> Flying;
    // Sends the first copies of tile u on their way (the last line, which may end early, comes first), from what look_up found.
    auto begin = [&](const Tile& u, int parity) {
        if constexpr (MODE != kDense) {
#pragma unroll
            for (int k = 0; k < kSLoads; ++k) {
                const int line = tid + kThreads * k;
                if (64 * wave + kThreads * k >= BM) continue;
                slots[parity * BM + line] = (int32_t)sslot[k];
                if constexpr (MODE == kDown) weights[parity * BM + line] = u.expert < a.E ? a.weights[sslot[k]] : 0.0f;
            }
            if (u.expert >= a.E) return;
        }
        op = Operands<MODE>(a, u);
#pragma unroll
        for (int k = 0; k < kWCopies; ++k) {
            const int line = 8 * (wave + kWaves * k) + (lane >> 3);
            woff[k] = w_row(line) * (uint32_t)a.w.code_stride + 16 * piece_in(line, lane & 7);
        }
#pragma unroll
        for (int k = 0; k < kXCopies; ++k) {
            const int line = 8 * (wave + kWaves * k) + (lane >> 3);
            xoff[k] = op.row_of(xslot[k]) * (uint32_t)a.x.code_stride + 16 * piece_in(line, lane & 7);
        }
#pragma unroll
        for (int k = 0; k < kSLoads; ++k)
            soff[k] = 64 * wave + kThreads * k < BM ? op.row_of(sslot[k]) * (uint32_t)a.x.scale_stride
                                                    : w_row(min(tid + kThreads * k - BM, BN - 1)) * (uint32_t)a.w.scale_stride;
#pragma unroll
        for (int k = 0; k < kWCopies; ++k) copy_w(w0, 0, nst - 1, k);
#pragma unroll
        for (int k = 0; k < kXCopies; ++k) copy_x(x0, 0, nst - 1, k);
#pragma unroll
        for (int k = 0; k < kSLoads; ++k) {
            sl[k] = scale_load(k, 8u * (nst - 1));
            sv[k] = scale_load(k, 0);
        }
#pragma unroll
        for (int k = 0; k < kWCopies; ++k) copy_w(w1, 1, 0, k);
        if constexpr (kRing > 2) {
#pragma unroll
            for (int k = 0; k < kXCopies; ++k) copy_x(x1, 1, 0, k);
#pragma unroll
            for (int k = 0; k < kWCopies; ++k) copy_w(w2, 2, 1, k);
        }
#pragma unroll
        for (int k = 0; k < kXEarly; ++k) copy_x(kRing > 2 ? x2 : x1, kRing - 1, kRing - 2, k);
    };
    look_up(t);
    begin(t, 0);
    for (int parity = 0;; parity ^= 1) {
        const bool live = MODE == kDense || t.expert < a.E, more = kTurns && id + gridDim.x < tiling.count();
        Tile next = t;
        if (more) next = tiling.at(a, id + gridDim.x);
        floatx4_t acc[MT][RT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[i][j] = (floatx4_t){0, 0, 0, 0};
        if (live) {
            auto stage = [&](auto P, uint8_t* x, uint8_t* w, uint8_t* xnext, uint8_t* wnext, uint8_t* xlast, int st) {
                constexpr int p = decltype(P)::value;
                each<2>([&](auto S) {
                    constexpr int s = decltype(S)::value;
                    each<kOps>([&](auto O) {
                        constexpr int o = decltype(O)::value, i = o / RT, j = o % RT;
                        if constexpr (s == 1 && o == 0) meet(std::integral_constant<int, 63>{});
                        if constexpr (s == 1 && o == kOps - kTail) meet(Flying{});
                        mfma_in_place<2 * p + s>(acc[i][j], wf[s][j], ws[p][j], xf[i % 4], xs[p][i]);
                        if constexpr (j == 0) {
                            if constexpr (i + 2 < MT) read_x(x, s, i + 2);
                            else read_x(s == 0 ? x : xnext, 1 - s, i + 2 - MT);
                        }
                        typedef std::integral_constant<int, 0> Begin;
                        typedef std::integral_constant<int, kOps - kTail> Meeting;
                        typedef std::integral_constant<int, kOps> End;
                        if constexpr (s == 0) {
                            spread(O, Begin{}, std::integral_constant<int, kOps / 2>{}, std::integral_constant<int, kXCopies - kXEarly>{},
                                   [&](int k) { copy_x(xlast, st + kRing - 1, st + kRing - 2, kXEarly + k); });
                            // (p == 0: scales of stages st + 2 and st + 3)
                            if constexpr (p == 0)
                                spread(O, std::integral_constant<int, kOps / 2>{}, End{}, std::integral_constant<int, kSLoads>{},
                                       [&](int k) { sv[k] = scale_load(k, 8u * (st + 1)); });
                            spread(O, Begin{}, Meeting{}, std::integral_constant<int, RT>{}, [&](int k) { read_w(w, 1, k); });
                        } else {
                            if constexpr (p == 1)
                                spread(O, Begin{}, Meeting{}, std::integral_constant<int, kSLoads>{}, [&](int k) {
                                    // the second of the pair may be past the end: its codes are zeros, but not its scales
                                    if (st + 2 >= nst) sv[k][2] = sv[k][3] = 0;
                                    scale_store((st + 1) >> 1, k);
                                });
                            spread(O, Begin{}, Meeting{}, WCopies{}, [&](int k) { copy_w(w, st + kRing, st + kRing - 1, k); });
                            spread(O, Meeting{}, End{}, std::integral_constant<int, RT>{}, [&](int k) { read_w(wnext, 0, k); });
                            spread(O, Meeting{}, End{}, std::integral_constant<int, RT + MT>{}, [&](int k) { read_scale(st + 1, 1 - p, k); });
                            spread(O, Meeting{}, End{}, XEarly{}, [&](int k) { copy_x(x, st + kRing, st + kRing - 1, k); });
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    });
                });
            };
            // scales of the first pair: the last line's, 1 past the end, then those of line 0
#pragma unroll
            for (int k = 0; k < kSLoads; ++k) {
                const int groups = (valid + kGroup - 1) / kGroup;
                const u32x4_t first = sv[k];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const int n = groups - 4 * d;
                    const uint32_t keep = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
                    sv[k][d] = (sl[k][d] & keep) | (0x7F7F7F7Fu & ~keep);
                    sv[k][2 + d] = nst > 1 ? first[d] : 0u;
                }
                scale_store(0, k);
            }
            meet(std::integral_constant<int, kWCopies + kXEarly + (kRing - 2) * (kWCopies + kXCopies)>{});
            if (more) look_up(next);
            if (valid < kLineK) {
                for (int l = tid; l < BM; l += kThreads) end_codes(x0 + 128 * l, l, valid);
                __syncthreads();
            }
#pragma unroll
            for (int j = 0; j < RT; ++j) read_w(w0, 0, j);
#pragma unroll
            for (int i = 0; i < 2; ++i) read_x(x0, 0, i);
#pragma unroll
            for (int k = 0; k < RT + MT; ++k) read_scale(0, 0, k);
            // (an odd number of stages is one more of zeros: a way out between the two costs the compiler the registers.  A way
            // past the loop would have it move sums to where the zeros of that way are, before they have settled.)
            const std::integral_constant<int, 0> even;
            const std::integral_constant<int, 1> odd;
            int st = 0;
            if constexpr (kRing == 2) {
                do {
                    stage(even, x0, w0, x1, w1, x1, st);
                    stage(odd, x1, w1, x0, w0, x0, st + 1);
                } while ((st += 2) < nst);
            } else {
                do {
                    stage(even, x0, w0, x1, w1, x2, st);
                    stage(odd, x1, w1, x2, w2, x0, st + 1);
                    if (st + 2 < nst) {
                        stage(even, x2, w2, x0, w0, x1, st + 2);
                        stage(odd, x0, w0, x1, w1, x2, st + 3);
                    }
                    if (st + 4 < nst) {
                        stage(even, x1, w1, x2, w2, x0, st + 4);
                        stage(odd, x2, w2, x0, w0, x1, st + 5);
                    }
                } while ((st += 6) < nst);
            }
            __builtin_amdgcn_s_waitcnt(0);                            // nothing on its way to LDS any more
            settle<MT, RT>(acc);
        } else if (more) {
            look_up(next);
        }
        if (more || !live) __syncthreads();                           // every wave is done with LDS; slots are there
        if (more) begin(next, parity ^ 1);
        store_wave<MODE>(a, t, slots + parity * BM, weights + parity * BM, wm * WM, MODE == kUp ? wn * (WN / 2) : wn * WN, acc);
        if (!more) return;
        t = next;
        id += gridDim.x;
    }
}

// ---------------------------------------------------------------------------
// Few rows: a workgroup makes 16 MT rows x 16 RT lines of W, its waves take every kWaves-th line of inputs and their sums
// meet in LDS, added in wave order.  A wave has three stages of its own and waits for nobody in the loop.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 4;

template <Mode MODE, int MT, int RT>
__global__ __launch_bounds__(kFewWaves * 64) void mx4_few_kernel(GemmArgs a) {
    constexpr int kLines = 16 * (MT + RT);
    constexpr int kStage = kLines * 128 + (kLines + 31) / 32 * 256;
    constexpr int kLoads = 2 * (MT + RT), kSLoads = (kLines + 31) / 32;
    constexpr int kBNo = MODE == kUp ? 8 * RT : 16 * RT;
    constexpr int kSum = MT * RT * 1024;                // bytes of a wave's sums
    static_assert(kSum <= kStage);
    __shared__ __align__(16) uint8_t lds0[kFewWaves * kStage];
    __shared__ __align__(16) uint8_t lds1[kFewWaves * kStage];
    __shared__ __align__(16) uint8_t lds2[kFewWaves * kStage];
    __shared__ int32_t slots[MODE == kDense ? 1 : 16 * MT];
    __shared__ float weights[MODE == kDown ? 16 * MT : 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, h = lane >> 4;
    const Tiling<MODE != kDense, 16 * MT, kBNo> tiling(a);
    if (blockIdx.x >= tiling.count()) return;
    const Tile t = tiling.at(a, blockIdx.x);
    floatx4_t acc[MT][RT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = (floatx4_t){0, 0, 0, 0};

    if (MODE == kDense || t.expert < a.E) {
        const Operands<MODE> op(a, t);
        auto w_row = [&](int b) {
            const int q = column_of<MODE, RT>(b);
            return MODE == kUp ? op.w_row(q % (8 * RT), q >= 8 * RT) : op.w_row(q, false);
        };
        uint32_t voff[kLoads], soff[kSLoads];
#pragma unroll
        for (int v = 0; v < kLoads; ++v) {
            const int line = 8 * v + (lane >> 3), piece = piece_in(line, lane & 7);
            voff[v] = v < 2 * MT ? op.row_of(slot_at<MODE>(a, t, line)) * (uint32_t)a.x.code_stride + 16 * piece
                                 : w_row(line - 16 * MT) * (uint32_t)a.w.code_stride + 16 * piece;
        }
        // scales: 32 lines an instruction, or two with half the lanes each where the first 16 are of X
#pragma unroll
        for (int v = 0; v < kSLoads; ++v) {
            const int line = 32 * v + (lane >> 1);
            soff[v] = 4 * (lane & 1) + (line < 16 * MT ? op.row_of(slot_at<MODE>(a, t, line)) * (uint32_t)a.x.scale_stride
                                                       : w_row(line - 16 * MT) * (uint32_t)a.w.scale_stride);
        }
        const int nst = (a.x.cols + kLineK - 1) / kLineK;
        auto load = [&](uint8_t* ring, int st) {
            uint8_t* dst = ring + wave * kStage;
            // past the row every offset is outside its buffer, and nothing is read (loads under a condition would leave the
            // waits below without a count)
            const uint32_t out = st < nst ? 0u : 0xFFFF0000u, c = st < nst ? 128u * st : 0u, s = st < nst ? 8u * st : 0u;
#pragma unroll
            for (int v = 0; v < kLoads; ++v) to_lds(v < 2 * MT ? op.xc : op.wc, dst + v * 1024, voff[v] | out, c);
#pragma unroll
            for (int v = 0; v < kSLoads; ++v) {
                const int first = 32 * v;                             // lines of X come first, 16 MT of them
                uint8_t* to = dst + kLines * 128 + v * 256;
                if (first + 32 <= 16 * MT) to_lds4(op.xs, to, soff[v] | out, s);
                else if (first >= 16 * MT) to_lds4(op.ws, to, soff[v] | out, s);
                else if (lane < 32) to_lds4(op.xs, to, soff[v] | out, s);
                else to_lds4(op.ws, to, soff[v] | out, s);
            }
        };
        auto compute = [&](const uint8_t* ring) {
            const uint8_t* src = ring + wave * kStage;
            int xs[MT], ws[RT];
#pragma unroll
            for (int i = 0; i < MT; ++i) xs[i] = *reinterpret_cast<const uint16_t*>(src + kLines * 128 + (16 * i + r) * 8 + 2 * h);
#pragma unroll
            for (int j = 0; j < RT; ++j) ws[j] = *reinterpret_cast<const uint16_t*>(src + kLines * 128 + (16 * (MT + j) + r) * 8 + 2 * h);
            auto half = [&](auto S) {
                constexpr int s = decltype(S)::value;
                const int at = r * 128 + 16 * slot_of(r, 2 * h + s);
                v4i_t x[MT], w[RT];
#pragma unroll
                for (int i = 0; i < MT; ++i) x[i] = *reinterpret_cast<const v4i_t*>(src + at + 2048 * i);
#pragma unroll
                for (int j = 0; j < RT; ++j) w[j] = *reinterpret_cast<const v4i_t*>(src + at + 2048 * (MT + j));
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < RT; ++j) acc[i][j] = mfma<s>(w[j], ws[j], x[i], xs[i], acc[i][j]);
            };
            half(std::integral_constant<int, 0>{});
            half(std::integral_constant<int, 1>{});
        };
        const int valid = a.x.cols - (nst - 1) * kLineK;
        // the last line of a row, by the wave that has it
        auto finish = [&](uint8_t* ring) {
            uint8_t* dst = ring + wave * kStage;
            for (int l = lane; l < kLines; l += 64) {
                end_scales(dst + kLines * 128 + 8 * l, valid);
                if (l < 16 * MT) end_codes(dst + 128 * l, l, valid);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        load(lds0, wave);
        load(lds1, wave + kFewWaves);
        auto step = [&](uint8_t* cur, uint8_t* next, int st) {
            load(next, st + 2 * kFewWaves);
            constexpr int kInFlight = 2 * (kLoads + kSLoads + (MT & 1));   // stages st + 1, st + 2
            __builtin_amdgcn_s_waitcnt((kInFlight & 15) | ((kInFlight >> 4) << 14) | 0x0F70);
            asm volatile("" ::: "memory");
            if (st == nst - 1 && valid < kLineK) finish(cur);
            compute(cur);
        };
        int st = wave;
        for (; st + 2 * kFewWaves < nst; st += 3 * kFewWaves) {
            step(lds0, lds2, st);
            step(lds1, lds0, st + kFewWaves);
            step(lds2, lds1, st + 2 * kFewWaves);
        }
        if (st < nst) step(lds0, lds2, st);
        if (st + kFewWaves < nst) step(lds1, lds0, st + kFewWaves);
        __builtin_amdgcn_s_waitcnt(0);                                // nothing on its way to LDS any more
        __syncthreads();
        // wave w adds up and stores columns w, w + kFewWaves, ... of the 16 x 16 blocks
        float* sums = reinterpret_cast<float*>(lds0);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j)
                *reinterpret_cast<floatx4_t*>(sums + wave * (kSum / 4) + ((i * RT + j) * 64 + lane) * 4) = acc[i][j];
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j) {
#pragma unroll
                for (int o = 1; o < kFewWaves; ++o)
                    acc[i][j] += *reinterpret_cast<const floatx4_t*>(sums + o * (kSum / 4) + ((i * RT + j) * 64 + lane) * 4);
            }
    }
    if (wave > 0) return;
    if constexpr (MODE != kDense) {
        if (lane < 16 * MT) {
            const uint32_t slot = slot_at<MODE>(a, t, lane);
            slots[lane] = (int32_t)slot;
            if constexpr (MODE == kDown) weights[lane] = t.expert < a.E ? a.weights[slot] : 0.0f;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    store_wave<MODE>(a, t, slots, weights, 0, 0, acc);
}

// ---------------------------------------------------------------------------
// The parts of each token's slots added in order.
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 256;

__global__ __launch_bounds__(kCombineThreads) void moe_combine_mx4_kernel(const float* __restrict__ part, void* y, int32_t dtype,
                                                                          int64_t T, int32_t top_k, int64_t H) {
    const int64_t quads = (H + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x;
    const int64_t tok = i / quads, col = (i - tok * quads) * 4;
    if (tok >= T) return;
    const int64_t left = H - col;
    floatx4_t sum = {0, 0, 0, 0};
    for (int32_t j = 0; j < top_k; ++j) {
        const float* p = part + (tok * top_k + j) * H + col;
        floatx4_t v = {0, 0, 0, 0};
        if (left >= 4) {
            __builtin_memcpy(&v, p, 16);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < left) v[q] = p[q];
        }
        sum += v;
    }
    const float out[4] = {sum[0], sum[1], sum[2], sum[3]};
    if (dtype == QK_F32) store_row<QK_F32, 4>(y, tok * H + col, out, left);
    else if (dtype == QK_BF16) store_row<QK_BF16, 4>(y, tok * H + col, out, left);
    else store_row<QK_F16, 4>(y, tok * H + col, out, left);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups of a launch of BM x BNo tiles.
template <Mode MODE>
int64_t grid_for(const GemmArgs& a, int64_t bm, int64_t bno) {
    if (MODE == kDense) return cdiv(a.M, bm) * cdiv(a.N, bno);
    // an expert's last tile may be partial
    return moe_most_tiles(a.slots, a.E) * cdiv(a.N, bno);
}

template <Mode MODE, int BM, int BN, int WM, int WN, int kRing>
hipError_t launch_tile(const GemmArgs& a, hipStream_t s) {
    const int64_t tiles = grid_for<MODE>(a, BM, MODE == kUp ? BN / 2 : BN);
    if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
    // workgroups that the LDS of the CUs holds
    constexpr int64_t kLds = (BM + BN) * (128 * kRing + 32) + (MODE == kDense ? 0 : MODE == kUp ? 8 : 16) * BM;
    const int64_t grid = std::min<int64_t>(tiles, takes_turns(BM, BN) ? device_cu_count() / kXcds * kXcds * (160 * 1024 / kLds) : tiles);
    mx4_tile_kernel<MODE, BM, BN, WM, WN, kRing><<<dim3((unsigned)grid), dim3((BM / WM) * (BN / WN) * 64), 0, s>>>(a);
    return hipGetLastError();
}

template <Mode MODE, int MT, int RT>
hipError_t launch_few(const GemmArgs& a, hipStream_t s) {
    const int64_t grid = grid_for<MODE>(a, 16 * MT, MODE == kUp ? 8 * RT : 16 * RT);
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    mx4_few_kernel<MODE, MT, RT><<<dim3((unsigned)grid), dim3(kFewWaves * 64), 0, s>>>(a);
    return hipGetLastError();
}

// Which tiles.  Times in us, weights in cache where they fit.
hipError_t launch_dense(const GemmArgs& a, hipStream_t s) {
    const int64_t cus = device_cu_count();
    // Workgroups that split the inputs among their waves where tiles would leave half of the CUs without one, and up to 16
    // rows always: 16 x 4096 x 11008 6.4, tiles of 64 x 64 16; 64 x 4096 x 4096 6.6 and 8.1; 64 x 11008 x 4096 12.1 and 8.6.
    // (A launch has fewer than 2^32 threads; tiles are made by as many workgroups as there is room for.)
    if (a.M <= 16 && a.N <= (int64_t)1 << 28) return launch_few<kDense, 1, 2>(a, s);
    if (a.M <= 128 && grid_for<kDense>(a, 64, 64) <= cus / 2)
        return a.M <= 32 ? launch_few<kDense, 2, 2>(a, s) : launch_few<kDense, 4, 2>(a, s);
    // The largest tiles where there is one for every CU: 4096 x 4096 x 4096 39.9, in tiles of 128 43.9; 2048 x 4096 x 4096 31.3 and
    // 24.0 (a bound of 3 / 4 of the CUs would do as well or better: 3000 x 4096 x 4096 33.8 and 34.4, 3800 37.8 and 42.6).  Two workgroups
    // a CU of tiles of 128 where there is more than one for each (1100 x 4096 x 4096 22.1, one workgroup and a ring of three stages
    // 25.2), one and a ring of three up to that (1000 13.7, of two 14.3), where tiles of 64 x 128 would be more than the CUs
    // (800 x 4096 x 4096 12.5, of 64 x 128 16.0; 560 11.6 and 17.8).  Below, those of 64 x 128 (512 x 4096 x 4096 10.6, of 128
    // 11.6, of 64 11.3) down to 5 / 8 of the CUs (300 x 4096 x 4096 9.4, of 64 10.6; 200 9.3 and 8.5), with a ring of three.
    if (grid_for<kDense>(a, 256, 256) >= cus) return launch_tile<kDense, 256, 256, 128, 128, 2>(a, s);
    if (grid_for<kDense>(a, 128, 128) > cus) return launch_tile<kDense, 128, 128, 64, 64, 2>(a, s);
    const int64_t tiles = grid_for<kDense>(a, 64, 128);
    if (tiles > cus) return launch_tile<kDense, 128, 128, 64, 64, 3>(a, s);
    if (tiles >= cus * 5 / 8) return launch_tile<kDense, 64, 128, 64, 32, 3>(a, s);
    return launch_tile<kDense, 64, 64, 64, 32, 3>(a, s);
}

template <Mode MODE>
hipError_t launch_experts(const GemmArgs& a, hipStream_t s) {
    const int64_t cus = device_cu_count(), half = MODE == kUp ? 2 : 1;
    if (moe_tile_rows(a.slots, a.E) == 128) {
        // Tiles of 128 x 256, a ring of three stages and one workgroup a CU, where there is about one for each CU (half of
        // an expert's last tile counted): top 2 of 8 experts of 4096 x 11008, down, 400 tokens (160 tiles) 58 us, in tiles of 128 x
        // 128 72; 512 (192) 60 and 69; 700 (224) 62 and 65; 800 (256, by then more than one) 106 and 100; 1000 (304) 105 and 97; 600
        // of 8 experts of 8192 inputs and 2048 outputs (104) 43 and 33.  And where there are so many that the last turn does not matter:
        // 8192 tokens down (2112) 594 and 616; 1400 up (2150) 208 and 239; 4096 tokens of 64 experts, up (2304), weights from memory 118
        // and 121, 8192 (4352) 214 and 220.  From 2 to 8 for each CU either is better, by what the last turn has left: 2600 down (704)
        // 204 and 223, 4096 down (1088) 317 and 307, 5000 (1312) 360 and 387; 2048 tokens of 64 experts, up (1280) 68 and 63.
        const int64_t experts = std::min<int64_t>(a.E, a.slots);
        const int64_t tiles = (a.slots / 128 + (experts + 1) / 2) * cdiv(a.N, 256 / half);
        if ((tiles > cus / 2 && tiles <= cus) || tiles > 8 * cus) return launch_tile<MODE, 128, 256, 64, 64, 3>(a, s);
        return launch_tile<MODE, 128, 128, 64, 64, 2>(a, s);
    }
    // A few slots of few outputs: the inputs split among the waves of a workgroup (one token's top 2 of 8 experts of
    // 4096 x 11008, down: 12.6, in tiles of 64 x 64 24, its up products, of more tiles than CUs, 22 and 17; two tokens' top 8 of
    // 64 of 2048 x 1024, down, 10.8 and 9.7).  Otherwise the larger tiles where they fill the CUs twice (200 tokens of the first,
    // up, 92, of 64 x 64 109; of the second, weights from memory, 38 and 40; 100 tokens of the first, down, once: 39 both).
    if (a.slots <= 16 && grid_for<MODE>(a, 64, 64 / half) <= cus) return launch_few<MODE, 1, 2>(a, s);
    if (grid_for<MODE>(a, 64, 128 / half) >= 2 * cus) return launch_tile<MODE, 64, 128, 64, 32, 2>(a, s);
    return launch_tile<MODE, 64, 64, 64, 32, 2>(a, s);
}

}  // namespace

hipError_t launch_mx4_gemm(const qk_mx4_state* x, const qk_mx4_state* w, void* y, int32_t y_dtype, hipStream_t s) {
    GemmArgs a{};
    a.x = view(x);
    a.w = view(w);
    a.y = y;
    a.y_dtype = y_dtype;
    a.M = x->rows;
    a.N = w->rows;
    a.w_rows = w->rows;
    return launch_dense(a, s);
}

namespace {
GemmArgs expert_args(const qk_mx4_state* x, const qk_mx4_state* w, const int32_t* plan, int32_t top_k, int32_t E) {
    GemmArgs a{};
    a.x = view(x);
    a.w = view(w);
    a.E = E;
    a.list = plan + moe_plan_list(E);
    a.per_token = top_k == 1 ? 0 : (uint32_t)(((1ull << 32) + top_k - 1) / top_k);
    a.w_rows = w->rows / E;
    return a;
}
}  // namespace

hipError_t launch_moe_up_mx4(const qk_mx4_state* x, const qk_mx4_state* gate_up, const int32_t* plan, int32_t top_k,
                             int32_t E, void* h, int32_t h_dtype, hipStream_t s) {
    GemmArgs a = expert_args(x, gate_up, plan, top_k, E);
    a.slots = (int32_t)(x->rows * top_k);
    a.tiles = plan + moe_plan_tiles(E, a.slots);
    a.y = h;
    a.y_dtype = h_dtype;
    a.N = a.w_rows / 2;
    return launch_experts<kUp>(a, s);
}

size_t moe_down_mx4_workspace_bytes(int64_t T, int32_t top_k, int64_t H) { return (size_t)(T * top_k) * (size_t)H * 4; }

hipError_t launch_moe_down_mx4(const qk_mx4_state* h, const qk_mx4_state* down, const int32_t* plan, const float* weights,
                               int32_t top_k, int32_t E, void* y, int32_t y_dtype, void* workspace, hipStream_t s) {
    GemmArgs a = expert_args(h, down, plan, top_k, E);
    a.slots = (int32_t)h->rows;
    a.tiles = plan + moe_plan_tiles(E, a.slots);
    a.y = workspace;
    a.weights = weights;
    a.N = a.w_rows;
    const hipError_t e = launch_experts<kDown>(a, s);
    if (e != hipSuccess) return e;
    // pieces of fewer than 2^32 threads
    const int64_t T = h->rows / top_k, quads = (a.N + 3) / 4, most = std::max<int64_t>(1, ((int64_t)1 << 30) / quads);
    for (int64_t t = 0; t < T; t += most) {
        const int64_t n = std::min(most, T - t);
        moe_combine_mx4_kernel<<<dim3((unsigned)cdiv(n * quads, kCombineThreads)), dim3(kCombineThreads), 0, s>>>(
            static_cast<const float*>(workspace) + t * top_k * a.N, static_cast<uint8_t*>(y) + t * a.N * (y_dtype == QK_F32 ? 4 : 2),
            y_dtype, n, top_k, a.N);
        const hipError_t c = hipGetLastError();
        if (c != hipSuccess) return c;
    }
    return hipSuccess;
}

}  // namespace qk
