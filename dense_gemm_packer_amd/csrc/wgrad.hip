// A weight's gradient (dgp_gemm_wgrad): for every group e of rows,
//
//   C[e][n][k] = sum over the rows m of e of Y[m][n] * x[rows ? rows[m] : m][k],
//
// Y the output's gradient in bf16 and x the forward product's operand A, bf16 or
// e4m3 codes with their scales.
//
// Both operands have the summed index as their slow one, where a matrix-core
// instruction wants it in a lane's consecutive elements.  The tile of each goes
// to LDS in blocks of 4 rows x 16 columns (128 bytes, row by row), and the
// transposing LDS read (ds_read_b64_tr_b16) hands lane i of 16 the four rows of
// column i: two of them are one operand fragment of the 16x16x32 instruction.
// The order of the rows inside a fragment is the same for both operands, so it
// cancels out.  x's fragment is the first operand and Y's the second, so a lane
// holds C[n = l % 16][k = 4 (l / 16) + r]: consecutive elements of one row of C.
//
// e4m3 codes become bf16 on their way into LDS.  An E8M0 scale times a code is
// exact in bf16 (one converting instruction); a per-tensor scale multiplies the
// sum at the end; a code times an fp32 block scale is kept as a sum of two bf16
// numbers, 2^-17 relative, and multiplied twice, whatever C's type: one of them
// would put 2^-9 more into every product, as much as a bf16 C's own rounding
// (32 experts of 585 to 2933 rows: 1.98e-3 from 64 bits, where exact operands
// give 1.66e-3).
//
// Pipeline, per step of 32 rows: the fragments of step s are in registers while
// those of s + 1 are read from LDS, the codes of s + 2 are converted and the
// copies of s + kD are sent off, all of it placed between the products by hand
// (one wave per SIMD: nothing else hides a stall).  One barrier a step.
// bf16 is bound by the matrix pipes (72 % busy) and the chip's power: 8192 rows,
// 8192 x 4096, 393-418 us by card (1.32-1.40 PFLOP/s).  mxfp8 to fp32 418-456 us
// (478 under a profiler): the conversion, which every workgroup along n does again,
// puts 375 cycles on the 1427 of a step (pipes 57 % busy; on zeros, where power
// does not bind, 396 us and bf16 314).  Block scales, with two products, 800-836;
// 32 experts of 585 to 2933 rows, 4096 x 2048, block scales to bf16, 994-1018
// (1109 under a profiler).
#include <algorithm>
#include <cmath>

#include "gemm_common.h"

namespace dgp {

namespace {

constexpr int kStep = 32;                  // rows per step
constexpr uint32_t kNowhere = 0xFFFFFFF0u; // an offset past every buffer's end: loads as zero

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

// Four rows of the 16 columns that start at p (in LDS, 32 bytes a row), a column a lane.
__device__ inline u32x2 transposed(const uint8_t *p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
}

// The async copies of gemm_common.h as inline assembly: behind the builtin the
// compiler waits for every copy in flight before each transposing read (it
// tells their LDS apart for ordinary reads only).  A copy waits out the write to
// m0; its scalar operands are made by scalar instructions, or by vector ones well
// before (5 wait states, which a test of the assembly counts).  The waits for
// the copies themselves are counted below.
template <int BYTES>
__device__ inline void copy_lds(const i32x4 &rsrc, uint8_t *lds_dst, uint32_t voff)
{
    const uint32_t at = (uint32_t)(uintptr_t)(lds_u8 *)lds_dst;
    if constexpr (kLdsPoison) {
        const int lane = (int)(threadIdx.x & 63);
        if constexpr (BYTES == 16)
            ((lds_i32x4 *)lds_dst)[lane] = i32x4{-1, -1, -1, -1};
        else
            ((lds_i32 *)lds_dst)[lane] = -1;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :: "s"(at), "v"(voff), "s"(rsrc) : "memory");
    else if constexpr (BYTES == 4)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                     :: "s"(at), "v"(voff), "s"(rsrc) : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, 0 offen lds"
                     :: "s"(at), "v"(voff), "s"(rsrc) : "memory");
}

// A run of bytes that a copy's range is cut from: `left` bytes from `base` on
// (none where it is not positive), moved on by one step at a time.
struct Run {
    uint64_t base;
    int64_t left;
    __device__ inline void next(int64_t bytes) { base += (uint64_t)bytes, left -= bytes; }
    __device__ inline i32x4 rsrc() const
    {
        const uint32_t n = left <= 0 ? 0u : left >= 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)left;
        return i32x4{(int)(uint32_t)base, (int)(uint32_t)(base >> 32), (int)n, 0x00020000};
    }
};

// f(0), f(1), ... f(N - 1) with compile-time numbers.
template <int... I, class Fn>
__device__ inline void each_of(std::integer_sequence<int, I...>, Fn f)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class Fn>
__device__ inline void each_of(Fn f)
{
    each_of(std::make_integer_sequence<int, N>{}, f);
}

// Accumulator in place in the AGPRs (F = 8: all 256 of them): the compiler
// would move it between register files.  Its inputs come straight from LDS.
template <bool AGPR>
__device__ inline void multiply_add(f32x4 &acc, const i32x4 &x, const i32x4 &y)
{
    if constexpr (AGPR)
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(x), "v"(y));
    else
        acc = mfma_op(x, y, acc);
}

// Two codes (the low or the HIGH half of four) -> two bf16 values.  `scale`: E8M0
// byte or fp32 bits.  `low` (block scales): what the rounding to bf16 left over,
// rounded to bf16 itself.
template <int MODE, bool HIGH>
__device__ inline uint32_t widen(int codes, uint32_t scale, uint32_t &low)
{
    if constexpr (MODE == kScaleBlock) {
        const float s = __builtin_bit_cast(float, scale);
        const auto c = __builtin_amdgcn_cvt_pk_f32_fp8(codes, HIGH);
        const float v[2] = {c[0] * s, c[1] * s};
        const uint32_t w = pack_bf16x2(v[0], v[1]);
        low = pack_bf16x2(v[0] - __builtin_bit_cast(float, w << 16), v[1] - __builtin_bit_cast(float, w & 0xFFFF0000u));
        return w;
    } else {
        // the instruction takes the exponent field of its fp32 scale: 2^(e - 127), NaN for e = 255
        const float s = __builtin_bit_cast(float, MODE == kScaleMx ? scale << 23 : 0x3F800000u);
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, HIGH));
    }
}

}  // namespace

// Tile `wg` of the grid in the order of the groups, in each a raster over 4 tile
// rows.  Workgroups go to the XCDs in turn (wg % 8) whatever they take, so an XCD
// gets every eighth run of 2^chunk_log2 neighbouring tiles (one group: one run): neighbours share their
// operands' panels in its L2, and each XCD has its part of every group, which
// groups of unequal size need (32 groups of 585 to 2933 rows, N 4096, K 2048,
// block scales by row list, one product: 997 us with four whole groups an XCD, 790
// where all have 1024).  Tiles behind the last whole round keep their number.
struct Tile {
    int n, k, s;
};
__device__ inline Tile tile_at(uint32_t wg, uint32_t tiles_n, uint32_t tiles_k, uint32_t groups, uint32_t chunk_log2)
{
    constexpr uint32_t kLog = 3;
    static_assert(kNumXcd == 1 << kLog, "");
    const uint32_t per = tiles_n * tiles_k, x = wg & (kNumXcd - 1), i = wg >> kLog;
    uint32_t t = wg;
    Tile r{0, 0, 0};
    if (groups == 1) {       // one run an XCD
        if (i < per >> kLog)
            t = x * (per >> kLog) + i;
    } else {
        if (wg < (per * groups >> (kLog + chunk_log2)) << (kLog + chunk_log2))
            t = (((i >> chunk_log2) << kLog | x) << chunk_log2) + (i & ((1u << chunk_log2) - 1));
        r.s = (int)(t / per);
        t -= (uint32_t)r.s * per;
    }
    const uint32_t strip = t / (4 * tiles_k), rows = tiles_n - 4 * strip, in = t - strip * 4 * tiles_k;
    if (rows >= 4)
        r.n = (int)(4 * strip + (in & 3)), r.k = (int)(in >> 2);
    else
        r.n = (int)(4 * strip + in % rows), r.k = (int)(in / rows);
    return r;
}

// F: fragments of a wave along n and along k (4 waves, 2 x 2: a tile of 32 F).
template <int MODE, int F, bool GATHER, bool BF16>
__global__ __launch_bounds__(256, F == 8 ? 1 : 2) void wgrad_kernel(const WgradArgs a, const int tiles_n, const int tiles_k, const int chunk_log2)
{
    constexpr bool kCodes = MODE != kScaleNone;
    constexpr int TERMS = MODE == kScaleBlock ? 2 : 1;   // bf16 numbers that make up a value of x
    constexpr bool kScaled = MODE == kScaleBlock || MODE == kScaleMx;
    constexpr int kCols = 32 * F;                        // tile
    constexpr int H = F / 4;                             // 128-column halves
    constexpr int kD = 3;                                // steps that the copies run ahead (4 and 5: the same times)
    constexpr int kRow4 = kCols * 8;                     // bytes of 4 rows x kCols in LDS
    constexpr int kTile = kStep * kCols * 2;             // bytes of a bf16 stage
    constexpr int kXStages = kCodes ? 2 : kD;
    // codes: H copies of 1 KiB a wave and step, their scales a dword a lane each
    constexpr int kCodeStage = kCodes ? 4 * H * 1024 : 0, kScaleStage = kScaled ? 4 * H * 256 : 0;
    constexpr int kIdx = kCodes ? H : 2;                 // row indices a lane and step
    constexpr int kIdxStage = GATHER ? 4 * kIdx * 256 : 0;
    constexpr int kOffX = kD * kTile, kOffCodes = kOffX + kXStages * TERMS * kTile;
    constexpr int kOffScales = kOffCodes + kD * kCodeStage, kOffIdx = kOffScales + kD * kScaleStage;
    constexpr int kIdxStages = 8;        // (a stage is read in the step after the one that its next copy sits in)
    constexpr int kLds = kOffIdx + kIdxStages * kIdxStage;
    static_assert(kLds <= 160 * 1024, "LDS");
    constexpr int kGroup = 2 * H + (kCodes ? H : 2 * H) + (kScaled ? H : 0) + (GATHER ? kIdx : 0);   // copies a step
    static_assert(kGroup * (kD - 1) < 64, "copies in flight");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    if constexpr (kLdsPoison) {
        lds_poison_fill(lds, kLds);
        __syncthreads();
    }

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tile tile = tile_at(blockIdx.x, tiles_n, tiles_k, (uint32_t)a.E * a.splits, chunk_log2);
    const int n0 = tile.n * kCols, k0 = tile.k * kCols;
    const int e = a.splits == 1 ? tile.s : tile.s / a.splits, split = tile.s - e * a.splits;

    // The rows of this workgroup.
    int64_t lo = 0, hi = a.M;
    if (a.offsets) {
        lo = a.offsets[e], hi = a.offsets[e + 1];
        lo = lo < 0 ? 0 : lo > a.M ? a.M : lo;
        hi = hi < lo ? lo : hi > a.M ? a.M : hi;
    }
    if (a.splits > 1) {
        const int64_t per = ((hi - lo + a.splits - 1) / a.splits + kStep - 1) / kStep * kStep;
        lo += split * per;
        hi = lo > hi ? lo : lo + per < hi ? lo + per : hi;
    }
    const int steps = __builtin_amdgcn_readfirstlane((int)((hi - lo + kStep - 1) / kStep));

    // ---- copies.  A 1 KiB copy fills 16-byte pieces of LDS in order: 8 blocks
    // of 4 rows x 16 columns.  Copy (rg, half) of a stage holds the rows 4 rg ..
    // 4 rg + 3 and 128 columns: a lane's piece is row 4 rg + lane % 8 / 2, eight
    // columns from 16 (lane / 8) + 8 (lane % 2).
    const int krow = (lane & 7) >> 1, kcol = (lane >> 3) * 16 + (lane & 1) * 8;
    const int64_t K = a.K;
    const uint32_t x_size = kCodes ? 1 : 2;
    // A lane's piece of codes: row crow of the copy's first row group, 16 columns.
    const int crow = (lane & 3) + (F == 8 ? 0 : (lane >> 5) * 4), ccol = (F == 8 ? lane >> 2 : (lane >> 2) & 7) * 16;

    // What a step's copies read, from its first row on: Y, x and x's scales (or,
    // by row list, all of the rows of X), the row list.
    const int64_t kb = K / 128, s_size = MODE == kScaleBlock ? 4 : 1, rows = hi - lo;
    const int64_t ldy2 = a.ldy * 2, ldx = K * x_size, lds_ = kb * s_size;
    const int64_t x_rows = GATHER ? a.x_rows : rows, x_first = GATHER ? 0 : lo;
    Run ry{(uint64_t)a.Y + (uint64_t)(lo * ldy2 + n0 * 2), (rows - 1) * ldy2 + (a.N - n0) * 2};
    Run rx{(uint64_t)a.X + (uint64_t)(x_first * ldx + k0 * x_size), x_rows * ldx - k0 * (int64_t)x_size};
    Run rs{(uint64_t)a.S + (uint64_t)(x_first * lds_ + k0 / 128 * s_size), x_rows * lds_ - k0 / 128 * s_size};
    Run ri{(uint64_t)a.rows + (uint64_t)(lo * 4), rows * 4};
    int x_left = (int)(rows < INT32_MAX ? rows : INT32_MAX);    // (by row list) rows from this step on

    // Rows (within the step) of the lane's pieces, and their offsets.
    uint32_t row_of[kIdx];
#pragma unroll
    for (int j = 0; j < kIdx; ++j)
        row_of[j] = kCodes ? (F == 8 ? 4 * (j * 4 + wave) : 8 * wave) + crow : 4 * (j * 4 + wave) + krow;
    const uint32_t x_col = kCodes ? (uint32_t)ccol : (uint32_t)kcol * 2, s_col = (uint32_t)ccol / 128 * (uint32_t)s_size;
    uint32_t y_off[2], x_off[kIdx], s_off[kIdx];
    auto place_x = [&](const int (&idx)[kIdx]) {
#pragma unroll
        for (int j = 0; j < kIdx; ++j) {
            const uint32_t r = GATHER ? (uint32_t)idx[j] : row_of[j];
            x_off[j] = r * (uint32_t)ldx + x_col;
            s_off[j] = r * (uint32_t)lds_ + s_col;
            if (GATHER && ((int)row_of[j] >= x_left || r >= (uint32_t)a.x_rows))
                x_off[j] = s_off[j] = kNowhere;
        }
    };
#pragma unroll
    for (int j = 0; j < 2; ++j)
        y_off[j] = (uint32_t)(4 * (j * 4 + wave) + krow) * (uint32_t)ldy2 + (uint32_t)kcol * 2;

    // Copies of one step, numbered 0 .. kGroup - 1; slot: the LDS stage of each kind.
    i32x4 dy, dx, ds, di;      // ranges of Y, x, scales and row list
    auto copy_y = [&](int j, int slot) {
        const int rg = (j / H) * 4 + wave, half = j % H;
        copy_lds<16>(dy, lds + slot * kTile + rg * kRow4 + half * 1024, y_off[j / H] + half * 256);
    };
    auto copy_x = [&](int j, int slot) {
        if constexpr (kCodes) {
            copy_lds<16>(dx, lds + kOffCodes + slot * kCodeStage + (j * 4 + wave) * 1024, x_off[j % kIdx]);
        } else {
            const int rg = (j / H) * 4 + wave, half = j % H;
            const uint32_t off = x_off[j / H] + half * 256;
            copy_lds<16>(dx, lds + kOffX + slot * kTile + rg * kRow4 + half * 1024, GATHER && x_off[j / H] == kNowhere ? kNowhere : off);
        }
    };
    auto copy_s = [&](int j, int slot) {
        copy_lds<MODE == kScaleBlock ? 4 : 1>(ds, lds + kOffScales + slot * kScaleStage + (j * 4 + wave) * 256, s_off[j % kIdx]);
    };
    auto copy_i = [&](int j, int slot) {
        copy_lds<4>(di, lds + kOffIdx + slot * kIdxStage + (j * 4 + wave) * 256, row_of[j % kIdx] * 4);
    };
    constexpr int kXCopies = kCodes ? H : 2 * H, kSCopies = kScaled ? H : 0, kICopies = GATHER ? kIdx : 0;
    static_assert(kGroup == 2 * H + kXCopies + kSCopies + kICopies, "");
    auto copy = [&](auto cc, int slot_y, int slot_x, int slot_i) {
        constexpr int c = decltype(cc)::value;
        if constexpr (c < 2 * H)
            copy_y(c, slot_y);
        else if constexpr (c < 2 * H + kXCopies)
            copy_x(c - 2 * H, slot_x);
        else if constexpr (c < 2 * H + kXCopies + kSCopies)
            copy_s(c - 2 * H - kXCopies, slot_x);
        else
            copy_i(c - 2 * H - kXCopies - kSCopies, slot_i);
    };
    // The next step's ranges.
    auto next_y = [&] { dy = ry.rsrc(), ry.next(kStep * ldy2); };
    auto next_x = [&] {
        dx = rx.rsrc(), ds = rs.rsrc();
        if constexpr (!GATHER)
            rx.next(kStep * ldx), rs.next(kStep * lds_);
    };
    auto next_i = [&] { di = ri.rsrc(), ri.next(kStep * 4); };

    // Pair v of 8 of the wave's own codes (copy j) of one step, as bf16; with every fourth one
    // eight values go to an LDS stage of x.
    constexpr int kPairs = kCodes ? 8 * H : 0;
    i32x4 wide[TERMS];
    auto convert = [&](auto vc, const i32x4 &c, uint32_t s, int x_slot) {
        constexpr int j = decltype(vc)::value / 8, v = decltype(vc)::value % 8;
        uint32_t low = 0;
        wide[0][v % 4] = (int)widen<MODE, v % 2 == 1>(c[v / 2], s, low);
        if constexpr (TERMS == 2)
            wide[1][v % 4] = (int)low;
        if constexpr (v % 4 == 3) {
            uint8_t *d = lds + kOffX + x_slot * (TERMS * kTile) + (row_of[j % kIdx] >> 2) * kRow4 + (ccol >> 4) * 128 + (crow & 3) * 32;
#pragma unroll
            for (int q = 0; q < TERMS; ++q)
                reinterpret_cast<i32x4 *>(d + q * kTile)[v / 4] = wide[q];
        }
    };
    auto read_codes = [&](int j, int slot, i32x4 &c, uint32_t &s) {
        c = *reinterpret_cast<const i32x4 *>(lds + kOffCodes + slot * kCodeStage + (j * 4 + wave) * 1024 + lane * 16);
        s = 0;
        if constexpr (kScaled)
            s = reinterpret_cast<const uint32_t *>(lds + kOffScales + slot * kScaleStage + (j * 4 + wave) * 256)[lane];
    };

    // ---- fragments.  Wave (wn, wk) of 2 x 2 owns 16 F columns of each operand.
    const int wn = wave >> 1, wk = wave & 1;
    const int frag = (lane >> 4) * kRow4 + (lane & 15) * 8;     // row groups 0..3 by lane / 16, then 4..7
    const uint8_t *const yfrag = lds + frag + wn * F * 128;
    const uint8_t *const xfrag = lds + kOffX + frag + wk * F * 128;
    i32x4 yf[2][F], xf[2][TERMS][F];
    f32x4 acc[F][F];                                            // [k fragment][n fragment]
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // Half h (four of a lane's eight rows) of fragment f: F of Y's, then x's.
    auto read_half = [&](auto pc, auto rc, int y_slot, int x_slot) {
        constexpr int P = decltype(pc)::value, f = decltype(rc)::value / 2, h = decltype(rc)::value % 2;
        i32x4 &d = f < F ? yf[P][f % F] : xf[P][f < F ? 0 : (f - F) / F][f % F];
        const u32x2 v = transposed((f < F ? yfrag + y_slot * kTile : xfrag + x_slot * (TERMS * kTile) + (f - F) / F * kTile) +
                                   f % F * 128 + h * 4 * kRow4);
        d[2 * h] = (int)v.x, d[2 * h + 1] = (int)v.y;
    };

    // Group g of copies (one per step, and before the first step those of -kD + 1 .. -1):
    // Y of step g + kD, x of g + kD (codes: kD + 1), the row list for x of group g + kD + 1.
    constexpr int kAhead = kCodes ? 1 : 0;
    constexpr int kReads = 2 * F * (1 + TERMS), kProducts = F * F * TERMS;
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    int idx[kIdx];
    // row indices of the steps before the list comes through LDS: all loads first
    int head[kD + kAhead + 1][kIdx];
#pragma unroll
    for (int t = 0; t <= kD + kAhead; ++t)
#pragma unroll
        for (int j = 0; j < kIdx; ++j) {
            const int64_t m = lo + (int64_t)t * kStep + row_of[j];
            head[t][j] = GATHER && m < hi ? a.rows[m] : 0;
        }
    auto first_idx = [&](int t) {
        place_x(head[t]);
        x_left -= kStep;
    };
    next_y();
    for (int c = 0; c < 2 * H; ++c)
        copy_y(c, 0);
#pragma unroll
    for (int t = 0; t <= kAhead; ++t) {
        first_idx(t);
        next_x();
        for (int c = 0; c < kXCopies; ++c)
            copy_x(c, t);
        for (int c = 0; c < kSCopies; ++c)
            copy_s(c, t);
    }
    if constexpr (GATHER) {
        ri.next((kD + kAhead + 1) * kStep * 4);
        next_i();
        for (int c = 0; c < kICopies; ++c)
            copy_i(c, 1 % kIdxStages);
    }
    auto first_group = [&](int g) {
        first_idx(g + kD + kAhead);
        next_y(), next_x(), next_i();
        each_of<kGroup>([&](auto c) { copy(c, (g + kD) % kD, (g + kD + kAhead) % kD, (g + kD + 1) % kIdxStages); });
    };
#pragma unroll
    for (int g = 1 - kD; g < -1; ++g)
        first_group(g);
    if constexpr (kCodes) {
        // (group -1 copies codes to where those of step 0 are)
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kD - 2) * kGroup) : "memory");
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            i32x4 c[H];
            uint32_t s[H];
#pragma unroll
            for (int j = 0; j < H; ++j)
                read_codes(j, t, c[j], s[j]);
            each_of<kPairs>([&](auto v) { convert(v, c[decltype(v)::value / 8], s[decltype(v)::value / 8], t); });
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    first_group(-1);
    first_idx(kD + kAhead);      // (the offsets of step 0's copies; GATHER waits for every load here)
    next_y(), next_x(), next_i();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kD - 1) * kGroup) : "memory");
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    each_of<kReads>([&](auto r) { read_half(I0{}, r, 0, 0); });
    // s % kD; stages s + 1 and s + 2
    int slot = 0;
    auto step = [&](auto pc, int s) {
        constexpr int P = decltype(pc)::value;
        const int slot1 = slot + 1 < kD ? slot + 1 : 0, slot2 = slot1 + 1 < kD ? slot1 + 1 : 0;
        // Y and x (codes: of the step after) of step s + 1 have landed, here and, behind
        // the barrier, in every wave; every wave has read the fragments of step s.
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kD - 2) * kGroup) : "memory");
        __builtin_amdgcn_sched_barrier(0);
        i32x4 codes[kCodes ? H : 1];
        uint32_t scales[kCodes ? H : 1];
        // Behind each product no more than the matrix unit's 16 cycles let through.  Counted in
        // products: the reads of codes and row indices first, the next step's fragments over the
        // first three quarters, the copies over all but the last four, the conversion of the codes
        // from an eighth on over five eighths, the next copies' ranges and offsets at the end.
        each_of<kProducts>([&](auto mc) {
            constexpr int m = decltype(mc)::value, q = m / (F * F), i = m / F % F, j = m % F;
            multiply_add<F == 8>(acc[i][j], xf[P][q][i], yf[P][j]);
            if constexpr (kCodes && m < H)
                read_codes(m, slot2, codes[m], scales[m]);
            if constexpr (GATHER && m == 2) {
#pragma unroll
                for (int t = 0; t < kIdx; ++t)
                    idx[t] = reinterpret_cast<const int *>(lds + kOffIdx + (s + 1) % kIdxStages * kIdxStage + (t * 4 + wave) * 256)[lane];
            }
            constexpr auto part = [](int x, int first, int over, int all) {      // items before product x
                return x <= first ? 0 : x >= first + over ? all : (x - first) * all / over;
            };
            constexpr int r0 = part(m, 0, kProducts * 3 / 4, kReads), r1 = part(m + 1, 0, kProducts * 3 / 4, kReads);
            each_of<r1 - r0>([&](auto r) {
                read_half(std::integral_constant<int, 1 - P>{}, std::integral_constant<int, r0 + decltype(r)::value>{}, slot1,
                          kCodes ? (s + 1) & 1 : slot1);
            });
            constexpr int c0 = part(m, 0, kProducts - 4, kGroup), c1 = part(m + 1, 0, kProducts - 4, kGroup);
            each_of<c1 - c0>([&](auto c) {
                copy(std::integral_constant<int, c0 + decltype(c)::value>{}, slot, kCodes ? slot1 : slot, (s + kD + 1) % kIdxStages);
            });
            constexpr int v0 = part(m, kProducts / 8, kProducts * 5 / 8, kPairs), v1 = part(m + 1, kProducts / 8, kProducts * 5 / 8, kPairs);
            each_of<v1 - v0>([&](auto v) {
                constexpr int at = v0 + decltype(v)::value;
                convert(std::integral_constant<int, at>{}, codes[at / 8], scales[at / 8], s & 1);
            });
            if constexpr (m == kProducts - 3)
                next_y();
            if constexpr (m == kProducts - 2)
                next_x();
            if constexpr (GATHER && m == kProducts - 1)
                next_i(), place_x(idx), x_left -= kStep;
            __builtin_amdgcn_sched_barrier(0);
        });
        slot = slot1;
    };
    // (in pairs, one at least: the accumulators of a loop with two ends would be copied at one of them;
    // a step past the last row multiplies zeros)
    int s = 0;
    do {
        step(I0{}, s);
        step(I1{}, s + 1);
        s += 2;
    } while (s < steps);
    // (copies of steps that do not come; the last products, which the compiler does not see as such)
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);

    // ---- results
    float scale = 1.0f;
    if (MODE == kScaleTensor && rows > 0)
        scale = static_cast<const float *>(a.S)[0];
    // N and K are multiples of 16, so a fragment is inside or outside as a whole.
    const int nf = n0 + wn * (F * 16), kf = k0 + wk * (F * 16);
    int l = lane;
    asm volatile("" : "+v"(l));     // (addresses that are worked out here, not held through the loop)
    const int64_t at = (int64_t)(nf + (l & 15)) * K + kf + (l >> 4) * 4, row16 = 16 * K;
    auto each = [&](auto *c, auto store) {
        c += at;
        auto all = [&](auto full) {
            auto *p = c;
#pragma unroll
            for (int j = 0; j < F; ++j, p += row16) {
                if (!full && nf + j * 16 >= a.N)
                    break;
#pragma unroll
                for (int i = 0; i < F; ++i)
                    if (full || kf + i * 16 < K) {
                        f32x4 v = acc[i][j];
                        // (read here, not all 64 of them at the loop's end)
                        asm volatile("" : "+v"(v));
                        if constexpr (MODE == kScaleTensor)
                            v = v * scale;
                        store(p + i * 16, v);
                    }
            }
        };
        if (n0 + kCols <= a.N && k0 + kCols <= K)
            all(std::true_type{});
        else
            all(std::false_type{});
    };
    const int64_t group = ((int64_t)split * a.E + e) * a.N * K;
    auto write = [](float *c, const f32x4 &v) { *reinterpret_cast<f32x4 *>(c) = v; };
    if constexpr (BF16) {
        if (a.splits > 1)
            each(a.ws + group, write);
        else
            each(static_cast<uint16_t *>(a.C) + group, [](uint16_t *c, const f32x4 &v) {
                *reinterpret_cast<u32x2 *>(c) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            });
    } else if (a.accumulate && a.splits == 1) {
        each(static_cast<float *>(a.C) + group, [](float *c, const f32x4 &v) { *reinterpret_cast<f32x4 *>(c) += v; });
    } else {
        each((a.splits > 1 ? a.ws : static_cast<float *>(a.C)) + group, write);
    }
}

// C (+)= the sum of `splits` partial results in order, rounded once.
template <bool BF16>
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float *ws, void *C, int64_t quads, int splits, int accumulate)
{
    const f32x4 *p = reinterpret_cast<const f32x4 *>(ws);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
        f32x4 v = p[i];
        for (int s = 1; s < splits; ++s)
            v += p[s * quads + i];
        if constexpr (BF16) {
            static_cast<u32x2 *>(C)[i] = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        } else {
            f32x4 *c = static_cast<f32x4 *>(C) + i;
            *c = accumulate ? *c + v : v;
        }
    }
}

// --------------------------------------------------------------- launches

// Tile and parts of a group's rows, by estimated time (us): with W workgroups of
// `steps` steps and out MB of results (fp32 partial ones where there are parts),
//
//   256: 5.5 + ceil(W / 256) (7.1 + steps (0.59 + 0.11 min(1, W / 256))) + out / 12.8
//   128: 4.7 + ceil(W / 256) (2.1 + 0.29 steps) + (0.075 steps, a workgroup a CU at most) + out / 12.8
//   parts: 3.6 + out / 6.4 for adding them up
//
// fitted to graph timings of 58 shapes (64 to 20000 rows, 256 x 256 to 8192 x 8192,
// 1 to 64 groups, up to 14 choices each): the choice is on average 0.5 % slower
// than the fastest (at worst 14 %: 2048 rows, 512 x 1024).  Groups count as even,
// as those of the fit were: the host does not know their rows, and a group that
// has most of them gets no more parts than the others (16 384 rows of 64 experts of
// 1024 x 1024, nearly all of one: 16 workgroups walk them, about 370 us by the
// formula above where that weight alone in 16 parts is at 54).  The 128 tile reads twice
// the bytes for a product, 14 TB/s out of the L2s with four workgroups a CU (1.2 us
// for a step of theirs, where the 256 tile takes 0.7 for the same products); it is
// there for weights with too few large tiles, as parts are (8192 rows, 2048 x 2048:
// 128 tile 80 us, 256 tile in one part 155, in four 74).
WgradPlan wgrad_plan(int64_t M, int64_t N, int64_t K, int64_t E)
{
    const int64_t rows = (M + E - 1) / E;
    WgradPlan best{128, 1};
    double least = 0;
    for (const int tile : {128, 256})
        for (const int parts : {1, 2, 3, 4, 6, 8, 16}) {
            if (parts > 1 && rows < parts * 96)
                break;
            const double w = (double)((N + tile - 1) / tile) * (double)((K + tile - 1) / tile) * (double)E * parts;
            const double rounds = std::ceil(w / kNumCu), steps = (double)((rows + parts * 64 - 1) / (parts * 64) * 2);
            const double out = (double)E * (double)N * (double)K * 4e-6 * parts;
            double us = out / 12.8 + (parts > 1 ? 3.6 + out / 6.4 : 0.0);
            if (tile == 256)
                us += 5.5 + rounds * (7.1 + steps * (0.59 + 0.11 * std::min(1.0, w / kNumCu)));
            else
                us += 4.7 + rounds * (2.1 + 0.29 * steps) + (w <= kNumCu ? 0.075 * steps : 0.0);
            if (least == 0 || us < least)
                best = {tile, parts}, least = us;
        }
    return best;
}

namespace {

template <int MODE, int F, bool BF16>
void launch_tile(const WgradArgs &a, hipStream_t s)
{
    const int64_t tile = 32 * F, tn = (a.N + tile - 1) / tile, tk = (a.K + tile - 1) / tile;
    const unsigned grid = (unsigned)(tn * tk * a.E * a.splits);
    // several groups: runs of an eighth of one's tiles, 4 to 32
    int chunk = 2;
    while (chunk < 5 && tn * tk >= (int64_t)kNumXcd << (chunk + 1))
        ++chunk;
    if (a.rows)
        wgrad_kernel<MODE, F, true, BF16><<<grid, 256, 0, s>>>(a, (int)tn, (int)tk, chunk);
    else
        wgrad_kernel<MODE, F, false, BF16><<<grid, 256, 0, s>>>(a, (int)tn, (int)tk, chunk);
}

template <int F, bool BF16>
hipError_t launch_mode(const WgradArgs &a, int mode, hipStream_t s)
{
    switch (mode) {
    case kScaleNone: launch_tile<kScaleNone, F, BF16>(a, s); break;
    case kScaleTensor: launch_tile<kScaleTensor, F, BF16>(a, s); break;
    case kScaleBlock: launch_tile<kScaleBlock, F, BF16>(a, s); break;
    case kScaleMx: launch_tile<kScaleMx, F, BF16>(a, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_wgrad(const WgradArgs &args, int mode, bool out_bf16, const WgradPlan &plan, hipStream_t s)
{
    WgradArgs a = args;
    a.splits = plan.splits;
    const hipError_t err = plan.tile == 256 ? (out_bf16 ? launch_mode<8, true>(a, mode, s) : launch_mode<8, false>(a, mode, s))
                                            : (out_bf16 ? launch_mode<4, true>(a, mode, s) : launch_mode<4, false>(a, mode, s));
    if (err != hipSuccess || plan.splits == 1)
        return err;
    const int64_t quads = a.E * a.N * a.K / 4;
    const unsigned grid = (unsigned)(quads / 256 + 1 < 4096 ? quads / 256 + 1 : 4096);
    if (out_bf16)
        wgrad_join_kernel<true><<<grid, 256, 0, s>>>(a.ws, a.C, quads, plan.splits, 0);
    else
        wgrad_join_kernel<false><<<grid, 256, 0, s>>>(a.ws, a.C, quads, plan.splits, a.accumulate);
    return hipGetLastError();
}

}  // namespace dgp
