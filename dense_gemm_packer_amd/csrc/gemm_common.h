// Device helpers shared by the GEMM kernel families (gemm_tiled.hip,
// gemm_stream.hip): matrix-core operations, LDS fragment reads, the async
// global->LDS copy, and the epilogue store.
//
// Matrix-core operands.  bf16 uses v_mfma_f32_16x16x32_bf16 (the K32 MFMA
// selected for bf16 on gfx950, FlyDSL PR #1008 review excerpt) and fp8 the
// 128-deep v_mfma_f32_16x16x128_f8f6f4 (same excerpt; scale operands left at
// 0, which selects the unscaled form).  The preshuffled B fragment is passed
// as the instruction's FIRST operand and the A fragment as its second, so the
// instruction produces the 16x16 tile of C^T: lane l holds
// C[m = l%16][n = 4*(l/16) + r], r = 0..3 -- four consecutive columns of one
// row, written with a single 8-byte (bf16) or 16-byte (fp32) store.  Both
// operands use the same in-register K order, so any K permutation the
// hardware applies inside one instruction is applied to both alike.
//
// A in LDS.  The A tile is stored in the same 1 KiB operand blocks as the
// preshuffled B: block (row group rg, 64-byte K chunk c) holds, at byte
// 16*l, the 16 bytes of row 16*rg + l%16 at K-bytes 64*c + 16*(l/16).  The
// writer (the async copy, whose LDS side is linear per wave) realises this
// permutation through the global addresses of its lanes; the reader reads
// 16 consecutive bytes per lane.  Writer and reader share the one mapping,
// and both sides touch 64 distinct 16-byte bank groups per wave: no bank
// conflicts by construction.  (The pages keep a row-major tile with an XOR
// swizzle whose writer and reader had to be made to agree, FlyDSL PR #1008
// "Changes" item 2; this mapping is the same idea -- a 16-byte-granular LDS
// permutation known to both sides -- chosen for the operand order.)
#pragma once

#include <type_traits>
#include <utility>

#include "common.h"
#include "launch.h"

namespace dgp {

// ---------------------------------------------------------------- MFMA

__device__ inline f32x4 mfma_op(const i32x4 &b, const i32x4 &a, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b),
                                                   __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
}

__device__ inline f32x4 mfma_op(const i32x8 &b, const i32x8 &a, const f32x4 &c)
{
    // cbsz = blgp = 0: both operands OCP e4m3; zero scale operands: unscaled.
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, 0, 0, 0, 0);
}

// Hardware-scaled e4m3 MFMA (mxfp8): eb, ea are E8M0 bytes (2^(e-127)) for the
// B fragment (first operand: lane l's byte scales row l%16 of it) and the A
// fragment (second operand: column l%16) over the K block lane l / 16 selects;
// in the operand order of this library that block is K [32q, 32q+32) of the
// 128-deep step, so an MX scale that is constant over the step (128-element
// blocks) applies to the whole step.
__device__ inline f32x4 mfma_mx(const i32x8 &b, const i32x8 &a, const f32x4 &c, int eb, int ea)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, 0, eb, 0, ea);
}

// Hardware-scaled E2M1 MFMA (mxfp4): 16 bytes = 32 values per lane, lane l
// holding K [32g, 32g+32) (g = l/16) of its row -- exactly one 32-element
// microscaling block -- whose E8M0 scales are eb (B fragment, first operand)
// and ea (A fragment, second operand).
__device__ inline f32x4 mfma_mx4(const i32x4 &b, const i32x4 &a, const f32x4 &c, int eb, int ea)
{
    const i32x8 b8 = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
    const i32x8 a8 = {a.x, a.y, a.z, a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b8, a8, c, 4, 4, 0, eb, 0, ea);
}

__device__ inline i32x8 cat(const i32x4 &lo, const i32x4 &hi)
{
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int DT>
struct Op;
template <>
struct Op<kDtypeBf16> {
    using Frag = i32x4;
    static constexpr int kBlocks = 1;   // 1 KiB operand blocks per MFMA step (64 K-bytes)
};
template <>
struct Op<kDtypeFp8> {
    using Frag = i32x8;
    static constexpr int kBlocks = 2;   // 128 K-bytes
};
template <>
struct Op<kDtypeFp4> {
    using Frag = i32x4;
    static constexpr int kBlocks = 1;   // 64 K-bytes = 128 elements
};

template <int DT>
__device__ inline typename Op<DT>::Frag lds_frag(const uint8_t *p)
{
    if constexpr (Op<DT>::kBlocks == 1) {
        return *reinterpret_cast<const i32x4 *>(p);
    } else {
        return cat(*reinterpret_cast<const i32x4 *>(p), *reinterpret_cast<const i32x4 *>(p + 1024));
    }
}

// ------------------------------------------------------------ LDS poison
//
// The LDS-poison debug build (the library compiled a second time with
// DGP_LDS_POISON=1, libdgp_lds_poison.so) turns a kernel that reads LDS its
// copies have not filled -- a tile only partly loaded, or a read that runs
// ahead of the wait for its copy -- into a parity failure instead of a quiet
// wrong answer at full speed.  Every kernel fills its LDS with 0xFF bytes
// before its first copy (a NaN in bf16, e4m3, E8M0 and fp32; -6 in E2M1),
// and every global -> LDS copy first overwrites its own destination with
// 0xFF and waits for that write, so LDS holds poison from the moment a
// stage is handed to a copy until the copy lands.  The library built
// without the flag (kLdsPoison false, common.h) compiles none of it.
typedef __attribute__((address_space(3))) i32x4 lds_i32x4;
typedef __attribute__((address_space(3))) int lds_i32;

// Poison build: fill bytes [0, bytes) of an LDS array (bytes a multiple of
// 16) with 0xFF, spread over the workgroup's threads.  The caller
// synchronises the workgroup before the first copy.
__device__ inline void lds_poison_fill(void *lds_base, int bytes)
{
    if constexpr (kLdsPoison) {
        lds_i32x4 *d = (lds_i32x4 *)lds_base;
        for (int i = (int)threadIdx.x; i < bytes / 16; i += (int)(blockDim.x * blockDim.y * blockDim.z))
            d[i] = i32x4{-1, -1, -1, -1};
    }
}

// Async global -> LDS copy of BYTES (16, 4, 2 or 1) per lane: lane l's
// 16 bytes land at lds_dst + 16 l, a narrow copy's value zero-extended in
// dword l.  Poison build: that destination is overwritten with 0xFF first.
template <int BYTES>
__device__ inline void lds_dma(__amdgpu_buffer_rsrc_t r, void *lds_dst, uint32_t voff, uint32_t soff)
{
    static_assert(BYTES == 16 || BYTES == 4 || BYTES == 2 || BYTES == 1, "copy width");
    if constexpr (kLdsPoison) {
        const int lane = (int)(threadIdx.x & 63);
        if constexpr (BYTES == 16)
            ((lds_i32x4 *)lds_dst)[lane] = i32x4{-1, -1, -1, -1};
        else
            ((lds_i32 *)lds_dst)[lane] = -1;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    auto *d = (__attribute__((address_space(3))) void *)lds_dst;
    if constexpr (BYTES == 16)   // (the size operand must be a literal)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, d, 16, voff, soff, 0, 0);
    else if constexpr (BYTES == 4)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, d, 4, voff, soff, 0, 0);
    else if constexpr (BYTES == 2)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, d, 2, voff, soff, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, d, 1, voff, soff, 0, 0);
}

__device__ inline void lds_dma16(__amdgpu_buffer_rsrc_t r, uint8_t *lds_dst, uint32_t voff, uint32_t soff)
{
    lds_dma<16>(r, lds_dst, voff, soff);
}

// ------------------------------------------------- product by expert
//
// GR = 1 forms of the kernels multiply the rows [offsets[e], offsets[e+1]) of
// the product with weight e.  The row counts are known on the device only, so
// the grid is the most tiles any counts give, and every wave finds its tile
// itself: a lane per expert takes its two offsets and its tile count, a DPP
// scan adds them up, and the tile's expert is the first whose running count
// passes it.  Tiles run expert by expert (an expert's weight is read by
// neighbouring workgroups), regrouped over the XCDs by the number of tiles
// there are, not by the grid; workgroups past it end at once.  The arguments
// are then narrowed to the expert's rows and weight, and the kernel runs as
// on one product.
// Offsets are clamped to [0, M] and to their predecessor, so whatever they
// hold no row outside the product is touched.

// Inclusive sum over the wave's lanes.
__device__ inline int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast 15 into rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast 31 into rows 2, 3
    return v;
}

// Rows [lo, hi) of this lane's expert e (none past the last one).
__device__ inline void expert_rows(const GemmArgs &p, int e, int &lo, int &hi)
{
    lo = hi = 0;
    if (e < p.groups) {
        lo = p.offsets[e];
        hi = p.offsets[e + 1];
        lo = lo < 0 ? 0 : lo > p.M ? p.M : lo;
        hi = hi < lo ? lo : hi > p.M ? p.M : hi;
    }
}

// This workgroup's tile; GR = 1: also narrows p to its expert.  False: none.
template <int GR, int TM, int SCALE>
__device__ inline bool locate_tile(GemmArgs &p, TileCoordT<int> &tc)
{
    if constexpr (GR == 0) {
        tc = tile_of_workgroup<int>((int)blockIdx.x, p.tiles_m, p.tiles_n, p.splits, p.remap, p.group_m);
        return true;
    } else {
        const int lane = threadIdx.x & 63;
        int lo, hi;
        expert_rows(p, lane, lo, hi);
        int n = (hi - lo + TM - 1) / TM;
        int incl = wave_scan(n);
        int total = __builtin_amdgcn_readlane(incl, 63);
        for (int e0 = 64; e0 < p.groups; e0 += 64) {
            int l2, h2;
            expert_rows(p, e0 + lane, l2, h2);
            total += __builtin_amdgcn_readlane(wave_scan((h2 - l2 + TM - 1) / TM), 63);
            total = total < p.tiles_m ? total : p.tiles_m;
        }
        total = total < p.tiles_m ? total : p.tiles_m;
        const int wg = (int)blockIdx.x;
        if (wg >= total * p.tiles_n)
            return false;
        int logical = wg;
        if (p.remap) {
            const int per = total * p.tiles_n / kNumXcd;
            if (wg < per * kNumXcd)
                logical = (wg % kNumXcd) * per + wg / kNumXcd;
        }
        const int rt = logical / p.tiles_n;          // row tile, counted over all experts
        int before = 0, e0 = 0;                      // row tiles before expert e0
        uint64_t past = __ballot(incl > rt);
        while (past == 0) {                          // (rt < total: an expert is found)
            before += __builtin_amdgcn_readlane(incl, 63);
            e0 += 64;
            expert_rows(p, e0 + lane, lo, hi);
            n = (hi - lo + TM - 1) / TM;
            incl = wave_scan(n);
            past = __ballot(before + incl > rt);
            if (e0 >= p.groups)
                return false;
        }
        const int at = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
        const int first = __builtin_amdgcn_readlane(lo, at), last = __builtin_amdgcn_readlane(hi, at);
        const int tiles = __builtin_amdgcn_readlane(n, at);
        before += __builtin_amdgcn_readlane(incl, at) - tiles;
        raster_tile<int>(logical - before * p.tiles_n, tiles, p.tiles_n, p.group_m < 1 ? 1 : p.group_m, tc.tm, tc.tn);
        tc.s = 0;
        const int64_t e = e0 + at;
        const int64_t kblk = SCALE == kScaleMx32 ? p.K / 32 : p.K / 128;
        p.M = last - first;
        p.Bs += e * p.N * (int64_t)p.Kb;
        p.C = static_cast<uint8_t *>(p.C) + (int64_t)first * p.N * 2;
        if constexpr (SCALE == kScaleTensor)
            p.sB = static_cast<const float *>(p.sB) + e;
        if constexpr (SCALE == kScaleBlock)
            p.sB = static_cast<const float *>(p.sB) + e * (p.N / 128) * kblk;
        if constexpr (SCALE == kScaleMx || SCALE == kScaleMx32)
            p.sB = static_cast<const uint8_t *>(p.sB) + e * p.N * kblk;
        if (p.rows) {
            p.rows += first;
        } else {
            p.A += (int64_t)first * p.Kb;
            if constexpr (SCALE == kScaleBlock)
                p.sA = static_cast<const float *>(p.sA) + (int64_t)first * kblk;
            if constexpr (SCALE == kScaleMx || SCALE == kScaleMx32)
                p.sA = static_cast<const uint8_t *>(p.sA) + (int64_t)first * kblk;
        }
        return true;
    }
}

// The buffer range of a tile's rows of A (or of A's scales), rows row_bytes
// long, and the byte offset of the tile's row r in it.  Rows past M lie past
// the range.  With a row list the range is all of A, and a row past M, or one
// that A does not have, goes to an offset past every range (the host keeps A
// below it, with room for the K offsets that are added).
constexpr uint32_t kNoRow = 0xFF000000u;

template <int GR>
__device__ inline __amdgpu_buffer_rsrc_t row_rsrc(const GemmArgs &p, const void *base, int m0, int64_t row_bytes)
{
    if constexpr (GR != 0) {
        if (p.rows)
            return make_rsrc(base, clamp_bytes((int64_t)p.a_rows * row_bytes));
    }
    return make_rsrc(static_cast<const uint8_t *>(base) + (int64_t)m0 * row_bytes,
                     clamp_bytes((int64_t)(p.M - m0) * row_bytes));
}

// In two steps: the row of A (with a row list: a load), and its offset.
template <int GR>
__device__ inline uint32_t row_index(const GemmArgs &p, int m0, int r)
{
    if constexpr (GR != 0) {
        if (p.rows)
            return m0 + r < p.M ? (uint32_t)p.rows[m0 + r] : 0xFFFFFFFFu;
    }
    return (uint32_t)r;
}
template <int GR>
__device__ inline uint32_t index_offset(const GemmArgs &p, uint32_t i, uint32_t row_bytes)
{
    if constexpr (GR != 0) {
        if (p.rows)
            return i < (uint32_t)p.a_rows ? i * row_bytes : kNoRow;
    }
    return i * row_bytes;
}
template <int GR>
__device__ inline uint32_t row_offset(const GemmArgs &p, int m0, int r, uint32_t row_bytes)
{
    return index_offset<GR>(p, row_index<GR>(p, m0, r), row_bytes);
}

// ------------------------------------------------------------ load ring
//
// ring_run<DEPTH>(n, load, consume) -- one wave's slice of n steps through a
// ring of DEPTH slots: load(d, i) issues step i's loads into slot d and
// consume(d, i) uses them, slot d = i % DEPTH (a compile-time index).  Loads
// run DEPTH steps ahead and are issued for steps < n only.  Every stretch of
// code is branch-free with loads and consumes in slot order (scheduling
// fences), so the compiler waits for exactly the slot a step needs: a loop
// whose iterations consume and refill DEPTH slots while at least 2*DEPTH
// steps remain, then one of 2*DEPTH straight-line tails chosen by the count
// left (a wave-uniform branch).

// The last t < 2*DEPTH steps from step i0; with PRE their first min(t, DEPTH)
// loads are issued here, else they are already in flight in slot order.
template <int DEPTH, int T, bool PRE, class Load, class Consume>
__device__ __attribute__((always_inline)) inline void ring_tail(int i0, Load &load, Consume &consume)
{
    constexpr int L = T < DEPTH ? T : DEPTH;
    if constexpr (PRE) {
#pragma unroll
        for (int d = 0; d < L; ++d) {
            load(d, i0 + d);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int d = 0; d < L; ++d) {
        consume(d, i0 + d);
        if constexpr (DEPTH < T) {
            if (d + DEPTH < T)   // compile-time after unrolling
                load(d, i0 + DEPTH + d);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int d = 0; d + DEPTH < T; ++d) {
        consume(d, i0 + DEPTH + d);
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int DEPTH, bool PRE, class Load, class Consume, int... Ts>
__device__ __attribute__((always_inline)) inline void ring_tail_of(int t, int i0, Load &load, Consume &consume, std::integer_sequence<int, Ts...>)
{
    ((t == Ts ? ring_tail<DEPTH, Ts, PRE>(i0, load, consume) : void()), ...);
}

template <int DEPTH, class Load, class Consume>
__device__ __attribute__((always_inline)) inline void ring_run(int n, Load &&load, Consume &&consume)
{
    using Counts = std::make_integer_sequence<int, 2 * DEPTH>;
    if (n < 2 * DEPTH) {
        ring_tail_of<DEPTH, true>(n, 0, load, consume, Counts{});
        return;
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
        load(d, d);
        __builtin_amdgcn_sched_barrier(0);
    }
    int i0 = 0;
    for (; i0 + 2 * DEPTH <= n; i0 += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            consume(d, i0 + d);
            load(d, i0 + DEPTH + d);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    ring_tail_of<DEPTH, false>(n - i0, i0, load, consume, Counts{});
}

// ------------------------------------------------------------- epilogue

template <int OUT>
__device__ inline void store_tile(const GemmArgs &p, int split, int m, int n, f32x4 v)
{
    if (m >= p.M || n >= p.N)
        return;
    if constexpr (OUT == kOutBf16) {
        u32x2 packed;
        packed.x = pack_bf16x2(v.x, v.y);
        packed.y = pack_bf16x2(v.z, v.w);
        *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(p.C) + ((int64_t)m * p.N + n) * 2) = packed;
    } else {
        *reinterpret_cast<f32x4 *>(p.ws + ((int64_t)split * p.M + m) * p.N + n) = v;
    }
}

// Per-wave counts of a TM x TN workgroup tile split over WM x WN waves, with
// KT-byte k-tiles (the tiled kernel families).
template <int DT, int TM, int TN, int WM, int WN, int KT>
struct TiledShape {
    static constexpr int kWaves = WM * WN;
    static constexpr int kThreads = kWaves * 64;
    static constexpr int kMT = TM / WM / 16;             // 16-row tiles per wave
    static constexpr int kNT = TN / WN / 16;             // 16-column strips per wave
    static constexpr int kCH = KT / 64;                  // 64-byte K chunks per k-tile
    static constexpr int kStepCh = Op<DT>::kBlocks;
    static constexpr int kSteps = kCH / kStepCh;         // MFMA k-steps per k-tile
    static constexpr int kABlocks = (TM / 16) * kCH;     // 1 KiB A blocks per k-tile
    static constexpr int kDmaPerWave = kABlocks / kWaves;
    static constexpr int kBufBytes = TM * KT;
    static constexpr int kBLoads = kNT * kCH;            // B loads per wave per k-tile
    static_assert(TM % (16 * WM) == 0 && TN % (16 * WN) == 0, "tile must split into 16x16 wave tiles");
    // The A-tile granularity rule of FlyDSL PR #974's follow-up commit (item 1):
    // the tile must split into whole 16-byte loads per thread, i.e.
    // TM*KT % (threads*16) == 0 -- with fewer loads the tail of the tile is
    // never fetched and the kernel computes on stale LDS.
    static_assert((TM * KT) % (kThreads * 16) == 0, "A tile must split into whole 16-byte loads");
    static_assert(kCH % kStepCh == 0, "k-tile must hold whole MFMA steps");
    static_assert(kCH <= 4, "B block offsets must fit the 12-bit immediate");
};

}  // namespace dgp
