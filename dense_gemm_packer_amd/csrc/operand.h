// Device helpers of the operators that read or write a product's operand:
// loads and stores of rows, reductions over lanes, scales and codes.
#pragma once

#include "common.h"

namespace dgp {

constexpr float kTop = 448.0f;                 // largest e4m3 value
constexpr uint32_t kInfBits = 0x7F800000u;

// ------------------------------------------------------------ input loads

// 8 consecutive elements in flight: their 16 (bf16, fp16) or 32 (fp32) bytes.
template <int XT>
struct Raw8 {
    i32x4 v[XT == kTypeF32 ? 2 : 1];
};

template <int XT>
__device__ inline Raw8<XT> load_raw8(const void *base, int64_t elem)
{
    Raw8<XT> r;
    const i32x4 *p = reinterpret_cast<const i32x4 *>(static_cast<const uint8_t *>(base) + elem * (XT == kTypeF32 ? 4 : 2));
    r.v[0] = p[0];
    if constexpr (XT == kTypeF32)
        r.v[1] = p[1];
    return r;
}

template <int XT>
__device__ inline void to_float8(const Raw8<XT> &r, float (&x)[8])
{
    if constexpr (XT == kTypeF32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = __builtin_bit_cast(float, (int)r.v[i / 4][i % 4]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = (uint32_t)r.v[0][i];
            if constexpr (XT == kDtypeBf16) {
                x[2 * i] = __builtin_bit_cast(float, w << 16);
                x[2 * i + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
            } else {
                x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)w);
                x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
            }
        }
    }
}

template <int XT>
__device__ inline void store8(void *base, int64_t elem, const float (&x)[8])
{
    i32x4 *p = reinterpret_cast<i32x4 *>(static_cast<uint8_t *>(base) + elem * (XT == kTypeF32 ? 4 : 2));
    if constexpr (XT == kTypeF32) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            p[h] = __builtin_bit_cast(i32x4, f32x4{x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]});
    } else {
        i32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (XT == kDtypeBf16) {
                v[i] = (int)pack_bf16x2(x[2 * i], x[2 * i + 1]);
            } else {
                const uint16_t lo = __builtin_bit_cast(uint16_t, (_Float16)x[2 * i]);
                const uint16_t hi = __builtin_bit_cast(uint16_t, (_Float16)x[2 * i + 1]);
                v[i] = (int)((uint32_t)lo | ((uint32_t)hi << 16));
            }
        }
        *p = v;
    }
}

// ------------------------------------------------------- block reductions

__device__ inline uint32_t mag_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }
__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int N>
__device__ inline uint32_t amax_bits(const float (&x)[N])
{
    uint32_t m = mag_bits(x[0]);
#pragma unroll
    for (int i = 1; i < N; ++i)
        m = umax(m, mag_bits(x[i]));
    return m;
}

template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kRowHalfMirror = 0x141, kRowMirror = 0x140;

// Maximum over groups of 4 or 16 consecutive lanes, in every lane of them.
__device__ inline uint32_t max4(uint32_t m)
{
    m = umax(m, dpp<kQuadXor1>(m));
    return umax(m, dpp<kQuadXor2>(m));
}
__device__ inline uint32_t max16(uint32_t m)
{
    m = max4(m);
    m = umax(m, dpp<kRowHalfMirror>(m));
    return umax(m, dpp<kRowMirror>(m));
}
__device__ inline uint32_t max64(uint32_t m)
{
    m = max16(m);
    m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
    return umax(m, (uint32_t)__shfl_xor((int)m, 32));
}
__device__ inline float fdpp_add(float s, uint32_t other) { return s + __builtin_bit_cast(float, other); }
__device__ inline float sum64(float s)
{
    s = fdpp_add(s, dpp<kQuadXor1>(__builtin_bit_cast(uint32_t, s)));
    s = fdpp_add(s, dpp<kQuadXor2>(__builtin_bit_cast(uint32_t, s)));
    s = fdpp_add(s, dpp<kRowHalfMirror>(__builtin_bit_cast(uint32_t, s)));
    s = fdpp_add(s, dpp<kRowMirror>(__builtin_bit_cast(uint32_t, s)));
    s += __shfl_xor(s, 16);
    return s + __shfl_xor(s, 32);
}

// The sum over the wave as a scalar, without a trip through LDS: rows of 16
// lanes, then rows 0 and 2 onto 1 and 3, then 1 onto 2 and 3; lane 63 has it.
__device__ inline float total64(float s)
{
    s = fdpp_add(s, dpp<kQuadXor1>(__builtin_bit_cast(uint32_t, s)));
    s = fdpp_add(s, dpp<kQuadXor2>(__builtin_bit_cast(uint32_t, s)));
    s = fdpp_add(s, dpp<kRowHalfMirror>(__builtin_bit_cast(uint32_t, s)));
    s = fdpp_add(s, dpp<kRowMirror>(__builtin_bit_cast(uint32_t, s)));
    s = fdpp_add(s, (uint32_t)__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), 0x142, 0xA, 0xF, false));   // row_bcast 15
    s = fdpp_add(s, (uint32_t)__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), 0x143, 0xC, 0xF, false));   // row_bcast 31
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s), 63));
}

// ----------------------------------------------------------------- scales

// fp32 scale of a block (NaN for a block that is not finite).
__device__ inline float scale_f32(uint32_t amax)
{
    if (amax >= kInfBits)
        return __builtin_bit_cast(float, 0x7FC00000u);
    return __builtin_fmaxf(__builtin_bit_cast(float, amax) / kTop, 0x1p-126f);
}

// E8M0 byte of a block: 448 = 1.75 * 2^8, so a mantissa above 1.75 (bits
// above 0x600000) carries into the exponent before 8 is taken off; 6 = 1.5 *
// 2^2, floor(log2) is the exponent itself.
template <int MODE>
__device__ inline int scale_e8m0(uint32_t amax)
{
    if (amax >= kInfBits)
        return 255;
    const int e = MODE == kScaleMx32 ? (int)(amax >> 23) - 2 : (int)((amax + 0x1FFFFFu) >> 23) - 8;
    return e > 0 ? e : 0;
}

// 2^(127 - e), what the block is multiplied by (e <= 253: a normal number);
// NaN for e = 255.
__device__ inline float e8m0_multiplier(int e)
{
    return __builtin_bit_cast(float, e == 255 ? 0x7FC00000u : (uint32_t)(254 - e) << 23);
}

// ------------------------------------------------------------------ codes

// 4 values -> 4 e4m3 codes (round to nearest even).  SAT: values above 448
// saturate (a NaN stays one); without it the caller's scale rules them out.
template <bool SAT>
__device__ inline uint32_t pack_e4m3(float a, float b, float c, float d)
{
    if constexpr (SAT) {
        auto sat = [](float v) { v = v > kTop ? kTop : v; return v < -kTop ? -kTop : v; };
        a = sat(a), b = sat(b), c = sat(c), d = sat(d);
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// 8 values -> 8 E2M1 codes, element 0 in the lowest nibble; |v| saturates
// at 6 (round to nearest even).
__device__ inline uint32_t pack_e2m1(const float *v)
{
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c[i] = __builtin_amdgcn_fmed3f(v[i], -6.0f, 6.0f);
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, c[0], c[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[2], c[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[4], c[5], 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[6], c[7], 1.0f, 3);
}

// Codes and scale of 8 elements y of a row whose block is the 16 (128
// blocks) or 4 (32 blocks) consecutive lanes around this one; `idx` = the
// element's index / 8 in the output.  tmul: the per-tensor multiplier 1/s.
template <int MODE, bool SAT>
__device__ inline void emit8(const float (&y)[8], int64_t idx, void *Q, void *S, float tmul)
{
    if constexpr (MODE == kScaleNone) {
        store8<kDtypeBf16>(Q, idx * 8, y);
    } else if constexpr (MODE == kScaleMx32) {
        const uint32_t m = max4(amax_bits(y));
        const int e = scale_e8m0<MODE>(m);
        const float f = e8m0_multiplier(e);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = y[i] * f;
        static_cast<uint32_t *>(Q)[idx] = e == 255 ? 0u : pack_e2m1(v);
        if ((threadIdx.x & 3) == 0)
            static_cast<uint8_t *>(S)[idx >> 2] = (uint8_t)e;
    } else {
        float f = tmul;
        if constexpr (MODE == kScaleBlock) {
            const float s = scale_f32(max16(amax_bits(y)));
            f = 1.0f / s;
            if ((threadIdx.x & 15) == 0)
                static_cast<float *>(S)[idx >> 4] = s;
        } else if constexpr (MODE == kScaleMx) {
            const int e = scale_e8m0<MODE>(max16(amax_bits(y)));
            f = e8m0_multiplier(e);
            if ((threadIdx.x & 15) == 0)
                static_cast<uint8_t *>(S)[idx >> 4] = (uint8_t)e;
        }
        u32x2 w;
        w.x = pack_e4m3<SAT>(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
        w.y = pack_e4m3<SAT>(y[4] * f, y[5] * f, y[6] * f, y[7] * f);
        static_cast<u32x2 *>(Q)[idx] = w;
    }
}

// ------------------------------------------------- kept activations, 8 bits

// 8 consecutive elements of a kept activation in flight: its own bytes, or
// e4m3 codes and the scale of their 128 block (fp32 bits; E8M0: the byte).
template <int XT, int MODE>
struct Kept8 {
    u32x2 codes;
    uint32_t scale;
};
template <int XT>
struct Kept8<XT, kScaleNone> {
    Raw8<XT> raw;
};

// Element `col` (a multiple of 8) of the row whose values or codes start at
// X + row * ld and whose block scales start at S + row * lds.
template <int XT, int MODE>
__device__ inline Kept8<XT, MODE> load_kept8(const void *X, const void *S, int64_t row, int64_t ld, int64_t lds, int col)
{
    Kept8<XT, MODE> k;
    if constexpr (MODE == kScaleNone) {
        k.raw = load_raw8<XT>(X, row * ld + col);
    } else {
        k.codes = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(X) + row * ld + col);
        if constexpr (MODE == kScaleMx)
            k.scale = static_cast<const uint8_t *>(S)[row * lds + col / 128];
        else
            k.scale = static_cast<const uint32_t *>(S)[MODE == kScaleBlock ? row * lds + col / 128 : 0];
    }
    return k;
}

// 2^(e - 127) for an E8M0 byte (255: NaN; 0: a subnormal fp32 number).
__device__ inline float e8m0_value(uint32_t e)
{
    return __builtin_bit_cast(float, e == 255u ? 0x7FC00000u : e == 0u ? 0x00400000u : e << 23);
}

template <int XT, int MODE>
__device__ inline void kept_floats(const Kept8<XT, MODE> &k, float (&x)[8])
{
    if constexpr (MODE == kScaleNone) {
        to_float8<XT>(k.raw, x);
    } else {
        const float s = MODE == kScaleMx ? e8m0_value(k.scale) : __builtin_bit_cast(float, k.scale);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)k.codes[h], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)k.codes[h], true);
            x[4 * h] = lo[0] * s, x[4 * h + 1] = lo[1] * s;
            x[4 * h + 2] = hi[0] * s, x[4 * h + 3] = hi[1] * s;
        }
    }
}

}  // namespace dgp
