// Operators that write a GEMM operand: quantisation of activations and of
// weights, the root-mean-square norm (with the residual's addition) and the
// gated activation, each with its result in one of the operand forms of
// include/dgp.h (dgp_quantize and the entry points after it).
//
// All arithmetic is fp32.  The one rounding to fewer bits is the output's:
// e4m3, E2M1 or bf16, to nearest even (and the residual stream's own type).
//
// Scales.  With amax the largest magnitude of a block:
//   fp32 (per tensor, 128 blocks): s = max(amax / 448, 2^-126), codes
//     e4m3(x * (1 / s)); the lower bound keeps 1/s finite and gives an
//     all-zero block the codes 0.
//   E8M0, 128 blocks of e4m3: the smallest power of two with amax <= 448 *
//     2^(e-127): e4m3's relative step is the same at every exponent, so the
//     larger scale costs no precision where the next smaller one would
//     saturate the block's largest values.
//   E8M0, 32 blocks of E2M1: 2^(floor(log2 amax) - 2), values above 6
//     saturate (OCP MX 1.0, 6.3): with one mantissa bit the larger scale
//     would cost every other value of the block a bit.
// A block that holds a NaN or an infinity gets a NaN scale.  Magnitudes are
// compared as integers (the bits of |x|), which orders NaN above infinity
// above every finite value.
#include "common.h"
#include "launch.h"

namespace dgp {

namespace {

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

// silu(g) * u = g / (1 + exp(-g)) * u, for g >= -80: 1 + exp(-g) and its
// reciprocal (which gives no subnormal numbers) stay in the normal range.
// exp is exp2 of one fp32 product, whose rounding puts up to 2 |g| half steps of
// fp32 on the result (2.4e-6 at g = -20, where bf16's half step is 4e-3).  With
// the product's remainder added it would be a step or two at every g, and cost
// 2 to 7 % (16 391 x 2048 bf16 to mxfp8 32.0 us for 30.8, 4096 x 2048 to fp32
// block scales 11.0 for 10.2).
__device__ inline float swiglu(float g, float u)
{
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Gates below -80: there 1 + exp(-g) is exp(-g) to 2^-115, and the result is
// g exp(g) u, in four factors exp(g / 4), so that no product on the way leaves
// the normal range before the result does.  The largest bits of |g| < 0 among a
// thread's gates say if it has any (four instructions for 8 gates; a wave that
// has none skips the rest: 16 391 x 2048 bf16 to mxfp8 30.9 us, 30.7 without).
constexpr uint32_t kFarGate = 0xC2A00000u;     // -80.0f; more negative numbers have larger bits
template <int XT>
__device__ inline void swiglu8(const Raw8<XT> &rg, const Raw8<XT> &ru, float (&y)[8])
{
    float g[8], u[8];
    to_float8<XT>(rg, g);
    to_float8<XT>(ru, u);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        top = umax(top, __builtin_bit_cast(uint32_t, g[j]));
        y[j] = swiglu(g[j], u[j]);
    }
    if (top > kFarGate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = __expf(0.25f * g[j]);
            y[j] = g[j] < -80.0f ? g[j] * q * u[j] * q * q * q : y[j];
        }
    }
}

// The tensor's scale from the per-workgroup maxima of amax_kernel, by a whole
// workgroup of 256 threads (kAmaxParts <= 256 parts).
__device__ inline float tensor_scale(const uint32_t *parts, int n)
{
    __shared__ uint32_t red[4];
    uint32_t m = (int)threadIdx.x < n ? parts[threadIdx.x] : 0u;
    m = max64(m);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = m;
    __syncthreads();
    return scale_f32(umax(umax(red[0], red[1]), umax(red[2], red[3])));
}

}  // namespace

// ---------------------------------------------------------- row operators

// Elementwise operators (quantisation; the gated activation): thread = 8
// consecutive elements, so a 128 block is 16 lanes and its maximum four DPP
// steps.  Reads each input once, writes codes and scales once: HBM-bound
// (4096 x 8192 bf16 to e4m3 and fp32 block scales: 16.7 us, 6.1 TB/s; the gated
// activation of 16 391 x 2048 to mxfp8: 30 us, 5.6 TB/s).
template <int XT, int MODE, bool GATED, int U>
__global__ __launch_bounds__(256) void row_quant_kernel(const RowQuantArgs a)
{
    const uint32_t k8 = (uint32_t)(a.K / 8);
    const uint32_t total = (uint32_t)(a.M * (int64_t)k8);    // the launcher keeps it below 2^31
    const uint32_t base = blockIdx.x * (256u * U) + threadIdx.x;
    const bool flat = a.ldx == a.K && (!GATED || a.ldu == a.K);
    Raw8<XT> rx[U];
    [[maybe_unused]] Raw8<XT> ru[GATED ? U : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = base + u * 256u;
        if (i < total) {
            int64_t ox, ou;
            if (flat) {
                ox = ou = (int64_t)i * 8;
            } else {
                const uint32_t row = i / k8, col = (i - row * k8) * 8u;
                ox = (int64_t)row * a.ldx + col;
                ou = (int64_t)row * a.ldu + col;
            }
            rx[u] = load_raw8<XT>(a.X, ox);
            if constexpr (GATED)
                ru[u] = load_raw8<XT>(a.U, ou);
        }
    }
    float tmul = 1.0f;
    if constexpr (MODE == kScaleTensor) {
        if (a.parts) {
            const float s = tensor_scale(a.parts, a.nparts);
            tmul = 1.0f / s;
            if (blockIdx.x == 0 && threadIdx.x == 0)
                static_cast<float *>(a.S)[0] = s;
        } else {
            tmul = 1.0f / a.scale[0];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = base + u * 256u;
        if (i < total) {
            float y[8];
            if constexpr (GATED)
                swiglu8<XT>(rx[u], ru[u], y);
            else
                to_float8<XT>(rx[u], y);
            emit8<MODE, MODE == kScaleTensor>(y, i, a.Q, a.S, tmul);
        }
    }
}

// Per-tensor quantisation of a small matrix in one launch: one workgroup holds
// it all in registers between the maximum and the codes.  16 x 4096 (the most
// it takes; bf16 and fp32 alike) 5.8 us in a captured graph and 5.4 a call,
// where two launches take 4.9 and 6.5 at 16 x 4224; 16 x 2048 4.1 and 3.8.
constexpr int kSmallTensor = 65536;
template <int XT>
__global__ __launch_bounds__(1024) void small_tensor_quant_kernel(const RowQuantArgs a)
{
    constexpr int U = kSmallTensor / 8 / 1024;
    const uint32_t k8 = (uint32_t)(a.K / 8), total = (uint32_t)a.M * k8;
    Raw8<XT> r[U];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = threadIdx.x + u * 1024u;
        if (i < total) {
            const uint32_t row = i / k8, col = (i - row * k8) * 8u;
            r[u] = load_raw8<XT>(a.X, (int64_t)row * a.ldx + col);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (threadIdx.x + u * 1024u < total) {
            float x[8];
            to_float8<XT>(r[u], x);
            m = umax(m, amax_bits(x));
        }
    }
    __shared__ uint32_t red[16];
    m = max64(m);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < 16; ++w)
        m = umax(m, red[w]);
    const float s = scale_f32(m), f = 1.0f / s;
    if (threadIdx.x == 0)
        static_cast<float *>(a.S)[0] = s;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = threadIdx.x + u * 1024u;
        if (i < total) {
            float x[8];
            to_float8<XT>(r[u], x);
            emit8<kScaleTensor, false>(x, i, a.Q, a.S, f);
        }
    }
}

// Largest magnitude of a matrix (of each of gridDim.y stacked ones), one
// partial per workgroup: parts[group][gridDim.x].  The maximum is taken in
// integers, so the order of the partials never matters.  HBM-bound: with it a
// measured scale costs 34 us for 4096 x 8192 bf16 (20 with block scales, inputs
// not in cache; a read at 7.2 TB/s and a copy at 4.95: 30), and a weight of
// 16384 x 7168 fp32 184 us (105 to mxfp8; 184).
template <int XT>
__global__ __launch_bounds__(256) void amax_kernel(const void *X, int64_t ldx, int64_t M, int64_t K, uint32_t *parts)
{
    const int64_t k8 = K / 8, total = M * k8;
    const int64_t first = (int64_t)blockIdx.y * M;           // first row of the group
    const bool flat = ldx == K;
    uint32_t m = 0;
    constexpr int U = 4;
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x; i0 < total; i0 += stride * U) {
        Raw8<XT> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * stride;
            const int64_t j = i < total ? i : i0;            // past the end: the thread's first piece again
            if (flat) {
                r[u] = load_raw8<XT>(X, first * K + j * 8);
            } else {
                const int64_t row = j / k8;
                r[u] = load_raw8<XT>(X, (first + row) * ldx + (j - row * k8) * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[8];
            to_float8<XT>(r[u], x);
            m = umax(m, amax_bits(x));
        }
    }
    __shared__ uint32_t red[4];
    m = max64(m);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0)
        parts[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = umax(umax(red[0], red[1]), umax(red[2], red[3]));
}

// ---------------------------------------------------------------- weights

// Weight quantisation straight into the preshuffled layout (dgp_preshuffle_b).
// A wave owns 16 rows x 128 code bytes = two 1 KiB operand blocks; lane l
// makes the 16 bytes of row l % 16, piece l / 16 of each, which it stores as
// one 16-byte piece at byte 16 l of the block.  A row's 128-element e4m3
// block is then the four lanes l, l + 16, l + 32, l + 48; an E2M1 piece is
// one whole 32-element block.  fp32 128 x 128 scales: eight waves own the 128
// rows and join their maxima in LDS.  HBM-bound; reads B once (twice per
// tensor scale), writes codes and scales once (16384 x 7168 fp32 to mxfp8: 102
// us, 5.7 TB/s).
template <int XT, int MODE>
__global__ __launch_bounds__(MODE == kScaleBlock ? 512 : 256) void quantize_b_kernel(const WeightQuantArgs a)
{
    constexpr int kWaves = MODE == kScaleBlock ? 8 : 4;
    constexpr int kPer = MODE == kScaleMx32 ? 32 : 16;       // elements per 16-byte piece
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t cols = (uint32_t)(a.K / (8 * kPer));      // 128-byte column units per row
    // unit = (16-row strip, column unit); the waves of a 128 x 128 block take
    // its 8 strips, elsewhere four consecutive units of the row-major order
    uint32_t strip, cu;
    if constexpr (MODE == kScaleBlock) {
        strip = (blockIdx.x / cols) * 8 + wave;
        cu = blockIdx.x % cols;
    } else {
        const uint32_t unit = blockIdx.x * 4 + wave;
        strip = unit / cols;
        cu = unit % cols;
    }
    const bool live = strip < (uint32_t)(a.rows / 16);
    const int64_t row = (int64_t)strip * 16 + (lane & 15);
    float x[2][kPer];
    if (live) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < kPer / 8; ++q) {
                float v[8];
                to_float8<XT>(load_raw8<XT>(a.B, row * a.K + (int64_t)cu * (8 * kPer) + j * (4 * kPer) +
                                                     (lane >> 4) * kPer + q * 8), v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[j][q * 8 + i] = v[i];
            }
    }
    float f[2] = {1.0f, 1.0f};
    int e[2] = {0, 0};
    if constexpr (MODE == kScaleTensor) {
        // the four waves' strips may lie in two matrices of the stack: each
        // takes the scale of its own
        const uint32_t g = live ? (uint32_t)(strip / (uint32_t)(a.N / 16)) : 0u;
        uint32_t m = 0;
        for (int i = lane; i < a.nparts; i += 64)
            m = umax(m, a.parts[(int64_t)g * a.nparts + i]);
        const float s = scale_f32(max64(m));
        f[0] = f[1] = 1.0f / s;
        if (live && cu == 0 && strip % (uint32_t)(a.N / 16) == 0 && lane == 0)
            static_cast<float *>(a.S)[g] = s;
    } else if constexpr (MODE == kScaleBlock) {
        __shared__ uint32_t red[kWaves];
        uint32_t m = live ? umax(amax_bits(x[0]), amax_bits(x[1])) : 0u;
        m = max64(m);
        if (lane == 0)
            red[wave] = m;
        __syncthreads();
        m = red[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            m = umax(m, red[w]);
        const float s = scale_f32(m);
        f[0] = f[1] = 1.0f / s;
        if (threadIdx.x == 0)
            static_cast<float *>(a.S)[(int64_t)(strip / 8) * cols + cu] = s;
    } else if constexpr (MODE == kScaleMx) {
        uint32_t m = live ? umax(amax_bits(x[0]), amax_bits(x[1])) : 0u;
        m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
        m = umax(m, (uint32_t)__shfl_xor((int)m, 32));
        e[0] = scale_e8m0<MODE>(m);
        f[0] = f[1] = e8m0_multiplier(e[0]);
        if (live && lane < 16)
            static_cast<uint8_t *>(a.S)[row * cols + cu] = (uint8_t)e[0];
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            e[j] = scale_e8m0<MODE>(live ? amax_bits(x[j]) : 0u);
            f[j] = e8m0_multiplier(e[j]);
            if (live)   // 8 blocks of 32 per column unit
                static_cast<uint8_t *>(a.S)[(row * cols + cu) * 8 + j * 4 + (lane >> 4)] = (uint8_t)e[j];
        }
    }
    if (!live)
        return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        i32x4 w;
        if constexpr (MODE == kScaleMx32) {
            float v[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                v[i] = x[j][i] * f[j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = e[j] == 255 ? 0 : (int)pack_e2m1(v + 8 * i);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (int)pack_e4m3<false>(x[j][4 * i] * f[j], x[j][4 * i + 1] * f[j], x[j][4 * i + 2] * f[j],
                                             x[j][4 * i + 3] * f[j]);
        }
        // block (strip, 2 cu + j) of Kb / 64 = 2 cols blocks per strip
        *reinterpret_cast<i32x4 *>(static_cast<uint8_t *>(a.Q) +
                                   ((int64_t)strip * (2 * cols) + 2 * cu + j) * 1024 + lane * 16) = w;
    }
}

// ------------------------------------------------------------------- norm

// y = h / sqrt(mean(h^2) + eps) * w with h = x (+ residual), the sum taken
// and kept in fp32; the residual stream is written back in the input's type.
// T threads own a row (256 / T rows per workgroup where T < 256), C pieces of
// 8 elements each, kept in registers between the two uses.  C = 0: rows longer
// than the registers hold are read again for the second use.  HBM-bound: each
// input is read and each output written once (4096 x 8192 bf16 with residual,
// e4m3 codes and fp32 block scales: 235 MB in 47 us, 5.0 TB/s, the rate of a
// copy; one row of 7168 to mxfp8: 3.1 us, the latency of one workgroup).
template <int XT, int MODE, int T, int C>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rmsnorm_kernel(const NormArgs a)
{
    constexpr int kThreads = T < 256 ? 256 : T;
    constexpr int kWaves = T / 64;
    const int t = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / T) + threadIdx.x / T;
    if (T < 256 && row >= a.M)       // whole waves; no barrier follows for T = 64
        return;
    const int k8 = (int)(a.K / 8);
    auto load_h = [&](int c, float(&h)[8]) {
        to_float8<XT>(load_raw8<XT>(a.X, row * a.ldx + c * 8), h);
        if (a.R) {
            float r[8];
            to_float8<XT>(load_raw8<XT>(a.R, row * a.ldr + c * 8), r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[i] += r[i];
        }
    };
    float h[C > 0 ? C : 1][8];
    float ss = 0.0f;
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (t + c * T < k8)
                load_h(t + c * T, h[c]);
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (t + c * T < k8) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ss = __builtin_fmaf(h[c][i], h[c][i], ss);
            }
    } else {
        for (int c = t; c < k8; c += T) {
            load_h(c, h[0]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss = __builtin_fmaf(h[0][i], h[0][i], ss);
        }
    }
    ss = sum64(ss);
    if constexpr (kWaves > 1) {
        __shared__ float red[kWaves];
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = ss;
        __syncthreads();
        ss = red[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            ss += red[w];
    }
    const float rstd = 1.0f / __builtin_sqrtf(ss / (float)a.K + a.eps);
    float tmul = 1.0f;
    if constexpr (MODE == kScaleTensor)
        tmul = 1.0f / a.scale[0];
    auto finish = [&](int c, float(&v)[8]) {
        if (a.H)
            store8<XT>(a.H, row * a.K + c * 8, v);
        float w[8];
        if (a.wt == kTypeF32)
            to_float8<kTypeF32>(load_raw8<kTypeF32>(a.W, (int64_t)c * 8), w);
        else
            to_float8<XT>(load_raw8<XT>(a.W, (int64_t)c * 8), w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = v[i] * rstd * w[i];
        emit8<MODE, MODE == kScaleTensor>(v, row * (int64_t)k8 + c, a.Q, a.S, tmul);
    };
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (t + c * T < k8)
                finish(t + c * T, h[c]);
    } else {
        for (int c = t; c < k8; c += T) {
            load_h(c, h[0]);
            finish(c, h[0]);
        }
    }
}

// --------------------------------------------------------------- launches

template <int XT, int MODE, bool GATED>
static hipError_t launch_rows(RowQuantArgs a, hipStream_t s)
{
    // Pieces per thread: the gated activation has two loads a piece already (128
    // x 2048: one 2.1 us, two 2.6; 4096 x 2048: 10.0, 11.0); quantisation of
    // 4096 x 8192: one 19.9, two 18.8, four 20.0 us, of 16 x 7168: 2.0, 2.2, 2.9.
    constexpr int U = GATED ? 1 : 2;
    // Slabs of rows whose piece count fits 32 bits (a slab is one launch).
    const int64_t k8 = a.K / 8;
    const int64_t slab = (int64_t(1) << 31) / k8 - 1;
    const int64_t M = a.M;
    constexpr int kIn = XT == kTypeF32 ? 4 : 2;
    const int64_t blk = MODE == kScaleMx32 ? 32 : 128, ssz = MODE == kScaleBlock ? 4 : 1;
    for (int64_t r = 0; r < M; r += slab) {
        RowQuantArgs b = a;
        b.M = M - r < slab ? M - r : slab;
        b.X = static_cast<const uint8_t *>(a.X) + r * a.ldx * kIn;
        if (GATED)
            b.U = static_cast<const uint8_t *>(a.U) + r * a.ldu * kIn;
        b.Q = static_cast<uint8_t *>(a.Q) + (MODE == kScaleNone ? 2 * r * a.K : MODE == kScaleMx32 ? r * a.K / 2 : r * a.K);
        if (MODE != kScaleNone && MODE != kScaleTensor)
            b.S = static_cast<uint8_t *>(a.S) + r * (a.K / blk) * ssz;
        const unsigned grid = (unsigned)((b.M * k8 + 256 * U - 1) / (256 * U));
        row_quant_kernel<XT, MODE, GATED, U><<<grid, 256, 0, s>>>(b);
    }
    return hipGetLastError();
}

template <int XT, bool GATED>
static hipError_t launch_rows_mode(const RowQuantArgs &a, int mode, hipStream_t s)
{
    switch (mode) {
    case kScaleNone:
        if constexpr (GATED)
            return launch_rows<XT, kScaleNone, GATED>(a, s);
        return hipErrorInvalidValue;
    case kScaleTensor: return launch_rows<XT, kScaleTensor, GATED>(a, s);
    case kScaleBlock: return launch_rows<XT, kScaleBlock, GATED>(a, s);
    case kScaleMx: return launch_rows<XT, kScaleMx, GATED>(a, s);
    case kScaleMx32: return launch_rows<XT, kScaleMx32, GATED>(a, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_row_quant(const RowQuantArgs &a, int x_type, int mode, bool gated, hipStream_t s)
{
    switch (x_type) {
    case kDtypeBf16: return gated ? launch_rows_mode<kDtypeBf16, true>(a, mode, s) : launch_rows_mode<kDtypeBf16, false>(a, mode, s);
    case kTypeF16: return gated ? launch_rows_mode<kTypeF16, true>(a, mode, s) : launch_rows_mode<kTypeF16, false>(a, mode, s);
    case kTypeF32: return gated ? launch_rows_mode<kTypeF32, true>(a, mode, s) : launch_rows_mode<kTypeF32, false>(a, mode, s);
    default: return hipErrorInvalidValue;
    }
}

bool small_tensor(int64_t M, int64_t K) { return M * K <= kSmallTensor; }

hipError_t launch_small_tensor_quant(const RowQuantArgs &a, int x_type, hipStream_t s)
{
    switch (x_type) {
    case kDtypeBf16: small_tensor_quant_kernel<kDtypeBf16><<<1, 1024, 0, s>>>(a); break;
    case kTypeF16: small_tensor_quant_kernel<kTypeF16><<<1, 1024, 0, s>>>(a); break;
    case kTypeF32: small_tensor_quant_kernel<kTypeF32><<<1, 1024, 0, s>>>(a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

hipError_t launch_amax(const void *X, int64_t ldx, int x_type, int64_t groups, int64_t M, int64_t K, int parts_per_group,
                       uint32_t *parts, hipStream_t s)
{
    const dim3 grid((unsigned)parts_per_group, (unsigned)groups);
    switch (x_type) {
    case kDtypeBf16: amax_kernel<kDtypeBf16><<<grid, 256, 0, s>>>(X, ldx, M, K, parts); break;
    case kTypeF16: amax_kernel<kTypeF16><<<grid, 256, 0, s>>>(X, ldx, M, K, parts); break;
    case kTypeF32: amax_kernel<kTypeF32><<<grid, 256, 0, s>>>(X, ldx, M, K, parts); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int XT, int MODE>
static void launch_qb(const WeightQuantArgs &a, hipStream_t s)
{
    const int64_t cols = a.K / (MODE == kScaleMx32 ? 256 : 128);
    if constexpr (MODE == kScaleBlock)
        quantize_b_kernel<XT, MODE><<<(unsigned)(a.rows / 128 * cols), 512, 0, s>>>(a);
    else
        quantize_b_kernel<XT, MODE><<<(unsigned)((a.rows / 16 * cols + 3) / 4), 256, 0, s>>>(a);
}

hipError_t launch_quantize_b(const WeightQuantArgs &a, int x_type, int mode, hipStream_t s)
{
    auto typed = [&](auto xt) {
        constexpr int XT = decltype(xt)::value;
        switch (mode) {
        case kScaleTensor: launch_qb<XT, kScaleTensor>(a, s); return hipGetLastError();
        case kScaleBlock: launch_qb<XT, kScaleBlock>(a, s); return hipGetLastError();
        case kScaleMx: launch_qb<XT, kScaleMx>(a, s); return hipGetLastError();
        case kScaleMx32: launch_qb<XT, kScaleMx32>(a, s); return hipGetLastError();
        default: return hipErrorInvalidValue;
        }
    };
    switch (x_type) {
    case kDtypeBf16: return typed(std::integral_constant<int, kDtypeBf16>{});
    case kTypeF16: return typed(std::integral_constant<int, kTypeF16>{});
    case kTypeF32: return typed(std::integral_constant<int, kTypeF32>{});
    default: return hipErrorInvalidValue;
    }
}

template <int XT, int MODE, int T, int C>
static void launch_norm_rows(const NormArgs &a, hipStream_t s)
{
    constexpr int kThreads = T < 256 ? 256 : T, kRows = kThreads / T;
    constexpr int kIn = XT == kTypeF32 ? 4 : 2;
    // Slabs of rows whose threads fit the 32 bits of a launch.
    constexpr int64_t slab = (int64_t(1) << 31) / T;
    const int64_t qrow = MODE == kScaleNone ? 2 * a.K : MODE == kScaleMx32 ? a.K / 2 : a.K;
    const int64_t srow = MODE == kScaleBlock ? a.K / 128 * 4 : MODE == kScaleMx ? a.K / 128 : MODE == kScaleMx32 ? a.K / 32 : 0;
    for (int64_t r = 0; r < a.M; r += slab) {
        NormArgs b = a;
        b.M = a.M - r < slab ? a.M - r : slab;
        b.X = static_cast<const uint8_t *>(a.X) + r * a.ldx * kIn;
        if (a.R)
            b.R = static_cast<const uint8_t *>(a.R) + r * a.ldr * kIn;
        if (a.H)
            b.H = static_cast<uint8_t *>(a.H) + r * a.K * kIn;
        b.Q = static_cast<uint8_t *>(a.Q) + r * qrow;
        if (srow)
            b.S = static_cast<uint8_t *>(a.S) + r * srow;
        rmsnorm_kernel<XT, MODE, T, C><<<(unsigned)((b.M + kRows - 1) / kRows), kThreads, 0, s>>>(b);
    }
}

// Threads per row and pieces per thread by the row's length: one or two pieces
// each keep the row's latency short and leave registers for many workgroups
// (us for rows of bf16 with a residual, fp32 block scales out; "a/b" = T/C):
//   1024: 256/1 2.6 and 64/2 3.2 for one row, 61 and 54 for 39 062
//   2048: 256/1 2.7, 14.2, 51 for 1, 4096, 19 531 rows (64/4: 16.3, 61 for the latter two)
//   4096: 512/1 2.9, 25.0, 51 for 1, 4096, 9765 rows (1024/1: 2.9, 30, 66)
//   7168: 1024/1 3.3, 5.2, 9.6 and 512/2 3.6, 5.6, 9.0 for 1, 256, 600 rows
//   (4096 x 8192: 512/2 47.2, 256/4 52.8)
// Just past a border up to half of the threads hold nothing (1237 x 2112 fp16 to
// bf16, 264 pieces on 512 threads: 4.3 us where a copy's rate gives 2.1).  fp32
// rows and other outputs take the same rule, which was not measured on them.
template <int XT, int MODE>
static void launch_norm(const NormArgs &a, hipStream_t s)
{
    const int64_t k8 = a.K / 8;
    if (k8 <= 64)
        launch_norm_rows<XT, MODE, 64, 1>(a, s);
    else if (k8 <= 128 && a.M > 8192)
        launch_norm_rows<XT, MODE, 64, 2>(a, s);
    else if (k8 <= 256)
        launch_norm_rows<XT, MODE, 256, 1>(a, s);
    else if (k8 <= 512)
        launch_norm_rows<XT, MODE, 512, 1>(a, s);
    else if (k8 <= 1024 && a.M > 384)
        launch_norm_rows<XT, MODE, 512, 2>(a, s);
    else if (k8 <= 1024)
        launch_norm_rows<XT, MODE, 1024, 1>(a, s);
    else if (k8 <= 4096)
        launch_norm_rows<XT, MODE, 1024, 4>(a, s);
    else
        launch_norm_rows<XT, MODE, 1024, 0>(a, s);
}

hipError_t launch_rmsnorm(const NormArgs &a, int x_type, int mode, hipStream_t s)
{
    auto typed = [&](auto xt) {
        constexpr int XT = decltype(xt)::value;
        switch (mode) {
        case kScaleNone: launch_norm<XT, kScaleNone>(a, s); return hipGetLastError();
        case kScaleTensor: launch_norm<XT, kScaleTensor>(a, s); return hipGetLastError();
        case kScaleBlock: launch_norm<XT, kScaleBlock>(a, s); return hipGetLastError();
        case kScaleMx: launch_norm<XT, kScaleMx>(a, s); return hipGetLastError();
        case kScaleMx32: launch_norm<XT, kScaleMx32>(a, s); return hipGetLastError();
        default: return hipErrorInvalidValue;
        }
    };
    switch (x_type) {
    case kDtypeBf16: return typed(std::integral_constant<int, kDtypeBf16>{});
    case kTypeF16: return typed(std::integral_constant<int, kTypeF16>{});
    case kTypeF32: return typed(std::integral_constant<int, kTypeF32>{});
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dgp
