// Gradient of the gated activation (dgp_swiglu_backward).  With s = 1 / (1 +
// exp(-g)), y = g s u, so
//
//   dg = dy u s (1 + g (1 - s)),   du = dy g s.
//
// 1 - s is exp(-g) s, which keeps its digits where s is near 1.  All arithmetic
// is fp32, rounded once to the gradients' type: at most 9 half steps of fp32 for
// du and 10 of |dy u s| (|g (1 - s)| + |1 + g (1 - s)|) for dg (gates below -80: 19 of
// either), whatever the gate's size.
#include "common.h"
#include "launch.h"
#include "operand.h"

namespace dgp {

namespace {

// exp(x) = 2^t (1 + r ln 2) with t the fp32 product x log2(e) and r what t is off
// by: 2^t alone is off by |x| half steps (16 391 x 2048 from mxfp8 41.3 us with r and
// 40.3 without, bf16 52.8 and 53.2, 8195 x 2048 fp32 58.8 and 57.9).  For finite x
// below where exp(x) is infinite.
__device__ inline float exponential(float x)
{
    constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f;   // log2(e) to 2^-50
    const float t = x * kLog2e;
    const float r = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -t));
    const float p = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(p, r * 0x1.62e43p-1f, p);
}

// For g >= -80 (see kFar).  exp(-g) is infinite nowhere in that range.
__device__ inline void grads(float dy, float g, float u, float &dg, float &du)
{
    // (exp(-200) is 0 as well, and infinity has no remainder)
    const float e = exponential(g > 200.0f ? -200.0f : -g), s = __builtin_amdgcn_rcpf(1.0f + e);
    const float a = dy * s;
    dg = a * u * __builtin_fmaf(g, e * s, 1.0f);
    du = a * g;
}

// Gates below -80: there s is exp(g) and 1 - s is 1 to 2^-115; exp(g) goes in
// as four factors exp(g / 4), between dy and u, so that with those of ordinary
// size no product leaves the normal range before the results do.
constexpr uint32_t kFar = 0xC2A00000u;     // -80.0f; more negative numbers have larger bits

template <int XT, int MODE>
__device__ inline void grads8(const float (&dy)[8], const float (&g)[8], const float (&u)[8], float (&dg)[8], float (&du)[8])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        top = umax(top, __builtin_bit_cast(uint32_t, g[i]));
        grads(dy[i], g[i], u[i], dg[i], du[i]);
    }
    if (top > kFar) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = exponential(0.25f * g[i]);
            const bool far = g[i] < -80.0f;
            dg[i] = far ? (1.0f + g[i]) * q * dy[i] * q * u[i] * q * q : dg[i];
            du[i] = far ? g[i] * q * dy[i] * q * q * q : du[i];
        }
    }
}

}  // namespace

// Thread = 8 consecutive elements of dy, gate and up.  HBM-bound: reads each
// once, writes both gradients once (16 391 x 2048 bf16, gate and up an mxfp8
// checkpoint: 269 MB in 41 us, 6.5 TB/s; 128 x 2048 in 2.9 us, a launch).
template <int XT, int MODE>
__global__ __launch_bounds__(256) void swiglu_grad_kernel(const SwigluGradArgs a)
{
    const uint32_t k8 = (uint32_t)(a.K / 8);
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    if (i >= (uint32_t)(a.M * (int64_t)k8))    // the launcher keeps it below 2^31
        return;
    const uint32_t row = i / k8;
    const int col = (int)((i - row * k8) * 8u);
    const auto ry = load_raw8<XT>(a.Y, (int64_t)row * a.ldy + col);
    const auto rg = load_kept8<XT, MODE>(a.G, a.SG, row, a.ldg, a.ldsg, col);
    const auto ru = load_kept8<XT, MODE>(a.U, a.SU, row, a.ldu, a.ldsu, col);
    float y[8], g[8], u[8], dg[8], du[8];
    to_float8<XT>(ry, y);
    kept_floats<XT, MODE>(rg, g);
    kept_floats<XT, MODE>(ru, u);
    grads8<XT, MODE>(y, g, u, dg, du);
    const int64_t o = (int64_t)row * (2 * a.K) + col;
    store8<XT>(a.D, o, dg);
    store8<XT>(a.D, o + a.K, du);
}

template <int XT, int MODE>
static hipError_t launch_typed(const SwigluGradArgs &a, hipStream_t s)
{
    // Slabs of rows whose piece count fits 31 bits (a slab is one launch).
    const int64_t k8 = a.K / 8, slab = (int64_t(1) << 31) / k8 - 1;
    constexpr int64_t kIn = XT == kTypeF32 ? 4 : 2, kKept = MODE == kScaleNone ? kIn : 1;
    constexpr int64_t kScale = MODE == kScaleBlock ? 4 : MODE == kScaleMx ? 1 : 0;
    auto at = [](const void *p, int64_t bytes) { return static_cast<const void *>(static_cast<const uint8_t *>(p) + bytes); };
    for (int64_t r = 0; r < a.M; r += slab) {
        SwigluGradArgs b = a;
        b.M = a.M - r < slab ? a.M - r : slab;
        b.Y = at(a.Y, r * a.ldy * kIn);
        b.G = at(a.G, r * a.ldg * kKept), b.U = at(a.U, r * a.ldu * kKept);
        if (kScale)
            b.SG = at(a.SG, r * a.ldsg * kScale), b.SU = at(a.SU, r * a.ldsu * kScale);
        b.D = static_cast<uint8_t *>(a.D) + r * 2 * a.K * kIn;
        swiglu_grad_kernel<XT, MODE><<<(unsigned)((b.M * k8 + 255) / 256), 256, 0, s>>>(b);
    }
    return hipGetLastError();
}

template <int XT>
static hipError_t launch_mode(const SwigluGradArgs &a, int mode, hipStream_t s)
{
    switch (mode) {
    case kScaleNone: return launch_typed<XT, kScaleNone>(a, s);
    case kScaleTensor: return launch_typed<XT, kScaleTensor>(a, s);
    case kScaleBlock: return launch_typed<XT, kScaleBlock>(a, s);
    case kScaleMx: return launch_typed<XT, kScaleMx>(a, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_swiglu_grad(const SwigluGradArgs &a, int type, int mode, hipStream_t s)
{
    switch (type) {
    case kDtypeBf16: return launch_mode<kDtypeBf16>(a, mode, s);
    case kTypeF16: return launch_mode<kTypeF16>(a, mode, s);
    case kTypeF32: return launch_mode<kTypeF32>(a, mode, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dgp
