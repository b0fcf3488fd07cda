// The norms that write a product's operand: the kernel and its launch rule,
// instantiated for the root-mean-square norm in quantize.hip and for the layer
// norm in layernorm.hip.
#pragma once

#include "launch.h"
#include "operand.h"

namespace dgp {

// Sums of N values over the T threads of a row (64: one wave), in every thread.
// `red` holds N x T / 64 partial sums in LDS; a second call takes another array.
// (TOTAL: without LDS inside a wave, in another order; one row of 7168 to mxfp8
// with two such sums 3.3 us.)
template <int T, bool TOTAL, int N>
__device__ inline void row_sums(float (&v)[N], float (*red)[T / 64])
{
#pragma unroll
    for (int n = 0; n < N; ++n)
        v[n] = TOTAL ? total64(v[n]) : sum64(v[n]);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                red[n][threadIdx.x >> 6] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = red[n][0];
#pragma unroll
            for (int w = 1; w < T / 64; ++w)
                v[n] += red[n][w];
        }
    }
}

// LN = false: y = h / sqrt(mean(h^2) + eps) * w, with h = x (+ residual), the sum taken
// and kept in fp32; the residual stream is written back in the input's type.
// LN = true: y = (h - mean) / sqrt(var + eps) * w + b.  The variance is a sum of
// squares about the mean (the row is in registers, so a second reduction costs
// no memory), and what the fp32 mean is off by, the mean of h - mean, is taken
// out of both: rows far from zero keep their digits.
// T threads own a row (256 / T rows per workgroup where T < 256), C pieces of
// 8 elements each, kept in registers between the uses.  C = 0: rows longer
// than the registers hold are read again for each use.  HBM-bound: each
// input is read and each output written once (4096 x 8192 bf16 with residual,
// e4m3 codes and fp32 block scales: 235 MB in 47 us, 5.0 TB/s, the rate of a
// copy; one row of 7168 to mxfp8: 3.1 us, the latency of one workgroup).
template <int XT, int MODE, int T, int C, bool LN>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_kernel(const NormArgs a)
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
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (t + c * T < k8)
                load_h(t + c * T, h[c]);
    }
    // f(8 elements of the row) for every piece of this thread
    auto each = [&](auto f) {
        if constexpr (C > 0) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t + c * T < k8)
                    f(h[c]);
        } else {
            for (int c = t; c < k8; c += T) {
                load_h(c, h[0]);
                f(h[0]);
            }
        }
    };
    [[maybe_unused]] float mean = 0.0f, rest = 0.0f;
    float rstd;
    if constexpr (LN) {
        __shared__ float red1[1][kWaves], red2[2][kWaves];
        float s1[1] = {0.0f};
        each([&](const float(&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s1[0] += v[i];
        });
        row_sums<T, true>(s1, red1);
        mean = s1[0] / (float)a.K;
        float s2[2] = {0.0f, 0.0f};
        each([&](const float(&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = v[i] - mean;
                s2[0] += d;
                s2[1] = __builtin_fmaf(d, d, s2[1]);
            }
        });
        row_sums<T, true>(s2, red2);
        rest = s2[0] / (float)a.K;
        const float var = s2[1] / (float)a.K - rest * rest;
        rstd = 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + a.eps);    // (a NaN stays one)
    } else {
        __shared__ float red[1][kWaves];
        float ss[1] = {0.0f};
        each([&](const float(&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss[0] = __builtin_fmaf(v[i], v[i], ss[0]);
        });
        row_sums<T, false>(ss, red);
        rstd = 1.0f / __builtin_sqrtf(ss[0] / (float)a.K + a.eps);
    }
    float tmul = 1.0f;
    if constexpr (MODE == kScaleTensor)
        tmul = 1.0f / a.scale[0];
    auto load_w = [&](const void *p, int c, float(&w)[8]) {
        if (a.wt == kTypeF32)
            to_float8<kTypeF32>(load_raw8<kTypeF32>(p, (int64_t)c * 8), w);
        else
            to_float8<XT>(load_raw8<XT>(p, (int64_t)c * 8), w);
    };
    auto finish = [&](int c, float(&v)[8]) {
        if (a.H)
            store8<XT>(a.H, row * a.K + c * 8, v);
        float w[8];
        load_w(a.W, c, w);
        if constexpr (LN) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = ((v[i] - mean) - rest) * rstd * w[i];
            if (a.B) {
                load_w(a.B, c, w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] += w[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = v[i] * rstd * w[i];
        }
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

template <int XT, int MODE, int T, int C, bool LN>
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
        norm_kernel<XT, MODE, T, C, LN><<<(unsigned)((b.M + kRows - 1) / kRows), kThreads, 0, s>>>(b);
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
template <int XT, int MODE, bool LN>
static void launch_norm(const NormArgs &a, hipStream_t s)
{
    const int64_t k8 = a.K / 8;
    if (k8 <= 64)
        launch_norm_rows<XT, MODE, 64, 1, LN>(a, s);
    else if (k8 <= 128 && a.M > 8192)
        launch_norm_rows<XT, MODE, 64, 2, LN>(a, s);
    else if (k8 <= 256)
        launch_norm_rows<XT, MODE, 256, 1, LN>(a, s);
    else if (k8 <= 512)
        launch_norm_rows<XT, MODE, 512, 1, LN>(a, s);
    else if (k8 <= 1024 && a.M > 384)
        launch_norm_rows<XT, MODE, 512, 2, LN>(a, s);
    else if (k8 <= 1024)
        launch_norm_rows<XT, MODE, 1024, 1, LN>(a, s);
    else if (k8 <= 4096)
        launch_norm_rows<XT, MODE, 1024, 4, LN>(a, s);
    else
        launch_norm_rows<XT, MODE, 1024, 0, LN>(a, s);
}

template <bool LN>
static hipError_t launch_norm_typed(const NormArgs &a, int x_type, int mode, hipStream_t s)
{
    auto typed = [&](auto xt) {
        constexpr int XT = decltype(xt)::value;
        switch (mode) {
        case kScaleNone: launch_norm<XT, kScaleNone, LN>(a, s); return hipGetLastError();
        case kScaleTensor: launch_norm<XT, kScaleTensor, LN>(a, s); return hipGetLastError();
        case kScaleBlock: launch_norm<XT, kScaleBlock, LN>(a, s); return hipGetLastError();
        case kScaleMx: launch_norm<XT, kScaleMx, LN>(a, s); return hipGetLastError();
        case kScaleMx32: launch_norm<XT, kScaleMx32, LN>(a, s); return hipGetLastError();
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
