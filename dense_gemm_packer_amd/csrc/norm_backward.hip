// Gradients of the layer norm and of the root-mean-square norm
// (dgp_layernorm_backward, dgp_rmsnorm_backward).  With xhat = (x - mean) *
// rstd over a row and g = dy * w,
//
//   dx = rstd (g - mean(g) - xhat mean(g xhat)) (+ r),
//   dw = sum over rows of dy xhat,   db = sum over rows of dy,
//
// and without the two means (of x and of g) for the root-mean-square norm.  The
// row's statistics are taken again from x: it is read for xhat anyway, so they
// cost no memory, and with x an 8-bit checkpoint the result is the gradient at
// the values that the checkpoint holds.  All arithmetic is fp32.
//
// The sums over rows: a workgroup owns every G-th row and keeps its sums in
// registers (a thread has the same columns of every row), writes them once, and
// a second kernel adds the G partial sums in order: no atomics, the same bits in
// every run.
#include <algorithm>

#include "common.h"
#include "launch.h"
#include "operand.h"

namespace dgp {

namespace {

// Sums of N values over the T threads of a row, in every thread.  The W / T
// rows of the workgroup do this at the same time; `red` (N x W / 64 values) is
// not written again before the second barrier from here.
template <int T, int W, int N>
__device__ inline void sums(float (&v)[N], float (*red)[W / 64])
{
#pragma unroll
    for (int n = 0; n < N; ++n)
        v[n] = sum64(v[n]);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                red[n][threadIdx.x >> 6] = v[n];
        }
        __syncthreads();
        const int first = (int)(threadIdx.x / T) * (T / 64);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = red[n][first];
#pragma unroll
            for (int w = 1; w < T / 64; ++w)
                v[n] += red[n][first + w];
        }
    }
}

template <int XT>
__device__ inline void load_weight(const NormGradArgs &a, int c, float (&w)[8])
{
    if (a.wt == kTypeF32)
        to_float8<kTypeF32>(load_raw8<kTypeF32>(a.W, (int64_t)c * 8), w);
    else
        to_float8<XT>(load_raw8<XT>(a.W, (int64_t)c * 8), w);
}

}  // namespace

// T threads own a row (W / T rows of a workgroup at once), C pieces of 8
// elements each; the next row's loads are in flight while this one's sums go
// through the lanes.
template <int XT, int MODE, int T, int W, int C, bool LN>
__global__ __launch_bounds__(W) void norm_grad_kernel(const NormGradArgs a)
{
    constexpr int R = W / T;
    const int t = threadIdx.x % T, sub = threadIdx.x / T;
    const int k8 = (int)(a.K / 8);
    const float invk = 1.0f / (float)a.K;
    const int64_t stride = (int64_t)gridDim.x * R;
    __shared__ float red1[2][2][W / 64];
    [[maybe_unused]] __shared__ float red2[3][W / 64];

    Raw8<XT> ry[C], rr[C];
    Kept8<XT, MODE> rx[C];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int p = t + c * T;
            if (p < k8 && row < a.M) {
                ry[c] = load_raw8<XT>(a.Y, row * a.ldy + p * 8);
                rx[c] = load_kept8<XT, MODE>(a.X, a.S, row, a.ldx, a.K / 128, p * 8);
            }
        }
    };
    auto load_r = [&](int64_t row) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (t + c * T < k8 && row < a.M)
                rr[c] = load_raw8<XT>(a.R, row * a.ldr + (t + c * T) * 8);
    };

    float w[C][8], dw[C][8];
    [[maybe_unused]] float db[LN ? C : 1][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (t + c * T < k8)
            load_weight<XT>(a, t + c * T, w[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[c][i] = 0.0f;
            if constexpr (LN)
                db[c][i] = 0.0f;
        }
    }
    const int64_t row0 = (int64_t)blockIdx.x * R;
    load(row0 + sub);
    int turn = 0;
    for (int64_t base = row0; base < a.M; base += stride, turn ^= 1) {   // (the same count in every thread)
        const int64_t row = base + sub;
        const bool live = row < a.M;
        if (a.R)
            load_r(row);
        float x[C][8], y[C][8];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (live && t + c * T < k8) {
                to_float8<XT>(ry[c], y[c]);
                kept_floats<XT, MODE>(rx[c], x[c]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[c][i] = y[c][i] = 0.0f;
            }
        }
        load(row + stride);
        float rstd, mg = 0.0f, c2;
        if constexpr (LN) {
            float s1[2] = {0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t + c * T < k8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        s1[0] += x[c][i];
                        s1[1] = __builtin_fmaf(y[c][i], w[c][i], s1[1]);
                    }
                }
            sums<T, W>(s1, red1[turn]);
            const float mean = s1[0] * invk;
            mg = s1[1] * invk;
            float s2[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t + c * T < k8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[c][i] -= mean;
                        s2[0] += x[c][i];
                        s2[1] = __builtin_fmaf(x[c][i], x[c][i], s2[1]);
                        s2[2] = __builtin_fmaf(y[c][i] * w[c][i] - mg, x[c][i], s2[2]);
                    }
                }
            sums<T, W>(s2, red2);
            const float rest = s2[0] * invk;       // what the fp32 mean is off by
            const float var = s2[1] * invk - rest * rest;
            rstd = 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
            c2 = s2[2] * invk * rstd;              // (g - mean(g) sums to 0: `rest` adds nothing)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[c][i] -= rest;
        } else {
            float s1[2] = {0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t + c * T < k8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        s1[0] = __builtin_fmaf(x[c][i], x[c][i], s1[0]);
                        s1[1] = __builtin_fmaf(y[c][i] * w[c][i], x[c][i], s1[1]);
                    }
                }
            sums<T, W>(s1, red1[turn]);
            rstd = 1.0f / __builtin_sqrtf(s1[0] * invk + a.eps);
            c2 = s1[1] * invk * rstd;
        }
        if (live) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t + c * T < k8) {
                    float d[8], r[8];
                    if (a.R)
                        to_float8<XT>(rr[c], r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float xh = x[c][i] * rstd;
                        dw[c][i] = __builtin_fmaf(y[c][i], xh, dw[c][i]);
                        if constexpr (LN)
                            db[c][i] += y[c][i];
                        float g = y[c][i] * w[c][i];
                        if constexpr (LN)
                            g -= mg;
                        d[i] = rstd * (g - xh * c2);
                        if (a.R)
                            d[i] += r[i];
                    }
                    store8<XT>(a.D, row * a.K + (t + c * T) * 8, d);
                }
        }
    }

    // The rows of the workgroup join their sums, one after the other.
    if constexpr (R > 1) {
        __shared__ float join[LN ? 2 : 1][T * C * 8];
        for (int r = 1; r < R; ++r) {
            __syncthreads();
            if (sub == r) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        join[0][(c * 8 + i) * T + t] = dw[c][i];
                        if constexpr (LN)
                            join[1][(c * 8 + i) * T + t] = db[c][i];
                    }
            }
            __syncthreads();
            if (sub == 0) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dw[c][i] += join[0][(c * 8 + i) * T + t];
                        if constexpr (LN)
                            db[c][i] += join[1][(c * 8 + i) * T + t];
                    }
            }
        }
    }
    if (sub != 0)
        return;
    const bool alone = gridDim.x == 1;
    float *pw = alone ? a.dW : a.ws + (int64_t)blockIdx.x * (LN ? 2 : 1) * a.K;
    float *pb = alone ? a.dB : pw + a.K;
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (t + c * T < k8) {
            store8<kTypeF32>(pw, (t + c * T) * 8, dw[c]);
            if (LN && pb)
                store8<kTypeF32>(pb, (t + c * T) * 8, db[LN ? c : 0]);
        }
}

// Partial sums [parts][len] (len = one or two times K) -> dW, dB.  A workgroup
// takes 64 columns; its 16 threads per quad of columns each add every 16th part,
// and the 16 sums are added in order.
__global__ __launch_bounds__(256) void norm_grad_join_kernel(const float *ws, int parts, int64_t K, int64_t len, float *dW,
                                                             float *dB)
{
    const int q = threadIdx.x & 15, slice = threadIdx.x >> 4;
    const int64_t col = (int64_t)blockIdx.x * 64 + q * 4;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int g = slice; g < parts; g += 16)
        s += *reinterpret_cast<const f32x4 *>(ws + (int64_t)g * len + col);
    __shared__ f32x4 part[16][16];
    part[slice][q] = s;
    __syncthreads();
    if (slice != 0)
        return;
#pragma unroll
    for (int i = 1; i < 16; ++i)
        s += part[i][q];
    float *out = col < K ? dW + col : dB ? dB + (col - K) : nullptr;
    if (out)
        *reinterpret_cast<f32x4 *>(out) = s;
}

// Rows longer than the registers hold: dx row by row, reading the row for each
// use, with the row's statistics (mean, its remainder, rstd) kept for the sums
// over rows, which a second kernel takes column by column.
constexpr int kLongThreads = 1024;
template <int XT, int MODE, bool LN>
__global__ __launch_bounds__(kLongThreads) void norm_grad_long_kernel(const NormGradArgs a, float *stats)
{
    constexpr int T = kLongThreads;
    const int t = threadIdx.x, k8 = (int)(a.K / 8);
    const float invk = 1.0f / (float)a.K;
    __shared__ float red1[2][2][T / 64], red2[3][T / 64];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
        float x[8], y[8], w[8];
        auto load = [&](int c) {
            to_float8<XT>(load_raw8<XT>(a.Y, row * a.ldy + (int64_t)c * 8), y);
            kept_floats<XT, MODE>(load_kept8<XT, MODE>(a.X, a.S, row, a.ldx, a.K / 128, c * 8), x);
            load_weight<XT>(a, c, w);
        };
        float mean = 0.0f, rest = 0.0f, mg = 0.0f, rstd, c2;
        float s1[2] = {0.0f, 0.0f};
        for (int c = t; c < k8; c += T) {
            load(c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1[0] = LN ? s1[0] + x[i] : __builtin_fmaf(x[i], x[i], s1[0]);
                s1[1] = __builtin_fmaf(y[i] * w[i], LN ? 1.0f : x[i], s1[1]);
            }
        }
        sums<T, T>(s1, red1[turn]);
        if constexpr (LN) {
            mean = s1[0] * invk, mg = s1[1] * invk;
            float s2[3] = {0.0f, 0.0f, 0.0f};
            for (int c = t; c < k8; c += T) {
                load(c);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = x[i] - mean;
                    s2[0] += d;
                    s2[1] = __builtin_fmaf(d, d, s2[1]);
                    s2[2] = __builtin_fmaf(y[i] * w[i] - mg, d, s2[2]);
                }
            }
            sums<T, T>(s2, red2);
            rest = s2[0] * invk;
            const float var = s2[1] * invk - rest * rest;
            rstd = 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
            c2 = s2[2] * invk * rstd;
        } else {
            rstd = 1.0f / __builtin_sqrtf(s1[0] * invk + a.eps);
            c2 = s1[1] * invk * rstd;
        }
        if (t == 0)
            *reinterpret_cast<f32x4 *>(stats + row * 4) = f32x4{mean, rest, rstd, 0.0f};
        for (int c = t; c < k8; c += T) {
            load(c);
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] = rstd * (y[i] * w[i] - mg - ((x[i] - mean) - rest) * rstd * c2);
            if (a.R) {
                float r[8];
                to_float8<XT>(load_raw8<XT>(a.R, row * a.ldr + (int64_t)c * 8), r);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] += r[i];
            }
            store8<XT>(a.D, row * a.K + (int64_t)c * 8, d);
        }
    }
}

// Sums over rows of 512 columns: four waves take every fourth row of a slab.
template <int XT, int MODE, bool LN>
__global__ __launch_bounds__(256) void norm_grad_columns_kernel(const NormGradArgs a, const float *stats, float *parts)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = (int)blockIdx.x * 64 + lane;
    const bool live = c < (int)(a.K / 8);
    float dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        dw[i] = db[i] = 0.0f;
    for (int64_t row = (int64_t)blockIdx.y * 4 + wave; row < a.M && live; row += (int64_t)gridDim.y * 4) {
        float x[8], y[8];
        to_float8<XT>(load_raw8<XT>(a.Y, row * a.ldy + (int64_t)c * 8), y);
        kept_floats<XT, MODE>(load_kept8<XT, MODE>(a.X, a.S, row, a.ldx, a.K / 128, c * 8), x);
        const f32x4 st = *reinterpret_cast<const f32x4 *>(stats + row * 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[i] = __builtin_fmaf(y[i], ((x[i] - st[0]) - st[1]) * st[2], dw[i]);
            db[i] += y[i];
        }
    }
    __shared__ float join[3][16][64];
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            join[wave - 1][i][lane] = dw[i], join[wave - 1][8 + i][lane] = db[i];
    }
    __syncthreads();
    if (wave > 0 || !live)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int v = 0; v < 3; ++v)
            dw[i] += join[v][i][lane], db[i] += join[v][8 + i][lane];
    float *p = parts + (int64_t)blockIdx.y * (LN ? 2 : 1) * a.K;
    store8<kTypeF32>(p, (int64_t)c * 8, dw);
    if (LN)
        store8<kTypeF32>(p + a.K, (int64_t)c * 8, db);
}

// --------------------------------------------------------------- launches

namespace {

constexpr int64_t kLongRow = 8192;     // elements; longer rows take the two kernels above

// Workgroups of the row kernel: R rows of a workgroup at once.
struct Shape {
    int T, W, C;
};
Shape shape_of(int64_t K)
{
    const int64_t k8 = K / 8;
    if (k8 <= 64)
        return {64, 512, 1};
    if (k8 <= 128)
        return {64, 512, 2};
    if (k8 <= 256)
        return {256, 512, 1};
    if (k8 <= 512)
        return {512, 512, 1};
    return {512, 512, 2};
}

int64_t row_groups(int64_t M, int64_t K)
{
    const Shape p = shape_of(K);
    const int64_t rows = p.W / p.T, all = (M + rows - 1) / rows;
    return std::min<int64_t>(all, 512);
}

int64_t long_slabs(int64_t M) { return std::clamp<int64_t>(M / 32, 1, 64); }

template <int XT, int MODE, bool LN>
hipError_t launch_grad(const NormGradArgs &a, hipStream_t s)
{
    const int64_t len = (LN ? 2 : 1) * a.K;
    float *parts = a.ws;
    int64_t count = 0;
    if (a.M == 0) {
        // the sums of no rows: the last kernel writes zeros
    } else if (a.K > kLongRow) {
        float *stats = a.ws;
        parts = a.ws + a.M * 4;
        count = long_slabs(a.M);
        norm_grad_long_kernel<XT, MODE, LN><<<(unsigned)std::min<int64_t>(a.M, 1024), kLongThreads, 0, s>>>(a, stats);
        norm_grad_columns_kernel<XT, MODE, LN><<<dim3((unsigned)((a.K + 511) / 512), (unsigned)count), 256, 0, s>>>(a, stats, parts);
    } else {
        count = row_groups(a.M, a.K);
        const unsigned grid = (unsigned)count;
        const Shape p = shape_of(a.K);
        if (p.T == 64 && p.C == 1)
            norm_grad_kernel<XT, MODE, 64, 512, 1, LN><<<grid, 512, 0, s>>>(a);
        else if (p.T == 64)
            norm_grad_kernel<XT, MODE, 64, 512, 2, LN><<<grid, 512, 0, s>>>(a);
        else if (p.T == 256)
            norm_grad_kernel<XT, MODE, 256, 512, 1, LN><<<grid, 512, 0, s>>>(a);
        else if (p.T == 512 && p.C == 1)
            norm_grad_kernel<XT, MODE, 512, 512, 1, LN><<<grid, 512, 0, s>>>(a);
        else
            norm_grad_kernel<XT, MODE, 512, 512, 2, LN><<<grid, 512, 0, s>>>(a);
        if (count == 1)
            return hipGetLastError();
    }
    norm_grad_join_kernel<<<(unsigned)(len / 64), 256, 0, s>>>(parts, (int)count, a.K, len, a.dW, a.dB);
    return hipGetLastError();
}

template <int XT, bool LN>
hipError_t launch_mode(const NormGradArgs &a, int mode, hipStream_t s)
{
    switch (mode) {
    case kScaleNone: return launch_grad<XT, kScaleNone, LN>(a, s);
    case kScaleTensor: return launch_grad<XT, kScaleTensor, LN>(a, s);
    case kScaleBlock: return launch_grad<XT, kScaleBlock, LN>(a, s);
    case kScaleMx: return launch_grad<XT, kScaleMx, LN>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

bool norm_grad_in_place(int64_t K) { return K <= kLongRow; }

size_t norm_grad_workspace_bytes(int64_t M, int64_t K, bool layer)
{
    const int64_t len = (layer ? 2 : 1) * K;
    if (K > kLongRow)
        return (size_t)(M * 4 + long_slabs(M) * len) * sizeof(float);
    const int64_t n = row_groups(M, K);
    return n > 1 ? (size_t)(n * len) * sizeof(float) : 0;
}

hipError_t launch_norm_grad(const NormGradArgs &a, int type, int mode, bool layer, hipStream_t s)
{
    switch (type) {
    case kDtypeBf16: return layer ? launch_mode<kDtypeBf16, true>(a, mode, s) : launch_mode<kDtypeBf16, false>(a, mode, s);
    case kTypeF16: return layer ? launch_mode<kTypeF16, true>(a, mode, s) : launch_mode<kTypeF16, false>(a, mode, s);
    case kTypeF32: return layer ? launch_mode<kTypeF32, true>(a, mode, s) : launch_mode<kTypeF32, false>(a, mode, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dgp
