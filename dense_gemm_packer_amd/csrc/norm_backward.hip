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

// Sums of N values over the threads of a row, in every thread: up to WAVES waves
// (1, 4, 8 or 16), whose sums stand from `first` on in `red`; t: the thread of
// the row.  `red` holds zeros for waves that are not there, and is not written
// again before the second barrier from here.
template <int WAVES, int N>
__device__ inline void sums(float (&v)[N], f32x4 (*red)[WAVES == 16 ? 4 : 2], int first, int t)
{
#pragma unroll
    for (int n = 0; n < N; ++n)
        v[n] = total64(v[n]);
    if constexpr (WAVES > 1) {
        if ((t & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                reinterpret_cast<float *>(red[n])[first + (t >> 6)] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            f32x4 s = red[n][first / 4];
#pragma unroll
            for (int q = 1; q < WAVES / 4; ++q)
                s += red[n][first / 4 + q];
            v[n] = (s[0] + s[1]) + (s[2] + s[3]);
        }
    }
}

// Zeros in all of an array of `red`, before its first use (a barrier follows).
__device__ inline void clear(f32x4 *red, int n)
{
    if ((int)threadIdx.x < n)
        red[threadIdx.x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
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

// A row's pieces of 8 elements go to T = blockDim.x / R threads, C each; R rows
// of a workgroup at once (WAVE: a wave a row, no barriers).  The next row's loads
// are in flight while this one's sums go through the lanes.  To leave registers
// for two workgroups a CU the weight waits in LDS and dy as it was loaded.
template <int XT, int MODE, int C, int R, bool WAVE, int THREADS, bool LN>
__global__ __launch_bounds__(THREADS, C == 1 ? 4 : XT == kTypeF32 ? 2 : WAVE ? 3 : 4) void norm_grad_kernel(const NormGradArgs a)
{
    const int T = WAVE ? 64 : (int)blockDim.x / R;
    const int rows_at_once = WAVE ? (int)blockDim.x / 64 : R;
    const int sub = WAVE || R > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / T) : 0;
    const int t = (int)threadIdx.x - sub * T;
    constexpr int kWaves = WAVE ? 1 : 8 / R;       // of a row, at most
    const int k8 = (int)(a.K / 8), first_wave = WAVE ? 0 : sub * kWaves;
    const float invk = 1.0f / (float)a.K;
    const int64_t stride = (int64_t)gridDim.x * rows_at_once;
    constexpr int kPieces = WAVE ? 64 * C : THREADS / R * C;
    __shared__ f32x4 weight[2][kPieces];       // halves of pieces
    __shared__ f32x4 red1[2][2][2];
    [[maybe_unused]] __shared__ f32x4 red2[3][2];

    Raw8<XT> ry[C];
    Kept8<XT, MODE> rx[C];
    auto load = [&](int64_t row) {
        if (row < a.M) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int p = t + c * T;
                if (p < k8) {
                    ry[c] = load_raw8<XT>(a.Y, row * a.ldy + p * 8);
                    rx[c] = load_kept8<XT, MODE>(a.X, a.S, row, a.ldx, a.K / 128, p * 8);
                }
            }
        }
    };
    float dw[C][8];
    [[maybe_unused]] float db[LN ? C : 1][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[c][i] = 0.0f;
            if constexpr (LN)
                db[c][i] = 0.0f;
        }
    const int64_t row0 = (int64_t)blockIdx.x * rows_at_once;
    load(row0 + sub);
    for (int p = (int)threadIdx.x; p < k8; p += (int)blockDim.x) {
        float w[8];
        load_weight<XT>(a, p, w);
        weight[0][p] = f32x4{w[0], w[1], w[2], w[3]};
        weight[1][p] = f32x4{w[4], w[5], w[6], w[7]};
    }
    if constexpr (!WAVE) {
        clear(red1[0][0], 8);
        clear(red2[0], 6);
    }
    __syncthreads();
    int turn = 0;
    for (int64_t base = row0; base < a.M; base += stride, turn ^= 1) {   // (the same count in every thread)
        const int64_t row = base + sub;
        const bool live = row < a.M;
        Raw8<XT> rr[C], y[C];
        float x[C][8], g[C][8];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (live && t + c * T < k8) {
                if (a.R)
                    rr[c] = load_raw8<XT>(a.R, row * a.ldr + (t + c * T) * 8);
                y[c] = ry[c];
                kept_floats<XT, MODE>(rx[c], x[c]);
            } else {
                y[c] = Raw8<XT>{};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[c][i] = 0.0f;
            }
        }
        load(row + stride);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[8];
            to_float8<XT>(y[c], v);
            const int p = t + c * T < k8 ? t + c * T : 0;
            const f32x4 w0 = weight[0][p], w1 = weight[1][p];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[c][i] = v[i] * w0[i];
                g[c][i + 4] = v[i + 4] * w1[i];
            }
        }
        float rstd, mg = 0.0f, c2;
        if constexpr (LN) {
            float s1[2] = {0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s1[0] += x[c][i];
                    s1[1] += g[c][i];
                }
            sums<kWaves>(s1, red1[turn], first_wave, t);
            const float mean = s1[0] * invk;
            mg = s1[1] * invk;
            float s2[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t + c * T < k8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[c][i] -= mean;
                        g[c][i] -= mg;
                        s2[0] += x[c][i];
                        s2[1] = __builtin_fmaf(x[c][i], x[c][i], s2[1]);
                        s2[2] = __builtin_fmaf(g[c][i], x[c][i], s2[2]);
                    }
                }
            sums<kWaves>(s2, red2, first_wave, t);
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
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s1[0] = __builtin_fmaf(x[c][i], x[c][i], s1[0]);
                    s1[1] = __builtin_fmaf(g[c][i], x[c][i], s1[1]);
                }
            sums<kWaves>(s1, red1[turn], first_wave, t);
            rstd = 1.0f / __builtin_sqrtf(s1[0] * invk + a.eps);
            c2 = s1[1] * invk * rstd;
        }
        if (live) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t + c * T < k8) {
                    float d[8], v[8];
                    to_float8<XT>(y[c], v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float xh = x[c][i] * rstd;
                        dw[c][i] = __builtin_fmaf(v[i], xh, dw[c][i]);
                        if constexpr (LN)
                            db[c][i] += v[i];
                        d[i] = rstd * __builtin_fmaf(-xh, c2, g[c][i]);
                    }
                    if (a.R) {
                        to_float8<XT>(rr[c], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            d[i] += v[i];
                    }
                    store8<XT>(a.D, row * a.K + (t + c * T) * 8, d);
                }
        }
    }

    // The rows of the workgroup join their sums, one after the other.
    if constexpr (WAVE || R > 1) {
        __shared__ float join[LN ? 2 : 1][kPieces * 8];
        for (int r = 1; r < rows_at_once; ++r) {
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
    __shared__ f32x4 red1[2][2][4], red2[3][4];
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
        sums<16>(s1, red1[turn], 0, t);
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
            sums<16>(s2, red2, 0, t);
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

// Threads of the row kernel's workgroups, and rows of each at once.
struct Shape {
    int threads, rows;
};
Shape shape_of(int64_t K)
{
    const int k8 = (int)(K / 8);
    if (k8 <= 128)
        return {512, 8};                                 // a wave a row
    if (k8 <= 256)
        return {(k8 + 63) / 64 * 128, 2};
    const int each = k8 <= 512 ? 1 : 2;                  // pieces a thread
    return {((k8 + each - 1) / each + 63) / 64 * 64, 1};
}

int64_t row_groups(int64_t M, int64_t K)
{
    const Shape p = shape_of(K);
    return std::min<int64_t>((M + p.rows - 1) / p.rows, 512);
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
        const int threads = shape_of(a.K).threads;
        const int64_t k8 = a.K / 8;
        if (k8 <= 64)
            norm_grad_kernel<XT, MODE, 1, 1, true, 512, LN><<<grid, threads, 0, s>>>(a);
        else if (k8 <= 128)
            norm_grad_kernel<XT, MODE, 2, 1, true, 512, LN><<<grid, threads, 0, s>>>(a);
        else if (k8 <= 256)
            norm_grad_kernel<XT, MODE, 1, 2, false, 512, LN><<<grid, threads, 0, s>>>(a);
        else if (k8 <= 512)
            norm_grad_kernel<XT, MODE, 1, 1, false, 512, LN><<<grid, threads, 0, s>>>(a);
        else
            norm_grad_kernel<XT, MODE, 2, 1, false, 512, LN><<<grid, threads, 0, s>>>(a);
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
