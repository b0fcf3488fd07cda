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
// every run.  HBM-bound where rows are many (4096 x 8192 bf16 with a residual, x an
// 8-bit checkpoint with block scales: 236 MB in 44 us, 5.4 TB/s, and 5 us for the
// partial sums; 16 391 x 2048 mxfp8 without means 235 MB in 35 and 4), latency where
// they are few (128 x 7168: 6 and 2 to 3 us).
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
template <int WAVES, int N, int RED>
__device__ inline void sums(float (&v)[N], f32x4 (*red)[RED], int first, int t)
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

// Pieces of 8 elements of one row through a buffer resource that ends with the
// row (or holds nothing): a piece past the end loads as zeros and is not stored.
// Without branches around them the waits for loads in flight are exact.
template <int XT>
__device__ inline Raw8<XT> row_load(const __amdgpu_buffer_rsrc_t &r, uint32_t piece)
{
    constexpr uint32_t kSize = XT == kTypeF32 ? 32 : 16;
    Raw8<XT> v;
    v.v[0] = load16<kAuxNone>(r, piece * kSize);
    if constexpr (XT == kTypeF32)
        v.v[1] = load16<kAuxNone>(r, piece * kSize + 16);
    return v;
}

template <int XT>
__device__ inline void row_store(const __amdgpu_buffer_rsrc_t &r, uint32_t piece, const float (&x)[8])
{
    alignas(16) i32x4 v[XT == kTypeF32 ? 2 : 1];
    store8<XT>(v, 0, x);
    __builtin_amdgcn_raw_buffer_store_b128(v[0], r, piece * (XT == kTypeF32 ? 32 : 16), 0, 0);
    if constexpr (XT == kTypeF32)
        __builtin_amdgcn_raw_buffer_store_b128(v[1], r, piece * 32 + 16, 0, 0);
}

template <int XT, int MODE>
__device__ inline Kept8<XT, MODE> row_load_kept(const __amdgpu_buffer_rsrc_t &r, const __amdgpu_buffer_rsrc_t &rs, uint32_t piece)
{
    Kept8<XT, MODE> k;
    if constexpr (MODE == kScaleNone) {
        k.raw = row_load<XT>(r, piece);
    } else {
        k.codes = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, piece * 8, 0, 0));
        if constexpr (MODE == kScaleBlock)
            k.scale = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, piece / 16 * 4, 0, 0);
        else if constexpr (MODE == kScaleMx)
            k.scale = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, piece / 16, 0, 0);
    }
    return k;
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

// A row's pieces of 8 elements go to T threads (whole waves), one each; `side` =
// blockDim.x / T rows of a workgroup side by side.  WAVES: 1 (a wave a row, no
// barriers), 4, 8 or 16, room for the sums of a row's waves.  The next row's loads
// are in flight while this one's sums go through the lanes; to leave registers for
// four waves a SIMD the weight waits in LDS (4096 x 8192 bf16 with a residual,
// layer norm: 60 us, in registers 67) and dy as it was loaded.
template <int XT, int MODE, int WAVES, bool LN>
__global__ __launch_bounds__(1024, 4) void norm_grad_kernel(const NormGradArgs a, const int rows_side, const int T)
{
    constexpr bool kSide = WAVES < 16;                        // several rows
    const int side = kSide ? rows_side : 1;
    constexpr int kRed = WAVES == 4 ? 8 : WAVES == 8 ? 6 : 4; // 8 rows of 4, 3 of 8, 1 of 16
    const int sub = kSide ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / T) : 0;
    const int t = (int)threadIdx.x - sub * T;                 // the piece
    const bool mine = t < (int)(a.K / 8);
    const int first_wave = sub * WAVES;
    const float invk = 1.0f / (float)a.K;
    const int64_t stride = (int64_t)gridDim.x * side;
    constexpr int kPieces = WAVES * 64;
    __shared__ f32x4 weight[2][kPieces];                      // halves of pieces
    __shared__ f32x4 red1[2][2][kRed];
    [[maybe_unused]] __shared__ f32x4 red2[3][kRed];

    constexpr int64_t kSize = XT == kTypeF32 ? 4 : 2, kKept = MODE == kScaleNone ? kSize : 1;
    constexpr int64_t kScale = MODE == kScaleBlock ? 4 : MODE == kScaleMx ? 1 : 0;
    auto row_of = [&](const void *p, int64_t row, int64_t ld_bytes, int64_t bytes) {
        return make_rsrc(static_cast<const uint8_t *>(p) + row * ld_bytes, p && row < a.M ? (uint32_t)bytes : 0u);
    };
    [[maybe_unused]] uint32_t tensor = 0;
    if constexpr (MODE == kScaleTensor)
        tensor = *static_cast<const uint32_t *>(a.S);

    Raw8<XT> ry;
    Kept8<XT, MODE> rx;
    auto load = [&](int64_t row) {
        ry = row_load<XT>(row_of(a.Y, row, a.ldy * kSize, a.K * kSize), t);
        rx = row_load_kept<XT, MODE>(row_of(a.X, row, a.ldx * kKept, a.K * kKept),
                                     row_of(a.S, row, a.K / 128 * kScale, a.K / 128 * kScale), t);
        if constexpr (MODE == kScaleTensor)
            rx.scale = tensor;
    };
    const int64_t row0 = (int64_t)blockIdx.x * side;
    load(row0 + sub);
    float dw[8];
    [[maybe_unused]] float db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        dw[i] = db[i] = 0.0f;
    if (sub == 0) {
        float w[8] = {};
        if (mine)
            load_weight<XT>(a, t, w);
        weight[0][t] = f32x4{w[0], w[1], w[2], w[3]};
        weight[1][t] = f32x4{w[4], w[5], w[6], w[7]};
    }
    if constexpr (WAVES > 1) {
        clear(red1[0][0], 4 * kRed);
        clear(red2[0], 3 * kRed);
    }
    __syncthreads();
    auto step = [&](auto pc, int64_t row) {
        constexpr int P = decltype(pc)::value;
        const Raw8<XT> r = row_load<XT>(row_of(a.R, row, a.ldr * kSize, a.K * kSize), t), y = ry;
        float x[8], g[8];
        kept_floats<XT, MODE>(rx, x);
        load(row + stride);
        float v[8];
        to_float8<XT>(y, v);
        const f32x4 w0 = weight[0][t], w1 = weight[1][t];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g[i] = v[i] * w0[i];
            g[i + 4] = v[i + 4] * w1[i];
        }
        float rstd, c2;
        if constexpr (LN) {
            float s1[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1[0] += x[i];
                s1[1] += g[i];
            }
            sums<WAVES>(s1, red1[P], first_wave, t);
            const float mean = mine ? s1[0] * invk : 0.0f, mg = mine ? s1[1] * invk : 0.0f;
            float s2[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] -= mean;
                g[i] -= mg;
                s2[0] += x[i];
                s2[1] = __builtin_fmaf(x[i], x[i], s2[1]);
                s2[2] = __builtin_fmaf(g[i], x[i], s2[2]);
            }
            sums<WAVES>(s2, red2, first_wave, t);
            const float rest = s2[0] * invk;       // what the fp32 mean is off by
            const float var = s2[1] * invk - rest * rest;
            rstd = 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
            c2 = s2[2] * invk * rstd;              // (g - mean(g) sums to 0: `rest` adds nothing)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] -= rest;
        } else {
            float s1[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1[0] = __builtin_fmaf(x[i], x[i], s1[0]);
                s1[1] = __builtin_fmaf(g[i], x[i], s1[1]);
            }
            sums<WAVES>(s1, red1[P], first_wave, t);
            rstd = 1.0f / __builtin_sqrtf(s1[0] * invk + a.eps);
            c2 = s1[1] * invk * rstd;
        }
        // (a row past the last has nothing to add, whatever eps is)
        rstd = row < a.M ? rstd : 0.0f;
        float d[8];
        to_float8<XT>(y, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float xh = x[i] * rstd;
            dw[i] = __builtin_fmaf(v[i], xh, dw[i]);
            if constexpr (LN)
                db[i] += v[i];
            d[i] = rstd * __builtin_fmaf(-xh, c2, g[i]);
        }
        to_float8<XT>(r, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            d[i] += v[i];
        row_store<XT>(row_of(a.D, row, a.K * kSize, a.K * kSize), t, d);
    };
    for (int64_t base = row0; base < a.M; base += 2 * stride) {      // (the same count in every thread)
        step(std::integral_constant<int, 0>{}, base + sub);
        if (base + stride < a.M)
            step(std::integral_constant<int, 1>{}, base + stride + sub);
    }

    const bool alone = gridDim.x == 1;
    float *pw = alone ? a.dW : a.ws + (int64_t)blockIdx.x * (LN ? 2 : 1) * a.K;
    float *pb = alone ? a.dB : pw + a.K;
    if constexpr (!kSide) {
        if (!mine)
            return;
        store8<kTypeF32>(pw, t * 8, dw);
        if (LN && pb)
            store8<kTypeF32>(pb, t * 8, db);
    } else {
        // The rows side by side put their sums into LDS, and every thread adds up those
        // of a quad of columns, in order (16 391 x 512 bf16, sixteen rows: 17.3 us; row
        // after row, two barriers each, 19.5).
        constexpr int kQuads = LN ? 4 : 2;                    // dw, db: halves of pieces
        __shared__ f32x4 join[kQuads * 1024];
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            const float *v = (q < 2 ? dw : db) + q % 2 * 4;
            join[(q * side + sub) * T + t] = f32x4{v[0], v[1], v[2], v[3]};
        }
        __syncthreads();
        // (every wave is in one quad's range: T is whole waves)
        for (int c = (int)threadIdx.x; c < kQuads * T; c += (int)blockDim.x) {
            const int q = c / T, piece = c - q * T;
            float *p = q < 2 ? pw : pb;
            f32x4 sum = join[q * side * T + piece];
            for (int r = 1; r < side; ++r)
                sum += join[(q * side + r) * T + piece];
            if (p && piece < (int)(a.K / 8))
                *reinterpret_cast<f32x4 *>(p + piece * 8 + q % 2 * 4) = sum;
        }
    }
}

// Partial sums [parts][len] (len = one or two times K) -> dW, dB.  A workgroup
// takes 32 columns; its 32 threads per quad of columns each add every 32nd part,
// and the 32 sums are added in order (300 x 1024 bf16, layer norm: 7.6 us in all; 64
// columns a workgroup, sixteen threads a quad, 9.3).
constexpr int kSlices = 32;
__global__ __launch_bounds__(8 * kSlices) void norm_grad_join_kernel(const float *ws, int parts, int64_t K, int64_t len,
                                                                      float *dW, float *dB)
{
    const int q = threadIdx.x & 7, slice = threadIdx.x >> 3;
    const int64_t col = (int64_t)blockIdx.x * 32 + q * 4;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int g = slice; g < parts; g += 4 * kSlices) {      // (four loads in flight, whatever is left)
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = *reinterpret_cast<const f32x4 *>(ws + (int64_t)std::min(g + i * kSlices, parts - 1) * len + col);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s += g + i * kSlices < parts ? v[i] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __shared__ f32x4 part[kSlices][8];
    part[slice][q] = s;
    __syncthreads();
    if (slice != 0)
        return;
#pragma unroll
    for (int i = 1; i < kSlices; ++i)
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

// The row kernel: as many rows side by side as make up 16 waves.  One workgroup a
// CU writes the fewest partial sums, and side by side the short rows share its
// barriers: 16 391 x 2304 bf16, layer norm, three rows 65 us, two 71; 4096 x 4096
// two rows 30.7, one 33.2; 16 391 x 2048 mxfp8, root-mean-square norm, four rows
// 43.7, two in 8 waves (two workgroups a CU) 46.4.  With few rows the waves of one
// workgroup wait for each other to no end: 128 workgroups then (256 x 512 bf16 6.6
// us, sixteen rows in each of 16 workgroups 9.4; 256 workgroups, whose partial sums
// are more to add up, 7.5).
struct Shape {
    int side, waves;       // rows, waves of a row
    int threads() const { return side * waves * 64; }
};
Shape shape_of(int64_t M, int64_t K)
{
    const int waves = (int)((K + 511) / 512);
    return {(int)std::min<int64_t>(16 / waves, (M + 127) / 128), waves};
}

int64_t row_groups(int64_t M, int64_t K)
{
    const Shape p = shape_of(M, K);
    return std::min<int64_t>((M + p.side - 1) / p.side, 256);
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
        const Shape p = shape_of(a.M, a.K);
        const int T = p.waves * 64;
        if (p.waves == 1)
            norm_grad_kernel<XT, MODE, 1, LN><<<grid, p.threads(), 0, s>>>(a, p.side, T);
        else if (p.waves <= 4)
            norm_grad_kernel<XT, MODE, 4, LN><<<grid, p.threads(), 0, s>>>(a, p.side, T);
        else if (p.waves <= 8)
            norm_grad_kernel<XT, MODE, 8, LN><<<grid, p.threads(), 0, s>>>(a, p.side, T);
        else
            norm_grad_kernel<XT, MODE, 16, LN><<<grid, p.threads(), 0, s>>>(a, p.side, T);
        if (count == 1)
            return hipGetLastError();
    }
    norm_grad_join_kernel<<<(unsigned)(len / 32), 8 * kSlices, 0, s>>>(parts, (int)count, a.K, len, a.dW, a.dB);
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
