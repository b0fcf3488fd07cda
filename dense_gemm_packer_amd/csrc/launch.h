// Internal launch interface between the C-ABI layer (dgp_api.cpp) and the
// HIP kernels.  Not installed; callers use include/dgp.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dgp {

// Arguments shared by both GEMM kernel families.  All sizes are validated by
// the host layer before a launch; byte quantities fit in 32 bits there.
struct GemmArgs {
    const uint8_t *A;     // [M][K] elements, row-major
    const uint8_t *Bs;    // preshuffled B (dgp_preshuffle_b layout)
    void *C;              // [M][N] bf16 (direct epilogue)
    float *ws;            // [splits][M][N] fp32 (split-K partial epilogue)
    const void *sA;       // per-tensor: 1 fp32; blockscale: [M][K/128] fp32; mxfp8: [M][K/128] E8M0
    const void *sB;       // per-tensor: 1 fp32; blockscale: [N/128][K/128] fp32; mxfp8: [N][K/128] E8M0
    int M, N;
    int K;                // elements per row
    int Kb;               // bytes per row of A and B
    int Ks;               // bytes of K per split
    int tiles_m, tiles_n, splits;
    int remap, group_m;
    // Product grouped by expert only (the kernels' GR = 1 form): M is the
    // number of product rows, tiles_m the most row tiles any offsets give.
    const int32_t *offsets;   // [groups + 1] first row of each expert, then the end
    const int32_t *rows;      // row of A of each product row, or NULL (row m takes row m)
    int groups;
    int a_rows;               // rows of A
};

// Kernel family selectors.
enum Family { kTiled = 0, kStream = 1, kWave = 2 };

// Wave schedules of the tiled family (dgp_config.schedule).
enum Schedule { kSchedInterleaved = 1, kSchedPingPong = 2, kSchedBothLds = 3, kSchedW4 = 4 };

// A's layout in LDS (tiled kernels; dgp_config.a_layout - 1): 1 KiB operand
// blocks (gemm_common.h), or row-major 128-byte rows with XOR-swizzled
// 16-byte chunks (gemm_w4.hip).
enum ALayout { kLayBlocks = 0, kLaySwizzled = 1 };

// A's global -> LDS copy (tiled kernels; dgp_config.a_copy - 1): the async
// buffer load that writes LDS directly, or a buffer load into registers and
// an LDS write (gemm_w4.hip keeps it as an ablation).
enum ACopy { kCopyAsync = 0, kCopyRegs = 1 };

// One compiled kernel configuration.
struct KernelSpec {
    int family;
    int dtype;      // 0 bf16, 1 fp8
    int scale;      // 0 none, 1 tensor, 2 block128, 3 mxfp8 (E8M0, 128-K blocks)
    int out;        // 0 bf16 direct, 1 fp32 partial
    int tm, tn;     // workgroup output tile
    int kt;         // K bytes per main-loop step (tiled) / per LDS panel (stream)
    int waves;      // waves per workgroup
    int p0, p1;     // family-specific: tiled = (wm, wn); stream = (strips per wave, depth)
    int pv, pd;     // scheduling hint pair (tiled)
    int depth;      // prefetch distance: k-tiles (tiled) / steps (stream)
    int sched;      // tiled: kSchedInterleaved, kSchedPingPong, kSchedBothLds or kSchedW4; stream, wave: 0
    void (*launch)(const GemmArgs &, dim3 grid, hipStream_t);
    int lay = 0;    // tiled: A's LDS layout, kLayBlocks or kLaySwizzled
    int copy = 0;   // tiled: A's global -> LDS path, kCopyAsync or kCopyRegs
    int k_mult = 0; // K is a multiple of this and the scales start at whole dwords (0: any that the mode takes)
};

// The compiled GEMM kernels: the tiled family (gemm_tiled.hip), its
// both-in-LDS schedule (gemm_lds.hip), its one-wave-per-SIMD schedule
// (gemm_w4.hip), the streaming family (gemm_stream.hip), the one-row VALU
// kernels (gemm_wave.hip), and all of them in one table in that order
// (dgp_api.cpp) -- the numbering dgp_kernel_info uses.
const KernelSpec *tiled_kernels(int *count);
const KernelSpec *lds_kernels(int *count);
const KernelSpec *w4_kernels(int *count);
const KernelSpec *stream_kernels(int *count);
const KernelSpec *wave_kernels(int *count);
const KernelSpec *kernel_table(int *count);
// The forms compiled for the product grouped by expert (single pass), per
// family and all of them (dgp_api.cpp).
const KernelSpec *tiled_grouped_kernels(int *count);
const KernelSpec *w4_grouped_kernels(int *count);
const KernelSpec *stream_grouped_kernels(int *count);
const KernelSpec *grouped_table(int *count);

// Library-owned split-K workspace (noalloc.hip): the size of the fixed
// per-device array, and its device address on the current device (taken
// once per device).
constexpr size_t kNoAllocScratchBytes = (size_t)16 << 20;
constexpr int kMaxDevices = 64;
hipError_t noalloc_scratch(float **out);

hipError_t launch_preshuffle(const void *src, void *dst, int64_t N, int64_t Kb, bool inverse,
                             hipStream_t stream);
hipError_t launch_splitk_reduce(const float *ws, void *C, int64_t M, int64_t N, int splits,
                                hipStream_t stream);

// Operators that write a GEMM operand (quantize.hip).  Input types are
// kDtypeBf16, kTypeF16 or kTypeF32; strides are in elements.
struct RowQuantArgs {
    const void *X;          // [M][K] rows ldx apart (the gated activation: the gate)
    const void *U;          // the gated activation's second factor, rows ldu apart
    void *Q;                // [M][K] codes (bf16 without scales)
    void *S;                // scales, row-major
    const float *scale;     // per tensor: the given scale, where parts is NULL
    const uint32_t *parts;  // per tensor: nparts <= 256 partial maxima (bits of |x|)
    int64_t ldx, ldu, M, K;
    int nparts;
};
struct WeightQuantArgs {
    const void *B;          // [rows][K], rows = a stack of matrices of N rows
    void *Q;                // preshuffled codes
    void *S;                // scales, row-major
    const uint32_t *parts;  // per tensor: nparts partial maxima per matrix
    int64_t rows, N, K;
    int nparts;
};
struct NormArgs {
    const void *X, *R, *W;  // R: residual or NULL, rows ldr apart
    const void *B;          // the layer norm's bias (W's type) or NULL
    void *Q, *S, *H;        // H: the residual stream's new value ([M][K]) or NULL
    const float *scale;
    int64_t ldx, ldr, M, K;
    float eps;
    int wt;                 // W's type: X's or kTypeF32
};

// Gradients (norm_backward.hip, swiglu_backward.hip).  Types are kDtypeBf16,
// kTypeF16 or kTypeF32; a kept input X has the gradients' type (mode
// kScaleNone) or e4m3 codes with the scales of its mode.
struct NormGradArgs {
    const void *Y;          // the output's gradient, rows ldy apart
    const void *X, *S;      // the norm's input, rows ldx apart, and its scales
    const void *W;
    const void *R;          // a gradient to add (rows ldr apart) or NULL
    void *D;                // [M][K]
    float *dW, *dB;         // [K]; dB (layer norm) or NULL
    float *ws;              // norm_grad_workspace_bytes
    int64_t ldy, ldx, ldr, M, K;
    float eps;
    int wt;                 // W's type: Y's or kTypeF32
};
struct SwigluGradArgs {
    const void *Y;          // the output's gradient, rows ldy apart
    const void *G, *U;      // gate and up, rows ldg and ldu apart
    const void *SG, *SU;    // their scales, block rows ldsg and ldsu apart
    void *D;                // [M][2 K]: the gate's gradient, then up's
    int64_t ldy, ldg, ldu, ldsg, ldsu, M, K;
};
size_t norm_grad_workspace_bytes(int64_t M, int64_t K, bool layer);
bool norm_grad_in_place(int64_t K);   // a row is read once, before it is written
hipError_t launch_norm_grad(const NormGradArgs &a, int type, int mode, bool layer, hipStream_t s);
hipError_t launch_swiglu_grad(const SwigluGradArgs &a, int type, int mode, hipStream_t s);

// A weight's gradient (wgrad.hip): C[e] = Y[rows of e]^T X[rows of e].
struct WgradArgs {
    const void *Y;          // [M][N] bf16, rows ldy elements apart
    const void *X;          // [x_rows][K] bf16 or e4m3
    const void *S;          // X's scales
    void *C;                // [E][N][K], fp32 or bf16
    float *ws;              // splits > 1: [splits][E][N][K]
    const int32_t *offsets; // [E + 1] or NULL (one group of M rows)
    const int32_t *rows;    // row of X of each row of Y, or NULL (row m takes row m)
    int64_t ldy, M, N, K, E, x_rows;
    int splits, accumulate;
};
struct WgradPlan {
    int tile;               // n and k of a workgroup's tile: 256 or 128
    int splits;             // parts of a group's rows
};
WgradPlan wgrad_plan(int64_t M, int64_t N, int64_t K, int64_t E);
hipError_t launch_wgrad(const WgradArgs &a, int mode, bool out_bf16, const WgradPlan &plan, hipStream_t s);
constexpr int kAmaxParts = 256;   // most partial maxima per matrix
hipError_t launch_row_quant(const RowQuantArgs &a, int x_type, int mode, bool gated, hipStream_t s);
bool small_tensor(int64_t M, int64_t K);   // measured per-tensor scale in one launch
hipError_t launch_small_tensor_quant(const RowQuantArgs &a, int x_type, hipStream_t s);
hipError_t launch_amax(const void *X, int64_t ldx, int x_type, int64_t groups, int64_t M, int64_t K, int parts_per_group,
                       uint32_t *parts, hipStream_t s);
hipError_t launch_quantize_b(const WeightQuantArgs &a, int x_type, int mode, hipStream_t s);
hipError_t launch_rmsnorm(const NormArgs &a, int x_type, int mode, hipStream_t s);
hipError_t launch_layernorm(const NormArgs &a, int x_type, int mode, hipStream_t s);

// Probes (probe.hip).
hipError_t launch_probe_mfma(int which, const void *a, const void *b, float *out, hipStream_t s);
hipError_t launch_probe_lds_dma(const void *src, const int32_t *perm, void *dst, hipStream_t s);
hipError_t launch_probe_lds_dma_narrow(int width, const void *src, const int32_t *perm, void *dst, hipStream_t s);
hipError_t launch_probe_mfma_scaled(int which, const void *a, const void *b, const void *sa, const void *sb,
                                    float *out, hipStream_t s);
hipError_t launch_probe_copy(const void *src, void *dst, int64_t bytes, hipStream_t s);
hipError_t launch_probe_stream_read(const void *src, int64_t bytes, int blocks, uint32_t *sink, hipStream_t s);
hipError_t launch_probe_mfma_peak(int which, int rounds, int blocks, const void *ops, uint32_t *sink,
                                  hipStream_t s);

}  // namespace dgp
