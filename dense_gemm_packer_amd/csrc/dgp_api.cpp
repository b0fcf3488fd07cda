// C-ABI layer of the gfx950 preshuffled-B GEMM library (include/dgp.h).
//
// Every entry point validates its arguments on the host first -- no HIP call
// is made for a rejected call -- then checks the device architecture, picks a
// compiled kernel and enqueues it on the caller's stream.  Nothing here
// allocates device memory or synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <vector>

#include "../../include/dgp.h"
#include "../../include/dgp_diag.h"
#include "common.h"
#include "launch.h"

using namespace dgp;

namespace dgp {

const KernelSpec *kernel_table(int *count)
{
    static const std::vector<KernelSpec> all = [] {
        std::vector<KernelSpec> v;
        int n = 0;
        const KernelSpec *t = tiled_kernels(&n);
        v.insert(v.end(), t, t + n);
        t = lds_kernels(&n);
        v.insert(v.end(), t, t + n);
        t = w4_kernels(&n);
        v.insert(v.end(), t, t + n);
        t = stream_kernels(&n);
        v.insert(v.end(), t, t + n);
        t = wave_kernels(&n);
        v.insert(v.end(), t, t + n);
        return v;
    }();
    *count = (int)all.size();
    return all.data();
}

const KernelSpec *grouped_table(int *count)
{
    static const std::vector<KernelSpec> all = [] {
        std::vector<KernelSpec> v;
        int n = 0;
        // (the one-wave-per-SIMD kernels first: a tile that both have is theirs)
        const KernelSpec *t = w4_grouped_kernels(&n);
        v.insert(v.end(), t, t + n);
        t = tiled_grouped_kernels(&n);
        v.insert(v.end(), t, t + n);
        t = stream_grouped_kernels(&n);
        v.insert(v.end(), t, t + n);
        return v;
    }();
    *count = (int)all.size();
    return all.data();
}

}  // namespace dgp

namespace {

thread_local char g_err[512];

dgp_status fail(dgp_status st, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

#define DGP_TRY(expr)                                                                          \
    do {                                                                                       \
        const dgp_status st_ = (expr);                                                         \
        if (st_ != DGP_OK)                                                                     \
            return st_;                                                                        \
    } while (0)

dgp_status ok()
{
    g_err[0] = '\0';
    return DGP_OK;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Bytes of a row of K elements (fp4 packs two elements per byte).
int64_t row_bytes(int dtype, int64_t K) { return dtype == DGP_BF16 ? 2 * K : dtype == DGP_FP4_E2M1 ? K / 2 : K; }
bool known_dtype(int dtype) { return dtype == DGP_BF16 || dtype == DGP_FP8_E4M3 || dtype == DGP_FP4_E2M1; }

// Per-row byte limit: keeps every in-tile offset of the kernels in 32 bits.
constexpr int64_t kMaxRowBytes = int64_t(1) << 23;

// ---------------------------------------------------------------- arch

dgp_status check_device_arch()
{
    // Per-device answer, 0 unknown, 1 gfx950, 2 other.  Atomic: host threads
    // may make their first calls concurrently (both then store the same value).
    static std::atomic<int> cached[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return fail(DGP_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    if (dev >= 0 && dev < 64 && cached[dev].load(std::memory_order_acquire) == 1)
        return DGP_OK;
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess)
        return fail(DGP_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
    dgp_status st = dgp_check_arch(prop.gcnArchName);
    if (dev >= 0 && dev < 64)
        cached[dev].store(st == DGP_OK ? 1 : 2, std::memory_order_release);
    if (st != DGP_OK)
        return fail(DGP_ERR_ARCH, "device %d is %s; this library runs on gfx950 only", dev,
                    prop.gcnArchName);
    return DGP_OK;
}

dgp_status hip_status(hipError_t e, const char *what)
{
    if (e != hipSuccess)
        return fail(DGP_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return ok();
}

// ------------------------------------------------------- kernel choice

struct Plan {
    const KernelSpec *spec;
    int tiles_m, tiles_n;
    int remap, group_m;
};

bool spec_fits(const KernelSpec &k, int64_t Ks)
{
    if (k.family == kTiled)
        return Ks % k.kt == 0;
    return true;   // stream: any K range that is a multiple of 128 bytes
}

// A kernel-table query; -1 in a field means "any".
struct Query {
    int family, dtype, scale, out, tm, tn;
    int kt = -1, wm = -1, depth = -1, pv = -1, pd = -1, sched = -1, lay = -1, copy = -1;
    int64_t K = 0;   // for kernels that need K to be a multiple of something
    bool dwords = true;   // the scales start at whole dwords, which those kernels need too
};

const KernelSpec *find_spec(const Query &q, const KernelSpec *(*table)(int *) = kernel_table)
{
    int n = 0;
    const KernelSpec *t = table(&n);
    for (int i = 0; i < n; ++i) {
        const KernelSpec &k = t[i];
        const int wm = k.family == kTiled ? k.p0 : k.waves;
        if (k.family == q.family && k.dtype == q.dtype && k.scale == q.scale && k.out == q.out && k.tm == q.tm &&
            k.tn == q.tn && (q.kt < 0 || k.kt == q.kt) && (q.wm < 0 || wm == q.wm) &&
            (q.depth < 0 || k.depth == q.depth) && (q.pv < 0 || k.pv == q.pv) && (q.pd < 0 || k.pd == q.pd) &&
            (q.sched < 0 || k.sched == q.sched) && (q.lay < 0 || (k.family == kTiled && k.lay == q.lay)) &&
            (q.copy < 0 || (k.family == kTiled && k.copy == q.copy)) && (k.k_mult == 0 || (q.dwords && q.K % k.k_mult == 0)))
            return &k;
    }
    return nullptr;
}

// Built-in per-shape choice.
const KernelSpec *default_spec(int dtype, int scale, int out, int64_t M, int64_t N, int64_t Ks, int split_k)
{
    // Decode-sized M streams the weight through the 16-row and one-row
    // tiles.  Larger M takes the tiled kernels, every scale mode included.
    if (M <= 32) {
        // Rules from cold sweeps of every 16-row and one-row tile at K = 7168
        // (every mode; M = 1, 2, 4 and 16; N 2048-16384; split 1-4).
        // u = strips x splits; ks(t, w) = the K-split tile t columns wide
        // (w waves, 8 unless given), st(t) = the streaming tile, wv(t, w, d) = the one-row VALU
        // tile with w waves and a d-step ring.
        const int64_t u = N / 16 * split_k;
        const bool fp8t = dtype == DGP_FP8_E4M3 && scale == DGP_SCALE_TENSOR;
        const bool mx4 = scale == DGP_SCALE_MX32;
        const bool bs = scale == DGP_SCALE_BLOCK128, mx8 = scale == DGP_SCALE_MX128;
        const auto ks = [&](int tn, int waves = 8) {
            Query q{kStream, dtype, scale, out, 16, tn};
            q.wm = waves;
            return find_spec(q);
        };
        const auto st = [&](int tn) {
            Query q{kStream, dtype, scale, out, 16, tn};
            q.wm = tn == 64 ? 4 : 2;
            return find_spec(q);
        };
        const auto wv = [&](int tn, int waves, int depth) {
            Query q{kWave, dtype, scale, out, 1, tn};
            q.wm = waves, q.depth = depth;
            return find_spec(q);
        };
        // One row, bf16 or per-tensor fp8: the one-row VALU tile (split 1 at
        // N = 2048: 6.4 vs 8.3 us bf16, 4.5 vs 5.3 us fp8; 0-4 % ahead of
        // the 16-row tiles at larger N and 1-11 % with splits), half strips
        // while one pass has fewer strips than CUs.
        if (M == 1 && (dtype == DGP_BF16 || fp8t)) {
            const KernelSpec *k = nullptr;
            if (split_k == 1 && N / 16 < 256)
                k = wv(8, 4, 8);
            else if (split_k == 1)
                k = dtype == DGP_BF16 ? wv(16, 8, 8) : wv(16, 4, 8);
            else
                k = (dtype == DGP_BF16 || split_k == 2) ? wv(16, 4, 8) : wv(16, 4, 4);
            if (k)
                return k;
        }
        // Blockscale and mxfp8 from 4 splits over at least 2048 strips x
        // splits: the streaming 16x64 tile (5-19 % ahead), whose A panel in
        // LDS serves four strips per wave.
        if (u >= 2048 && (bs || mx8) && split_k >= 4)
            return st(64);
        // mxfp4 in one pass over at most 512 strips: 16 waves per workgroup,
        // so each wave's K slice is one 4-step group of the guarded loop
        // (N = 2048: 5.6 vs 6.1 us at M = 16, 4.4 vs 5.0 at M = 1; N = 4096:
        // 6.2 vs 6.7 and 4.9 vs 5.4).
        if (mx4 && split_k == 1 && u <= 512) {
            const KernelSpec *k = u < 256 ? ks(M <= 4 ? 16 : 8, 16) : ks(u < 512 ? 16 : 32, 16);
            if (k)
                return k;
        }
        // Fewer strips x splits than CUs: half a strip per workgroup doubles
        // the workgroups with no second pass.
        if (u < 256)
            return ks(8);
        if (M <= 4) {
            // A few rows: A is cheap to re-read.  One pass: one strip per
            // workgroup with K over 8 waves.  With splits each wave's slice
            // is short, so 2 strips per workgroup lead (4-13 %), until the
            // streaming tile takes over from 2048 strips x splits at 4
            // splits; bf16 keeps one strip at 2 splits.
            if (fp8t || dtype == DGP_BF16 || mx4) {
                if (split_k == 1)
                    return ks(16);
                if (dtype == DGP_BF16)
                    return split_k == 2 ? ks(16) : ks(32);
                if (u < 1024)
                    return ks(16);
                return (split_k == 2 || u == 1024) ? ks(32) : st(64);
            }
            if (u < 512)
                return ks(16);
            // (mxfp8 in one or two passes: the 32-column tile, whose 3-step
            // ring keeps two workgroups per CU: 20.3-20.7 vs 20.9-21.1 us at
            // N = 16384)
            return (mx8 && u >= 1024 && split_k > 2) ? ks(64) : ks(32);
        }
        // More rows: A is read once per workgroup, so wider K-split tiles
        // (2 or 4 strips sharing each A fragment) lead from 512 strips x
        // splits (4-22 %); for mxfp4 the streaming tile leads again from
        // 2048.
        if (u < 512)
            return ks(16);
        if (mx4 && u >= 2048)
            return st(64);
        // (mxfp8 at 2 splits: 24.9 vs 25.6 us for the streaming tile at M =
        // 16, N = 16384)
        if (u < 1024 || fp8t || (mx8 && split_k == 2))
            return ks(32);
        // bf16 in one pass: the same 4 strips over 16 waves (M = 16, N =
        // 16384: 37.5 vs 38.8 us)
        if (dtype == DGP_BF16 && split_k == 1)
            if (const KernelSpec *k = ks(64, 16))
                return k;
        return ks(64);
    }
    // Small grids above 32 rows (e.g. bf16 128 x 256 x 256): fewer than 64
    // tiles of 128 x 128 and a weight of at most 8 MiB, in one pass.  The
    // 16-row K-split tile over ceil(M / 16) row tiles spreads K over the 8
    // waves of each workgroup where the 128 x 128 tile runs two workgroups
    // through K in sequence (2.8 vs 7.6 us per launch in a graph at 128 x 256
    // x 256); each row tile re-reads the weight, which at this size stays in
    // the L2.
    if (split_k == 1 && M <= 256 && ((M + 127) / 128) * ((N + 127) / 128) < 64 && N * Ks <= (int64_t(8) << 20)) {
        Query q{kStream, dtype, scale, out, 16, 16};
        q.wm = 8;
        if (const KernelSpec *k = find_spec(q))
            return k;
    }
    // Larger M: the tile whose grid finishes first.  A grid of t tiles (x
    // splits) runs in ceil(t / 256) rounds over the 256 CUs, and one round of
    // a 256x256 or 128x128 tile takes about 1.45 : 1 (bf16, fp8, mxfp8,
    // mxfp4; K = 2048 and 8192; blockscale's 8-wave 256x256 tile about
    // 2.05 : 1): 4096 x 4096 and 3072 x 3072 take the 256x256 tile, 2048 x
    // 2048 the 128x128 tile (91 vs 134 us; bf16 there now takes the 128x256
    // tile below).  Ties go to the larger tile.
    // bf16 and per-tensor fp8 run their 128x256 tile one wave per SIMD, two
    // workgroups per CU at once: the busiest CU's k tiles cost about 1.05
    // rounds of the 256x256 tile per pair and 0.74 for one alone (K = 8192:
    // 4096 x 6144 281 vs 314 us for the 256x256 tile, 4096 x 5120 260 vs
    // 307, 3072 x 4096 168 vs 153, 4096 x 4096 187 vs 178; fp8 alike).  A
    // lone tile against a 128x128 round: bf16 0.95 (2048 x 2048 x 8192: 77.8
    // vs 89.7 us), fp8 1.07 (51.0 vs 48.1 us).
    const auto rounds = [&](int64_t tm, int64_t tn) {
        return ((M + tm - 1) / tm * ((N + tn - 1) / tn) * split_k + 255) / 256;
    };
    const bool has_128x256 = scale == DGP_SCALE_NONE || scale == DGP_SCALE_TENSOR;   // (bf16 and fp8 per-tensor)
    const int64_t k128x256 = rounds(128, 256);   // 128x256 tiles on the busiest CU
    const int64_t c256 = (scale == DGP_SCALE_BLOCK128 ? 205 : 145) * rounds(256, 256),
                  c128x256 = has_128x256 ? 153 * (k128x256 / 2) + (dtype == DGP_BF16 ? 95 : 107) * (k128x256 % 2)
                                         : INT64_MAX,
                  c128 = 100 * rounds(128, 128);
    const KernelSpec *k = nullptr;
    if (c256 <= c128x256 && c256 <= c128) {
        // bf16, per-tensor fp8, mxfp8 and mxfp4: the one-wave-per-SIMD tile
        // with swizzled A rows (measured 8-18 % ahead of the 8-wave tile at
        // 4096 x 4096 x 8192); blockscale: the 8-wave tile.
        Query q{kTiled, dtype, scale, out, 256, 256};
        q.kt = 128;
        if (scale != DGP_SCALE_BLOCK128) {
            q.sched = kSchedW4, q.lay = kLaySwizzled;
        } else {
            q.wm = 1, q.depth = 2, q.pv = 0, q.pd = 4;
        }
        k = find_spec(q);
    } else if (c128x256 < c128) {
        // bf16 and per-tensor fp8: the one-wave-per-SIMD tile, 128 rows
        // (2048 x 4096 x 8192: 105.9 vs 123.8 us bf16, 60.5 vs 66.6 us fp8
        // against the 8-wave 128x256 tile in a sweep; bit-identical results)
        Query q{kTiled, dtype, scale, out, 128, 256};
        q.kt = 128, q.sched = kSchedW4, q.lay = kLaySwizzled;
        k = find_spec(q);
        if (!k) {
            q.sched = -1, q.lay = -1;
            k = find_spec(q);
        }
    }
    if (!k || !spec_fits(*k, Ks)) {
        Query q{kTiled, dtype, scale, out, 128, 128};
        q.kt = 128, q.pv = 0, q.pd = 4;
        k = find_spec(q);
    }
    return (k && spec_fits(*k, Ks)) ? k : nullptr;
}

// ---------------------------------------------------------- validation

struct GemmCall {
    const void *A, *Bs;
    void *C;
    int64_t M, N, K;
    int dtype, scale;
    const void *sA, *sB;
    int split_k;
    float *ws;
    size_t ws_bytes;
    const dgp_config *cfg;
    bool select_only = false;   // shapes and configuration only: no buffers checked
    bool lib_scratch = false;   // split-K partials go to the library's fixed array (ws unused)
};

// Scales that start at whole dwords.  (E8M0 bytes of 128 blocks need not: the
// kernels that copy them many bytes at a time are then left out.)
bool dword_scales(const GemmCall &c) { return (((uintptr_t)c.sA | (uintptr_t)c.sB) & 3u) == 0; }

// The kernel of `table` that the call's configuration names.
dgp_status configured_spec(const GemmCall &c, int64_t Ks, const KernelSpec *(*table)(int *), const KernelSpec **out_spec)
{
    const int fam = c.cfg->tile_m == 16 ? kStream : c.cfg->tile_m == 1 ? kWave : kTiled;
    if (c.cfg->waves_m < 0 || c.cfg->prefetch < 0)
        return fail(DGP_ERR_CONFIG, "waves_m and prefetch must be >= 0");
    if (c.cfg->schedule < 0 || c.cfg->schedule > kSchedW4)
        return fail(DGP_ERR_CONFIG, "schedule must be 0, 1, 2, 3 or 4 (got %d)", c.cfg->schedule);
    if (c.cfg->a_layout < 0 || c.cfg->a_layout > 2)
        return fail(DGP_ERR_CONFIG, "a_layout must be 0, 1 or 2 (got %d)", c.cfg->a_layout);
    if (c.cfg->a_copy < 0 || c.cfg->a_copy > 2)
        return fail(DGP_ERR_CONFIG, "a_copy must be 0, 1 or 2 (got %d)", c.cfg->a_copy);
    Query q{fam, c.dtype, c.scale, c.split_k > 1 ? kOutPartial : kOutBf16, c.cfg->tile_m, c.cfg->tile_n};
    if (fam == kTiled) {
        q.kt = c.cfg->tile_k;
        q.wm = c.cfg->waves_m > 0 ? c.cfg->waves_m : -1;
        q.depth = c.cfg->prefetch > 0 ? c.cfg->prefetch : -1;
        // (0, 0) = this tile's tuned default hints; any other pair must
        // name a compiled kernel exactly.
        if (c.cfg->preload_vmem != 0 || c.cfg->preload_dsrd != 0) {
            q.pv = c.cfg->preload_vmem;
            q.pd = c.cfg->preload_dsrd;
        }
        if (c.cfg->schedule > 0)
            q.sched = c.cfg->schedule;
        if (c.cfg->a_layout > 0)
            q.lay = c.cfg->a_layout - 1;
        q.copy = c.cfg->a_copy > 0 ? c.cfg->a_copy - 1 : kCopyAsync;
    } else {
        if (c.cfg->preload_vmem != 0 || c.cfg->preload_dsrd != 0)
            return fail(DGP_ERR_CONFIG, "the 16-row and one-row kernels take no preload hints");
        if (c.cfg->schedule != 0)
            return fail(DGP_ERR_CONFIG, "the 16-row and one-row kernels have no schedule choice");
        if (c.cfg->a_layout != 0 || c.cfg->a_copy != 0)
            return fail(DGP_ERR_CONFIG, "the 16-row and one-row kernels have no A layout or copy choice");
        q.wm = c.cfg->waves_m > 0 ? c.cfg->waves_m : -1;   // matched against waves per workgroup
        q.depth = c.cfg->prefetch > 0 ? c.cfg->prefetch : -1;
    }
    q.K = c.K;
    q.dwords = dword_scales(c);
    const KernelSpec *spec = find_spec(q, table);
    if (!spec)
        return fail(DGP_ERR_CONFIG,
                    "no compiled kernel for tile %dx%dx%d (waves_m %d, prefetch %d, preload %d,%d, schedule %d, "
                    "a_layout %d, a_copy %d) with this dtype/scale", c.cfg->tile_m, c.cfg->tile_n, c.cfg->tile_k,
                    c.cfg->waves_m, c.cfg->prefetch, c.cfg->preload_vmem, c.cfg->preload_dsrd, c.cfg->schedule,
                    c.cfg->a_layout, c.cfg->a_copy);
    if (!spec_fits(*spec, Ks))
        return fail(DGP_ERR_CONFIG, "tile_k=%d does not divide the K range of a split (%lld bytes)",
                    spec->kt, (long long)Ks);
    *out_spec = spec;
    return DGP_OK;
}

// Kernel choice for a validated call: the configured tile, or the built-in
// per-shape table.
dgp_status select_kernel(const GemmCall &c, int64_t Ks, Plan *plan)
{
    const int out = c.split_k > 1 ? kOutPartial : kOutBf16;
    const KernelSpec *spec = nullptr;
    if (c.cfg && c.cfg->tile_m > 0) {
        const dgp_status st = configured_spec(c, Ks, kernel_table, &spec);
        if (st != DGP_OK)
            return st;
    } else {
        spec = default_spec(c.dtype, c.scale, out, c.M, c.N, Ks, c.split_k);
        if (!spec)
            return fail(DGP_ERR_CONFIG, "no compiled kernel fits this shape");
    }
    plan->spec = spec;
    plan->tiles_m = (int)((c.M + spec->tm - 1) / spec->tm);
    plan->tiles_n = (int)((c.N + spec->tn - 1) / spec->tn);
    if (c.cfg && c.cfg->tile_m > 0) {
        plan->remap = c.cfg->xcd_remap;
        plan->group_m = c.cfg->group_m < 1 ? 1 : c.cfg->group_m;
    } else {
        plan->remap = spec->family == kTiled ? 1 : 0;
        plan->group_m = 8;
    }
    const int64_t grid = (int64_t)plan->tiles_m * plan->tiles_n * c.split_k;
    if (grid > INT32_MAX)
        return fail(DGP_ERR_SHAPE, "grid of %lld workgroups too large", (long long)grid);
    return ok();
}

// Types, sizes, scale mode and configuration of a call.
dgp_status validate_shape(const GemmCall &c)
{
    if (!known_dtype(c.dtype))
        return fail(DGP_ERR_DTYPE, "dtype %d is not DGP_BF16, DGP_FP8_E4M3 or DGP_FP4_E2M1", c.dtype);
    if (c.M < 0 || c.N < 0 || c.K < 0)
        return fail(DGP_ERR_SHAPE, "negative size M=%lld N=%lld K=%lld", (long long)c.M, (long long)c.N,
                    (long long)c.K);
    if (c.scale < DGP_SCALE_NONE || c.scale > DGP_SCALE_MX32)
        return fail(DGP_ERR_SCALE_MODE, "unknown scale mode %d", c.scale);
    if ((c.dtype == DGP_FP4_E2M1) != (c.scale == DGP_SCALE_MX32))
        return fail(DGP_ERR_SCALE_MODE, "DGP_FP4_E2M1 takes DGP_SCALE_MX32, and only it");
    if (c.dtype == DGP_BF16 && c.scale != DGP_SCALE_NONE)
        return fail(DGP_ERR_SCALE_MODE, "bf16 takes DGP_SCALE_NONE");
    if (c.dtype == DGP_FP8_E4M3 && (c.scale == DGP_SCALE_NONE || c.scale == DGP_SCALE_MX32))
        return fail(DGP_ERR_SCALE_MODE, "fp8 takes DGP_SCALE_TENSOR, DGP_SCALE_BLOCK128 or DGP_SCALE_MX128");
    if (c.split_k < 1)
        return fail(DGP_ERR_SPLITK, "split_k %d < 1", c.split_k);
    if (c.cfg) {
        if (c.cfg->preload_vmem < 0 || c.cfg->preload_dsrd < 0)
            return fail(DGP_ERR_CONFIG, "preload must be a pair of non-negative integers (got %d, %d)",
                        c.cfg->preload_vmem, c.cfg->preload_dsrd);
        if (c.cfg->xcd_remap != 0 && c.cfg->xcd_remap != 1)
            return fail(DGP_ERR_CONFIG, "xcd_remap must be 0 or 1");
        if (c.cfg->xcd_remap == 1 && c.cfg->group_m < 1)
            return fail(DGP_ERR_CONFIG, "group_m must be >= 1");
    }
    if (c.N % 16 != 0)
        return fail(DGP_ERR_SHAPE, "N=%lld is not a multiple of 16 (preshuffle block rows)", (long long)c.N);
    if (c.dtype == DGP_FP4_E2M1 && c.K % 2 != 0)
        return fail(DGP_ERR_SHAPE, "fp4 K=%lld is odd", (long long)c.K);
    const int64_t Kb = row_bytes(c.dtype, c.K);
    if (Kb % 128 != 0)
        return fail(DGP_ERR_SHAPE, "row bytes %lld (K=%lld) are not a multiple of 128", (long long)Kb, (long long)c.K);
    if (Kb > kMaxRowBytes)
        return fail(DGP_ERR_SHAPE, "K*element_bytes=%lld exceeds %lld", (long long)Kb, (long long)kMaxRowBytes);
    if (c.M > INT32_MAX / 2 || c.N > INT32_MAX / 2)
        return fail(DGP_ERR_SHAPE, "M or N too large");
    if (c.scale == DGP_SCALE_BLOCK128 && (c.K % 128 != 0 || c.N % 128 != 0))
        return fail(DGP_ERR_SHAPE, "blockscale needs K %% 128 == 0 and N %% 128 == 0 (K=%lld N=%lld)",
                    (long long)c.K, (long long)c.N);
    if (c.scale == DGP_SCALE_MX128 && c.K % 128 != 0)
        return fail(DGP_ERR_SHAPE, "mxfp8 needs K %% 128 == 0 (K=%lld)", (long long)c.K);
    if (c.K % c.split_k != 0)
        return fail(DGP_ERR_SPLITK, "split_k=%d does not divide K=%lld", c.split_k, (long long)c.K);
    const int64_t Ks = Kb / c.split_k;
    if (Ks % 128 != 0)
        return fail(DGP_ERR_SPLITK, "K range per split (%lld bytes) is not a multiple of 128", (long long)Ks);
    if ((c.scale == DGP_SCALE_BLOCK128 || c.scale == DGP_SCALE_MX128) && (c.K / c.split_k) % 128 != 0)
        return fail(DGP_ERR_SPLITK, "block scales need (K/split_k) %% 128 == 0");
    return DGP_OK;
}

// Operands and scales of a call with K > 0.
dgp_status validate_operands(const GemmCall &c)
{
    if (!c.A || !c.Bs)
        return fail(DGP_ERR_NULL, "A or Bs is NULL");
    if (!aligned16(c.A) || !aligned16(c.Bs))
        return fail(DGP_ERR_ALIGN, "A and Bs must be 16-byte aligned");
    if (c.scale != DGP_SCALE_NONE) {
        if (!c.sA || !c.sB)
            return fail(DGP_ERR_NULL, "scale mode needs sA and sB");
        if (c.scale != DGP_SCALE_MX128 && (((uintptr_t)c.sA & 3u) || ((uintptr_t)c.sB & 3u)))
            return fail(DGP_ERR_ALIGN, "fp32 scales sA and sB must be 4-byte aligned");
    }
    return DGP_OK;
}

dgp_status validate(const GemmCall &c, Plan *plan)
{
    dgp_status st = validate_shape(c);
    if (st != DGP_OK)
        return st;
    const int64_t Ks = row_bytes(c.dtype, c.K) / c.split_k;
    if (c.M == 0 || c.N == 0 || (c.select_only && c.K == 0)) {
        plan->spec = nullptr;
        return ok();
    }
    if (c.select_only)
        return select_kernel(c, Ks, plan);
    if (!c.C)
        return fail(DGP_ERR_NULL, "C is NULL");
    if (!aligned16(c.C))
        return fail(DGP_ERR_ALIGN, "C is not 16-byte aligned");
    if (c.K == 0) {
        plan->spec = nullptr;
        return ok();
    }
    st = validate_operands(c);
    if (st != DGP_OK)
        return st;
    if (c.split_k > 1) {
        const size_t need = dgp_splitk_workspace_bytes(c.M, c.N, c.split_k);
        if (c.lib_scratch) {
            if (need > kNoAllocScratchBytes)
                return fail(DGP_ERR_WORKSPACE,
                            "split_k*M*N*4 = %zu bytes exceeds the library's fixed scratch of %zu bytes "
                            "(DGP_NOALLOC_SCRATCH_BYTES); pass a workspace to dgp_gemm_preshuffle_splitk",
                            need, kNoAllocScratchBytes);
        } else {
            if (!c.ws)
                return fail(DGP_ERR_WORKSPACE, "split_k > 1 needs a workspace");
            if (!aligned16(c.ws))
                return fail(DGP_ERR_ALIGN, "workspace is not 16-byte aligned");
            if (c.ws_bytes < need)
                return fail(DGP_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", c.ws_bytes, need);
        }
    }

    return select_kernel(c, Ks, plan);
}

dgp_status run_gemm(const GemmCall &c, hipStream_t stream)
{
    Plan plan{};
    dgp_status st = validate(c, &plan);
    if (st != DGP_OK)
        return st;
    if (c.M == 0 || c.N == 0)
        return ok();
    st = check_device_arch();
    if (st != DGP_OK)
        return st;
    if (c.K == 0)
        return hip_status(launch_splitk_reduce(nullptr, c.C, c.M, c.N, 0, stream), "zero fill");
    float *ws = c.ws;
    if (c.lib_scratch && c.split_k > 1) {
        st = hip_status(noalloc_scratch(&ws), "address of the library's split-K scratch");
        if (st != DGP_OK)
            return st;
    }

    GemmArgs a{};
    a.A = (const uint8_t *)c.A;
    a.Bs = (const uint8_t *)c.Bs;
    a.C = c.C;
    a.ws = ws;
    a.sA = c.sA;
    a.sB = c.sB;
    a.M = (int)c.M;
    a.N = (int)c.N;
    a.K = (int)c.K;
    a.Kb = (int)row_bytes(c.dtype, c.K);
    a.Ks = a.Kb / c.split_k;
    a.tiles_m = plan.tiles_m;
    a.tiles_n = plan.tiles_n;
    a.splits = c.split_k;
    a.remap = plan.remap;
    a.group_m = plan.group_m;
    const dim3 grid((unsigned)((int64_t)plan.tiles_m * plan.tiles_n * c.split_k));
    plan.spec->launch(a, grid, stream);
    st = hip_status(hipGetLastError(), "GEMM launch");
    if (st != DGP_OK || c.split_k == 1)
        return st;
    return hip_status(launch_splitk_reduce(ws, c.C, c.M, c.N, c.split_k, stream), "split-K reduce launch");
}

// ------------------------------------------------- product by expert

// Most row tiles of tm rows that M rows split over E experts can make.
int64_t most_row_tiles(int64_t M, int64_t E, int64_t tm)
{
    const int64_t live = E < M ? E : M;   // experts that can have a row
    return (M + live * (tm - 1)) / tm;
}

// Built-in choice for M rows over E experts, of which the host knows the
// average only: the tile with the least estimated time, the fourth root of
// c^4 + m^4 (a maximum that is smooth where both count) of
//
//   c = (a + b k) (1 + s (x - 1)),  k = 128-byte k-steps, x = tiles on the busiest CU,
//   m = a + weight bytes / w,
//
// with a, b, s, w fitted per element type and tile to graph timings of 210
// random shapes (1 to 128 experts with 1 to 1000 rows each, unevenly filled, N
// 128 to 7168, K 256 to 8192; weights of 0.1 MB to 4 GB): a (us) is the launch,
// the search for the tile and the epilogue, b (us) the k-step of a tile that
// has its CU to itself, s what a further tile on the same CU adds (below 1
// where two overlap, above it where they contend), w (MB/us, at most the
// memory's 8) the rate at which the tile streams weights.  The fit is within
// 6-22 % of a timing, and the tile that it picks is on average 2-3 % slower
// than the fastest one of its shape (at worst 26-59 %, where the rows are far
// from evenly spread).  Any one tile left out costs up to 5 % more on average
// in some type, so all of them stay.
struct GroupedTile {
    int tm, tn;
    double a, b, s, w;
};
constexpr int kGroupedTiles = 8;
constexpr GroupedTile kGroupedCost[5][kGroupedTiles] = {
    // bf16
    {{16, 16, 1.17, 0.112, 0.64, 8.00}, {16, 32, 1.05, 0.153, 0.82, 8.00}, {16, 64, 1.51, 0.215, 1.01, 7.91},
     {64, 64, 2.19, 0.249, 1.15, 7.92}, {64, 128, 2.36, 0.283, 1.58, 6.26}, {64, 256, 3.00, 0.370, 1.78, 5.67},
     {128, 256, 4.41, 0.571, 1.61, 5.76}, {256, 256, 7.27, 0.986, 1.39, 6.92}},
    // fp8, per-tensor scales
    {{16, 16, 2.04, 0.104, 0.53, 8.00}, {16, 32, 1.95, 0.136, 0.61, 7.82}, {16, 64, 2.29, 0.186, 0.93, 6.77},
     {64, 64, 2.34, 0.260, 1.03, 8.00}, {64, 128, 2.61, 0.292, 1.44, 6.54}, {64, 256, 3.23, 0.360, 1.55, 5.85},
     {128, 256, 4.27, 0.671, 1.28, 5.66}, {256, 256, 7.24, 0.941, 1.44, 7.90}},
    // fp8, blockscale
    {{16, 16, 2.45, 0.103, 0.74, 8.00}, {16, 32, 1.98, 0.156, 0.64, 7.71}, {16, 64, 2.35, 0.197, 0.95, 6.58},
     {64, 64, 2.57, 0.317, 0.94, 8.00}, {64, 128, 2.87, 0.384, 1.33, 7.43}, {64, 256, 3.48, 0.598, 1.35, 6.20},
     {128, 256, 4.58, 0.857, 1.45, 7.21}, {256, 256, 5.63, 1.738, 1.19, 8.00}},
    // mxfp8
    {{16, 16, 2.39, 0.105, 0.75, 8.00}, {16, 32, 2.09, 0.155, 0.61, 8.00}, {16, 64, 2.37, 0.212, 0.95, 6.44},
     {64, 64, 2.52, 0.292, 0.96, 8.00}, {64, 128, 2.78, 0.352, 1.36, 6.77}, {64, 256, 3.36, 0.494, 1.48, 5.88},
     {128, 256, 4.46, 0.733, 1.51, 6.36}, {256, 256, 7.22, 1.031, 1.39, 8.00}},
    // mxfp4
    {{16, 16, 2.61, 0.128, 0.38, 8.00}, {16, 32, 2.48, 0.171, 0.52, 7.02}, {16, 64, 2.61, 0.245, 0.88, 5.83},
     {64, 64, 2.68, 0.379, 0.72, 8.00}, {64, 128, 3.01, 0.498, 1.08, 7.60}, {64, 256, 3.77, 0.569, 0.96, 5.43},
     {128, 256, 4.93, 0.811, 1.38, 6.20}, {256, 256, 7.05, 1.362, 1.25, 6.40}},
};

// Row tiles to expect: one expert's are known; several leave half a tile each
// unfilled on average once they have more rows than half a tile.
double expected_row_tiles(int64_t M, int64_t E, int tm)
{
    const int64_t live = E < M ? E : M;
    if (E == 1)
        return (double)((M + tm - 1) / tm);
    return 2 * M > live * tm ? std::max((double)live, (double)M / tm + 0.5 * live) : (double)live;
}

const KernelSpec *default_grouped_spec(const GemmCall &call, int64_t Kb, int64_t E)
{
    const int64_t M = call.M, N = call.N;
    const GroupedTile *best = nullptr;
    double least = 0;
    const double weights = (double)(E < M ? E : M) * (double)N * (double)Kb * 1e-6;
    for (const GroupedTile &t : kGroupedCost[call.scale]) {
        const double x = std::ceil(expected_row_tiles(M, E, t.tm) * (double)((N + t.tn - 1) / t.tn) / kNumCu);
        const double c = (t.a + t.b * (double)(Kb / 128)) * (1 + t.s * (x - 1)), m = t.a + weights / t.w;
        const double us4 = c * c * c * c + m * m * m * m;
        if (!best || us4 < least)
            best = &t, least = us4;
    }
    Query q{best->tm == 16 ? kStream : kTiled, call.dtype, call.scale, kOutBf16, best->tm, best->tn};
    q.K = call.K;
    q.dwords = dword_scales(call);
    return find_spec(q, grouped_table);
}

struct Experts {
    int64_t E, a_rows;
    const int32_t *offsets, *rows;
};

dgp_status run_grouped(const GemmCall &c, const Experts &x, hipStream_t stream)
{
    DGP_TRY(validate_shape(c));
    if (x.E < 0 || x.E > 65535 || x.a_rows < 0)
        return fail(DGP_ERR_SHAPE, "E=%lld experts, %lld rows of A", (long long)x.E, (long long)x.a_rows);
    if (c.K == 0)
        return fail(DGP_ERR_SHAPE, "the grouped product needs K > 0");
    if (c.M == 0 || c.N == 0 || x.E == 0)
        return ok();
    const int64_t Kb = row_bytes(c.dtype, c.K);
    if (!x.offsets)
        return fail(DGP_ERR_NULL, "offsets is NULL");
    if (((uintptr_t)x.offsets | (uintptr_t)x.rows) & 3u)
        return fail(DGP_ERR_ALIGN, "offsets and rows must be 4-byte aligned");
    if (x.rows ? x.a_rows < 1 : x.a_rows < c.M)
        return fail(DGP_ERR_SHAPE, "A has %lld rows, the product %lld", (long long)x.a_rows, (long long)c.M);
    if (x.rows && (x.a_rows > INT32_MAX / 2 || x.a_rows * Kb > (int64_t)0xFF000000))
        return fail(DGP_ERR_SHAPE, "with a row list A must be at most %lld bytes", (long long)0xFF000000);
    if (!c.C)
        return fail(DGP_ERR_NULL, "C is NULL");
    if (!aligned16(c.C))
        return fail(DGP_ERR_ALIGN, "C is not 16-byte aligned");
    DGP_TRY(validate_operands(c));
    const KernelSpec *spec = nullptr;
    if (c.cfg && c.cfg->tile_m > 0)
        DGP_TRY(configured_spec(c, Kb, grouped_table, &spec));
    else
        spec = default_grouped_spec(c, Kb, x.E);
    if (!spec)
        return fail(DGP_ERR_CONFIG, "no compiled grouped kernel fits this shape");
    const int64_t tiles_m = most_row_tiles(c.M, x.E, spec->tm), tiles_n = (c.N + spec->tn - 1) / spec->tn;
    // a launch's threads fit 32 bits, and so do the sums of the search for a
    // tile: 64 experts at a time, of which offsets that break the rule may give
    // each all M rows
    const int64_t scanned = std::min<int64_t>(x.E, 64) * ((c.M + spec->tm - 1) / spec->tm) + tiles_m;
    if (tiles_m * tiles_n > UINT32_MAX / (spec->waves * 64) || scanned > INT32_MAX)
        return fail(DGP_ERR_SHAPE, "M=%lld rows and N=%lld columns make too many %d x %d tiles", (long long)c.M,
                    (long long)c.N, spec->tm, spec->tn);
    DGP_TRY(check_device_arch());
    GemmArgs a{};
    a.A = (const uint8_t *)c.A, a.Bs = (const uint8_t *)c.Bs, a.C = c.C;
    a.sA = c.sA, a.sB = c.sB;
    a.M = (int)c.M, a.N = (int)c.N, a.K = (int)c.K;
    a.Kb = a.Ks = (int)Kb;
    a.tiles_m = (int)tiles_m, a.tiles_n = (int)tiles_n, a.splits = 1;
    const bool configured = c.cfg && c.cfg->tile_m > 0;
    a.remap = configured ? c.cfg->xcd_remap : 1;
    // (8 row tiles side by side: within 3 % of the best of 4, 8, 16 and 32 for 1 to
    // 32 experts in every mode; 2 and 1: 7 and 11 % slower on 16 experts of 1000
    // rows, bf16, N 4096, K 8192)
    a.group_m = configured && c.cfg->group_m > 0 ? c.cfg->group_m : 8;
    a.offsets = x.offsets, a.rows = x.rows;
    a.groups = (int)x.E, a.a_rows = (int)(x.rows ? x.a_rows : 0);
    spec->launch(a, dim3((unsigned)(tiles_m * tiles_n)), stream);
    return hip_status(hipGetLastError(), "grouped GEMM launch");
}

dgp_status shuffle(const void *src, void *dst, int64_t N, int64_t K, int dtype, void *stream, bool inverse)
{
    if (!known_dtype(dtype))
        return fail(DGP_ERR_DTYPE, "dtype %d is not DGP_BF16, DGP_FP8_E4M3 or DGP_FP4_E2M1", dtype);
    if (N < 0 || K < 0)
        return fail(DGP_ERR_SHAPE, "negative size N=%lld K=%lld", (long long)N, (long long)K);
    if (dtype == DGP_FP4_E2M1 && K % 2 != 0)
        return fail(DGP_ERR_SHAPE, "fp4 K=%lld is odd", (long long)K);
    const int64_t Kb = row_bytes(dtype, K);
    if (N % 16 != 0)
        return fail(DGP_ERR_SHAPE, "N=%lld is not a multiple of 16", (long long)N);
    if (Kb % 64 != 0)
        return fail(DGP_ERR_SHAPE, "K*element_bytes=%lld is not a multiple of 64", (long long)Kb);
    if (Kb >= (int64_t(1) << 27))
        return fail(DGP_ERR_SHAPE, "K*element_bytes=%lld too large", (long long)Kb);
    if (N / 16 > INT32_MAX)
        return fail(DGP_ERR_SHAPE, "N too large");
    if (N == 0 || K == 0)
        return ok();
    if (!src || !dst)
        return fail(DGP_ERR_NULL, "source or destination is NULL");
    if (!aligned16(src) || !aligned16(dst))
        return fail(DGP_ERR_ALIGN, "source and destination must be 16-byte aligned");
    const uintptr_t s = (uintptr_t)src, d = (uintptr_t)dst, n = (uintptr_t)(N * Kb);
    if (s < d + n && d < s + n)
        return fail(DGP_ERR_SHAPE, "source and destination overlap");
    dgp_status st = check_device_arch();
    if (st != DGP_OK)
        return st;
    return hip_status(launch_preshuffle(src, dst, N, Kb, inverse, (hipStream_t)stream), "preshuffle launch");
}

// ------------------------------------------------- quantising operators

// Rules shared by the operators that write a GEMM operand of `M` rows and `K`
// elements from rows of type x_type: types, sizes, the operand's own K rule.
int input_size(int x_type) { return x_type == DGP_F32 ? 4 : (x_type == DGP_BF16 || x_type == DGP_F16) ? 2 : 0; }

dgp_status check_operand(int x_type, int64_t M, int64_t K, int scale_mode, bool allow_none)
{
    if (!input_size(x_type))
        return fail(DGP_ERR_DTYPE, "input type %d is not DGP_BF16, DGP_F16 or DGP_F32", x_type);
    if (scale_mode < (allow_none ? DGP_SCALE_NONE : DGP_SCALE_TENSOR) || scale_mode > DGP_SCALE_MX32)
        return fail(DGP_ERR_SCALE_MODE, "scale mode %d is not one this operator writes", scale_mode);
    if (M < 0 || K < 0)
        return fail(DGP_ERR_SHAPE, "negative size M=%lld K=%lld", (long long)M, (long long)K);
    const int dtype = scale_mode == DGP_SCALE_NONE ? DGP_BF16 : scale_mode == DGP_SCALE_MX32 ? DGP_FP4_E2M1 : DGP_FP8_E4M3;
    if (K % 2 != 0 || row_bytes(dtype, K) % 128 != 0)
        return fail(DGP_ERR_SHAPE, "K=%lld: the operand's rows are not a multiple of 128 bytes", (long long)K);
    if (row_bytes(dtype, K) > kMaxRowBytes)
        return fail(DGP_ERR_SHAPE, "operand rows of %lld bytes exceed %lld", (long long)row_bytes(dtype, K),
                    (long long)kMaxRowBytes);
    if (M > INT32_MAX / 2)
        return fail(DGP_ERR_SHAPE, "M too large");
    return DGP_OK;
}

// A strided input: rows ld elements apart, every row 16-byte aligned.
dgp_status check_rows(const void *p, int64_t ld, int64_t K, int x_type, const char *what)
{
    if (!p)
        return fail(DGP_ERR_NULL, "%s is NULL", what);
    if (ld < K)
        return fail(DGP_ERR_SHAPE, "%s: row stride %lld below K=%lld", what, (long long)ld, (long long)K);
    if (!aligned16(p) || (ld * input_size(x_type)) % 16 != 0)
        return fail(DGP_ERR_ALIGN, "%s: rows must be 16-byte aligned", what);
    return DGP_OK;
}

// Codes and scales: Q 16-byte aligned; S present where the mode writes block
// scales, 4-byte aligned where they are fp32.
dgp_status check_codes(const void *Q, const void *S, const float *scale, int scale_mode)
{
    if (!Q)
        return fail(DGP_ERR_NULL, "Q is NULL");
    if (!aligned16(Q))
        return fail(DGP_ERR_ALIGN, "Q is not 16-byte aligned");
    const bool writes = scale_mode != DGP_SCALE_NONE && !(scale_mode == DGP_SCALE_TENSOR && scale);
    if (writes && !S)
        return fail(DGP_ERR_NULL, "S is NULL");
    if (scale && scale_mode != DGP_SCALE_TENSOR)
        return fail(DGP_ERR_SCALE_MODE, "a given scale goes with DGP_SCALE_TENSOR only");
    if ((scale_mode == DGP_SCALE_TENSOR || scale_mode == DGP_SCALE_BLOCK128) && (((uintptr_t)S | (uintptr_t)scale) & 3u))
        return fail(DGP_ERR_ALIGN, "fp32 scales must be 4-byte aligned");
    return DGP_OK;
}

// An output of M dense rows of out_row bytes against an input of M rows of
// in_row bytes, in_ld bytes apart: apart in memory, or (may_be_same: kernels
// that read a row's elements before the same threads write them) the same
// dense rows.
dgp_status check_apart(const void *out, int64_t out_row, const void *in, int64_t in_row, int64_t in_ld, int64_t M,
                       bool may_be_same, const char *what)
{
    if (!out || !in || (may_be_same && out == in && out_row == in_row && (M == 1 || in_ld == in_row)))
        return DGP_OK;
    const uintptr_t o = (uintptr_t)out, i = (uintptr_t)in;
    if (o < i + (uintptr_t)((M - 1) * in_ld + in_row) && i < o + (uintptr_t)(M * out_row))
        return fail(DGP_ERR_SHAPE, "%s overlap", what);
    return DGP_OK;
}

// Bytes of a row of codes and of its scales (0 where a row has none).
int64_t code_row(int64_t K, int scale_mode)
{
    return scale_mode == DGP_SCALE_NONE ? 2 * K : scale_mode == DGP_SCALE_MX32 ? K / 2 : K;
}
int64_t scale_row(int64_t K, int scale_mode)
{
    return scale_mode == DGP_SCALE_BLOCK128 ? K / 128 * 4 : scale_mode == DGP_SCALE_MX128 ? K / 128
           : scale_mode == DGP_SCALE_MX32 ? K / 32 : 0;
}

// Bytes of scales that a call of M rows writes (a given per-tensor scale: none).
int64_t scale_bytes(int64_t M, int64_t K, int scale_mode, const float *scale)
{
    return scale_mode == DGP_SCALE_TENSOR ? (scale ? 0 : 4) : M * scale_row(K, scale_mode);
}

// Q and S of an operand against one of its strided inputs.
dgp_status check_codes_apart(const void *Q, const void *S, const float *scale, int scale_mode, const void *X, int64_t ldx,
                             int x_type, int64_t M, int64_t K, const char *what)
{
    const int64_t in = input_size(x_type), s_bytes = scale_bytes(M, K, scale_mode, scale);
    DGP_TRY(check_apart(Q, code_row(K, scale_mode), X, K * in, ldx * in, M, x_type == DGP_BF16, what));
    // (S as one dense row against all of X as another)
    return check_apart(s_bytes ? S : nullptr, s_bytes, X, ((M - 1) * ldx + K) * in, 0, 1, false, what);
}

// Q, S and H (the norm's residual output, or NULL) against an input that every
// row reads: the norm's weight, a given scale.
dgp_status check_outputs_apart(const void *Q, const void *S, const void *H, const float *scale, int scale_mode, int x_type,
                               int64_t M, int64_t K, const void *in, int64_t in_bytes, const char *what)
{
    const int64_t s_bytes = scale_bytes(M, K, scale_mode, scale);
    DGP_TRY(check_apart(Q, M * code_row(K, scale_mode), in, in_bytes, 0, 1, false, what));
    DGP_TRY(check_apart(s_bytes ? S : nullptr, s_bytes, in, in_bytes, 0, 1, false, what));
    return check_apart(H, M * K * input_size(x_type), in, in_bytes, 0, 1, false, what);
}

// The scales against the codes, and (the norm) the residual output.
dgp_status check_scales_apart(const void *Q, const void *S, const void *H, const float *scale, int scale_mode, int x_type,
                              int64_t M, int64_t K)
{
    const int64_t s_bytes = scale_bytes(M, K, scale_mode, scale);
    if (s_bytes == 0)
        return DGP_OK;
    DGP_TRY(check_apart(S, s_bytes, Q, M * code_row(K, scale_mode), 0, 1, false, "Q and S"));
    return check_apart(S, s_bytes, H, M * K * input_size(x_type), 0, 1, false, "S and residual output");
}

dgp_status check_amax_workspace(int64_t groups, const float *ws, size_t ws_bytes)
{
    const size_t need = dgp_quantize_workspace_bytes(groups, DGP_SCALE_TENSOR);
    if (!ws)
        return fail(DGP_ERR_WORKSPACE, "DGP_SCALE_TENSOR without a given scale needs a workspace");
    if ((uintptr_t)ws & 3u)
        return fail(DGP_ERR_ALIGN, "workspace is not 4-byte aligned");
    if (ws_bytes < need)
        return fail(DGP_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
    return DGP_OK;
}

// Workgroups per matrix for the largest-magnitude pass: four 2 KiB (fp32: 4
// KiB) pieces each, at most kAmaxParts.
int amax_parts(int64_t M, int64_t K)
{
    const int64_t n = (M * K / 8 + 1023) / 1024;
    return (int)(n < 1 ? 1 : n > kAmaxParts ? kAmaxParts : n);
}

}  // namespace

// ====================================================================== ABI

extern "C" {

dgp_status dgp_preshuffle_b(const void *B, void *Bs, int64_t N, int64_t K, int dtype, void *stream)
{
    return shuffle(B, Bs, N, K, dtype, stream, false);
}

dgp_status dgp_unshuffle_b(const void *Bs, void *B, int64_t N, int64_t K, int dtype, void *stream)
{
    return shuffle(Bs, B, N, K, dtype, stream, true);
}

dgp_status dgp_gemm_preshuffle(const void *A, const void *Bs, void *C, int64_t M, int64_t N, int64_t K,
                               int dtype, int scale_mode, const void *sA, const void *sB,
                               const dgp_config *cfg, void *stream)
{
    GemmCall c{A, Bs, C, M, N, K, dtype, scale_mode, sA, sB, 1, nullptr, 0, cfg};
    return run_gemm(c, (hipStream_t)stream);
}

size_t dgp_splitk_workspace_bytes(int64_t M, int64_t N, int split_k)
{
    if (split_k <= 1 || M <= 0 || N <= 0)
        return 0;
    return (size_t)split_k * (size_t)M * (size_t)N * sizeof(float);
}

dgp_status dgp_gemm_preshuffle_splitk(const void *A, const void *Bs, void *C, int64_t M, int64_t N,
                                      int64_t K, int dtype, int scale_mode, const void *sA,
                                      const void *sB, int split_k, float *ws, size_t ws_bytes,
                                      const dgp_config *cfg, void *stream)
{
    GemmCall c{A, Bs, C, M, N, K, dtype, scale_mode, sA, sB, split_k, ws, ws_bytes, cfg};
    return run_gemm(c, (hipStream_t)stream);
}

dgp_status dgp_gemm_preshuffle_splitk_noalloc(const void *A, const void *Bs, void *C, int64_t M, int64_t N,
                                              int64_t K, int dtype, int scale_mode, const void *sA,
                                              const void *sB, int split_k, const dgp_config *cfg, void *stream)
{
    GemmCall c{A, Bs, C, M, N, K, dtype, scale_mode, sA, sB, split_k, nullptr, 0, cfg};
    c.lib_scratch = true;
    return run_gemm(c, (hipStream_t)stream);
}

size_t dgp_quantize_workspace_bytes(int64_t E, int scale_mode)
{
    return scale_mode == DGP_SCALE_TENSOR && E > 0 ? (size_t)E * kAmaxParts * sizeof(uint32_t) : 0;
}

dgp_status dgp_quantize(const void *X, int64_t ldx, int x_type, void *Q, void *S, const float *scale, int64_t M,
                        int64_t K, int scale_mode, float *ws, size_t ws_bytes, void *stream)
{
    DGP_TRY(check_operand(x_type, M, K, scale_mode, false));
    if (M == 0 || K == 0)
        return ok();
    DGP_TRY(check_rows(X, ldx, K, x_type, "X"));
    DGP_TRY(check_codes(Q, S, scale, scale_mode));
    const bool measure = scale_mode == DGP_SCALE_TENSOR && !scale;
    if (measure)
        DGP_TRY(check_amax_workspace(1, ws, ws_bytes));
    DGP_TRY(check_codes_apart(Q, S, scale, scale_mode, X, ldx, x_type, M, K, "X and Q or S"));
    DGP_TRY(check_outputs_apart(Q, S, nullptr, scale, scale_mode, x_type, M, K, scale, 4, "Q and the given scale"));
    DGP_TRY(check_scales_apart(Q, S, nullptr, scale, scale_mode, x_type, M, K));
    DGP_TRY(check_device_arch());
    RowQuantArgs a{};
    a.X = X, a.Q = Q, a.S = S, a.scale = scale;
    a.ldx = a.ldu = ldx, a.M = M, a.K = K;
    if (measure && small_tensor(M, K))
        return hip_status(launch_small_tensor_quant(a, x_type, (hipStream_t)stream), "quantisation launch");
    if (measure) {
        a.nparts = amax_parts(M, K);
        a.parts = (const uint32_t *)ws;
        DGP_TRY(hip_status(launch_amax(X, ldx, x_type, 1, M, K, a.nparts, (uint32_t *)ws, (hipStream_t)stream),
                           "largest-magnitude launch"));
    }
    return hip_status(launch_row_quant(a, x_type, scale_mode, false, (hipStream_t)stream), "quantisation launch");
}

dgp_status dgp_quantize_b(const void *B, int x_type, void *Bs, void *sB, int64_t E, int64_t N, int64_t K,
                          int scale_mode, float *ws, size_t ws_bytes, void *stream)
{
    DGP_TRY(check_operand(x_type, 0, K, scale_mode, false));
    if (E < 0 || N < 0 || E > 65535 || N > INT32_MAX / 2 || E * N > INT32_MAX / 2)
        return fail(DGP_ERR_SHAPE, "E=%lld matrices of N=%lld rows", (long long)E, (long long)N);
    if (N % 16 != 0)
        return fail(DGP_ERR_SHAPE, "N=%lld is not a multiple of 16 (preshuffle block rows)", (long long)N);
    if (scale_mode == DGP_SCALE_BLOCK128 && N % 128 != 0)
        return fail(DGP_ERR_SHAPE, "blockscale needs N %% 128 == 0 (N=%lld)", (long long)N);
    if (E * N / 16 * (K / 128) > INT32_MAX)
        return fail(DGP_ERR_SHAPE, "too many operand blocks");
    if (E == 0 || N == 0 || K == 0)
        return ok();
    DGP_TRY(check_rows(B, K, K, x_type, "B"));
    DGP_TRY(check_codes(Bs, sB, nullptr, scale_mode));
    const bool measure = scale_mode == DGP_SCALE_TENSOR;
    if (measure)
        DGP_TRY(check_amax_workspace(E, ws, ws_bytes));
    const int64_t b_row = K * input_size(x_type), scales = scale_mode == DGP_SCALE_BLOCK128 ? E * (N / 128) * (K / 128) * 4
                          : measure ? E * 4 : E * N * scale_row(K, scale_mode);
    DGP_TRY(check_apart(Bs, code_row(K, scale_mode), B, b_row, b_row, E * N, false, "B and Bs"));
    DGP_TRY(check_apart(sB, scales, B, E * N * b_row, E * N * b_row, 1, false, "B and sB"));
    DGP_TRY(check_apart(sB, scales, Bs, E * N * code_row(K, scale_mode), 0, 1, false, "Bs and sB"));
    DGP_TRY(check_device_arch());
    WeightQuantArgs a{};
    a.B = B, a.Q = Bs, a.S = sB;
    a.rows = E * N, a.N = N, a.K = K;
    if (measure) {
        a.nparts = amax_parts(N, K);
        a.parts = (const uint32_t *)ws;
        DGP_TRY(hip_status(launch_amax(B, K, x_type, E, N, K, a.nparts, (uint32_t *)ws, (hipStream_t)stream),
                           "largest-magnitude launch"));
    }
    return hip_status(launch_quantize_b(a, x_type, scale_mode, (hipStream_t)stream), "weight quantisation launch");
}

dgp_status dgp_rmsnorm_quantize(const void *X, int64_t ldx, const void *R, int64_t ldr, int x_type, const void *W,
                                int w_type, float eps, void *Q, void *S, const float *scale, void *H, int64_t M,
                                int64_t K, int scale_mode, void *stream)
{
    DGP_TRY(check_operand(x_type, M, K, scale_mode, true));
    if (w_type != x_type && w_type != DGP_F32)
        return fail(DGP_ERR_DTYPE, "weight type %d is neither X's type nor DGP_F32", w_type);
    if (!(eps >= 0.0f) || !(eps <= 3.0e38f))
        return fail(DGP_ERR_SHAPE, "eps must be finite and not negative");
    if (M == 0 || K == 0)
        return ok();
    DGP_TRY(check_rows(X, ldx, K, x_type, "X"));
    if (R)
        DGP_TRY(check_rows(R, ldr, K, x_type, "residual"));
    if (!W)
        return fail(DGP_ERR_NULL, "weight is NULL");
    if (!aligned16(W) || !aligned16(H))
        return fail(DGP_ERR_ALIGN, "weight and residual output must be 16-byte aligned");
    if (scale_mode == DGP_SCALE_TENSOR && !scale)
        return fail(DGP_ERR_NULL, "DGP_SCALE_TENSOR needs a given scale here");
    DGP_TRY(check_codes(Q, S, scale, scale_mode));
    DGP_TRY(check_codes_apart(Q, S, scale, scale_mode, X, ldx, x_type, M, K, "X and Q or S"));
    DGP_TRY(check_codes_apart(Q, S, scale, scale_mode, R, ldr, x_type, M, K, "residual and Q or S"));
    const int64_t in = input_size(x_type);
    DGP_TRY(check_apart(H, K * in, X, K * in, ldx * in, M, true, "X and residual output"));
    DGP_TRY(check_apart(H, K * in, R, K * in, ldr * in, M, true, "residual and residual output"));
    DGP_TRY(check_apart(H, K * in, Q, code_row(K, scale_mode), code_row(K, scale_mode), M, false, "Q and residual output"));
    DGP_TRY(check_outputs_apart(Q, S, H, scale, scale_mode, x_type, M, K, W, K * input_size(w_type), "weight and Q, S or residual output"));
    DGP_TRY(check_outputs_apart(Q, S, H, scale, scale_mode, x_type, M, K, scale, 4, "the given scale and Q or residual output"));
    DGP_TRY(check_scales_apart(Q, S, H, scale, scale_mode, x_type, M, K));
    DGP_TRY(check_device_arch());
    NormArgs a{};
    a.X = X, a.R = R, a.W = W, a.Q = Q, a.S = S, a.H = H, a.scale = scale;
    a.ldx = ldx, a.ldr = ldr, a.M = M, a.K = K;
    a.eps = eps, a.wt = w_type;
    return hip_status(launch_rmsnorm(a, x_type, scale_mode, (hipStream_t)stream), "norm launch");
}

dgp_status dgp_swiglu_quantize(const void *G, int64_t ldg, const void *U, int64_t ldu, int x_type, void *Q, void *S,
                               const float *scale, int64_t M, int64_t K, int scale_mode, void *stream)
{
    DGP_TRY(check_operand(x_type, M, K, scale_mode, true));
    if (M == 0 || K == 0)
        return ok();
    DGP_TRY(check_rows(G, ldg, K, x_type, "gate"));
    DGP_TRY(check_rows(U, ldu, K, x_type, "up"));
    if (scale_mode == DGP_SCALE_TENSOR && !scale)
        return fail(DGP_ERR_NULL, "DGP_SCALE_TENSOR needs a given scale here");
    DGP_TRY(check_codes(Q, S, scale, scale_mode));
    DGP_TRY(check_codes_apart(Q, S, scale, scale_mode, G, ldg, x_type, M, K, "gate and Q or S"));
    DGP_TRY(check_codes_apart(Q, S, scale, scale_mode, U, ldu, x_type, M, K, "up and Q or S"));
    DGP_TRY(check_outputs_apart(Q, S, nullptr, scale, scale_mode, x_type, M, K, scale, 4, "Q and the given scale"));
    DGP_TRY(check_scales_apart(Q, S, nullptr, scale, scale_mode, x_type, M, K));
    DGP_TRY(check_device_arch());
    RowQuantArgs a{};
    a.X = G, a.U = U, a.Q = Q, a.S = S, a.scale = scale;
    a.ldx = ldg, a.ldu = ldu, a.M = M, a.K = K;
    return hip_status(launch_row_quant(a, x_type, scale_mode, true, (hipStream_t)stream), "gated activation launch");
}

dgp_status dgp_gemm_preshuffle_grouped(const void *A, int64_t a_rows, const void *Bs, void *C, int64_t M, int64_t N,
                                       int64_t K, int64_t E, const int32_t *offsets, const int32_t *rows, int dtype,
                                       int scale_mode, const void *sA, const void *sB, const dgp_config *cfg,
                                       void *stream)
{
    GemmCall c{A, Bs, C, M, N, K, dtype, scale_mode, sA, sB, 1, nullptr, 0, cfg};
    return run_grouped(c, Experts{E, a_rows, offsets, rows}, (hipStream_t)stream);
}

dgp_status dgp_check_arch(const char *name)
{
    if (!name)
        return DGP_ERR_ARCH;
    // "gfx950" optionally followed by ":feature" suffixes.
    if (strncmp(name, "gfx950", 6) == 0 && (name[6] == '\0' || name[6] == ':'))
        return DGP_OK;
    return DGP_ERR_ARCH;
}

const char *dgp_status_string(int s)
{
    switch (s) {
    case DGP_OK: return "DGP_OK";
    case DGP_ERR_NULL: return "DGP_ERR_NULL";
    case DGP_ERR_SHAPE: return "DGP_ERR_SHAPE";
    case DGP_ERR_ALIGN: return "DGP_ERR_ALIGN";
    case DGP_ERR_DTYPE: return "DGP_ERR_DTYPE";
    case DGP_ERR_SCALE_MODE: return "DGP_ERR_SCALE_MODE";
    case DGP_ERR_SPLITK: return "DGP_ERR_SPLITK";
    case DGP_ERR_WORKSPACE: return "DGP_ERR_WORKSPACE";
    case DGP_ERR_CONFIG: return "DGP_ERR_CONFIG";
    case DGP_ERR_ARCH: return "DGP_ERR_ARCH";
    case DGP_ERR_HIP: return "DGP_ERR_HIP";
    default: return "DGP_ERR_UNKNOWN";
    }
}

const char *dgp_last_error(void) { return g_err; }

// ------------------------------------------------------------ diagnostics

dgp_status dgp_tile_of_workgroup(int64_t wg, int64_t tiles_m, int64_t tiles_n, int64_t splits, int xcd_remap,
                                 int group_m, int64_t out[3])
{
    if (!out)
        return fail(DGP_ERR_NULL, "out is NULL");
    if (tiles_m < 1 || tiles_n < 1 || splits < 1 || wg < 0 || wg >= tiles_m * tiles_n * splits ||
        (xcd_remap != 0 && xcd_remap != 1) || tiles_m * tiles_n * splits > INT32_MAX)
        return fail(DGP_ERR_SHAPE, "bad tile-map arguments");
    const TileCoord c = tile_of_workgroup<int64_t>(wg, tiles_m, tiles_n, splits, xcd_remap, group_m);
    out[0] = c.tm;
    out[1] = c.tn;
    out[2] = c.s;
    return ok();
}

dgp_status dgp_tile_map(int64_t tiles_m, int64_t tiles_n, int64_t splits, int xcd_remap, int group_m,
                        int64_t *out, int64_t out_len)
{
    if (!out)
        return fail(DGP_ERR_NULL, "out is NULL");
    if (tiles_m < 1 || tiles_n < 1 || splits < 1 || (xcd_remap != 0 && xcd_remap != 1) ||
        tiles_m * tiles_n * splits > INT32_MAX)
        return fail(DGP_ERR_SHAPE, "bad tile-map arguments");
    const int64_t total = tiles_m * tiles_n * splits;
    if (out_len < 3 * total)
        return fail(DGP_ERR_SHAPE, "out holds %lld values, the grid needs %lld", (long long)out_len,
                    (long long)(3 * total));
    for (int64_t wg = 0; wg < total; ++wg) {
        const TileCoord c = tile_of_workgroup<int64_t>(wg, tiles_m, tiles_n, splits, xcd_remap, group_m);
        out[3 * wg] = c.tm;
        out[3 * wg + 1] = c.tn;
        out[3 * wg + 2] = c.s;
    }
    return ok();
}

int dgp_lds_poison(void)
{
    return dgp::kLdsPoison ? 1 : 0;
}

int dgp_kernel_count(void)
{
    int n = 0;
    kernel_table(&n);
    return n;
}

dgp_status dgp_kernel_info(int index, dgp_config *cfg, int *dtype, int *scale_mode, int *split_out)
{
    int n = 0;
    const KernelSpec *t = kernel_table(&n);
    if (index < 0 || index >= n)
        return fail(DGP_ERR_SHAPE, "kernel index %d out of range [0, %d)", index, n);
    if (!cfg || !dtype || !scale_mode || !split_out)
        return fail(DGP_ERR_NULL, "NULL output");
    const KernelSpec &k = t[index];
    cfg->tile_m = k.tm;
    cfg->tile_n = k.tn;
    cfg->tile_k = k.family == kTiled ? k.kt : 0;
    cfg->xcd_remap = k.family == kTiled ? 1 : 0;
    cfg->group_m = 8;
    cfg->preload_vmem = k.pv;
    cfg->preload_dsrd = k.pd;
    cfg->waves_m = k.family == kTiled ? k.p0 : k.waves;
    cfg->prefetch = k.depth;
    cfg->schedule = k.sched;
    cfg->a_layout = k.family == kTiled ? k.lay + 1 : 0;
    cfg->a_copy = k.family == kTiled ? k.copy + 1 : 0;
    *dtype = k.dtype;
    *scale_mode = k.scale;
    *split_out = k.out == kOutPartial ? 1 : 0;
    return ok();
}

dgp_status dgp_select_kernel(int64_t M, int64_t N, int64_t K, int dtype, int scale_mode, int split_k,
                             const dgp_config *cfg, int *index)
{
    if (!index)
        return fail(DGP_ERR_NULL, "NULL index");
    GemmCall c{nullptr, nullptr, nullptr, M, N, K, dtype, scale_mode, nullptr, nullptr, split_k, nullptr, 0, cfg};
    c.select_only = true;
    Plan plan{};
    const dgp_status st = validate(c, &plan);
    if (st != DGP_OK)
        return st;
    *index = -1;
    if (plan.spec) {
        int n = 0;
        *index = (int)(plan.spec - kernel_table(&n));
    }
    return ok();
}

dgp_status dgp_probe_mfma_layout(int which, const void *a, const void *b, float *out, void *stream)
{
    if (which != 0 && which != 1)
        return fail(DGP_ERR_CONFIG, "which must be 0 or 1");
    if (!a || !b || !out)
        return fail(DGP_ERR_NULL, "NULL buffer");
    if (!aligned16(a) || !aligned16(b) || !aligned16(out))
        return fail(DGP_ERR_ALIGN, "buffers must be 16-byte aligned");
    dgp_status st = check_device_arch();
    if (st != DGP_OK)
        return st;
    return hip_status(launch_probe_mfma(which, a, b, out, (hipStream_t)stream), "probe launch");
}

dgp_status dgp_probe_mfma_scaled(int which, const void *a, const void *b, const void *sa, const void *sb,
                                 float *out, void *stream)
{
    if (which != 0 && which != 1)
        return fail(DGP_ERR_CONFIG, "which must be 0 or 1");
    if (!a || !b || !sa || !sb || !out)
        return fail(DGP_ERR_NULL, "NULL buffer");
    if (!aligned16(a) || !aligned16(b) || !aligned16(out))
        return fail(DGP_ERR_ALIGN, "a, b and out must be 16-byte aligned");
    dgp_status st = check_device_arch();
    if (st != DGP_OK)
        return st;
    return hip_status(launch_probe_mfma_scaled(which, a, b, sa, sb, out, (hipStream_t)stream), "probe launch");
}

dgp_status dgp_probe_lds_dma(const void *src, const int32_t *perm, void *dst, void *stream)
{
    if (!src || !perm || !dst)
        return fail(DGP_ERR_NULL, "NULL buffer");
    if (!aligned16(src) || !aligned16(dst))
        return fail(DGP_ERR_ALIGN, "buffers must be 16-byte aligned");
    dgp_status st = check_device_arch();
    if (st != DGP_OK)
        return st;
    return hip_status(launch_probe_lds_dma(src, perm, dst, (hipStream_t)stream), "probe launch");
}

dgp_status dgp_probe_lds_dma_narrow(int width, const void *src, const int32_t *perm, void *dst, void *stream)
{
    if (width != 1 && width != 2 && width != 4)
        return fail(DGP_ERR_CONFIG, "width must be 1, 2 or 4 (got %d)", width);
    if (!src || !perm || !dst)
        return fail(DGP_ERR_NULL, "NULL buffer");
    if (!aligned16(src) || !aligned16(dst))
        return fail(DGP_ERR_ALIGN, "buffers must be 16-byte aligned");
    dgp_status st = check_device_arch();
    if (st != DGP_OK)
        return st;
    return hip_status(launch_probe_lds_dma_narrow(width, src, perm, dst, (hipStream_t)stream), "probe launch");
}

dgp_status dgp_probe_copy(const void *src, void *dst, int64_t bytes, void *stream)
{
    if (bytes < 0 || bytes % 16 != 0)
        return fail(DGP_ERR_SHAPE, "bytes must be a non-negative multiple of 16");
    if (bytes == 0)
        return ok();
    if (!src || !dst)
        return fail(DGP_ERR_NULL, "NULL buffer");
    if (!aligned16(src) || !aligned16(dst))
        return fail(DGP_ERR_ALIGN, "buffers must be 16-byte aligned");
    dgp_status st = check_device_arch();
    if (st != DGP_OK)
        return st;
    return hip_status(launch_probe_copy(src, dst, bytes, (hipStream_t)stream), "probe launch");
}

dgp_status dgp_probe_stream_read(const void *src, int64_t bytes, int blocks, uint32_t *sink, void *stream)
{
    if (bytes < 0 || bytes % 16 != 0)
        return fail(DGP_ERR_SHAPE, "bytes must be a non-negative multiple of 16");
    if (blocks < 1 || blocks > 65536)
        return fail(DGP_ERR_SHAPE, "blocks must be in [1, 65536] (got %d)", blocks);
    if (bytes == 0)
        return ok();
    if (!src || !sink)
        return fail(DGP_ERR_NULL, "NULL buffer");
    if (!aligned16(src))
        return fail(DGP_ERR_ALIGN, "source must be 16-byte aligned");
    dgp_status st = check_device_arch();
    if (st != DGP_OK)
        return st;
    return hip_status(launch_probe_stream_read(src, bytes, blocks, sink, (hipStream_t)stream), "probe launch");
}

dgp_status dgp_probe_mfma_peak(int which, int rounds, int blocks, const void *operands, uint32_t *sink,
                               void *stream)
{
    if (which < 0 || which > 2)
        return fail(DGP_ERR_CONFIG, "which must be 0, 1 or 2");
    if (rounds < 1 || rounds > (1 << 24) || blocks < 1 || blocks > 65536)
        return fail(DGP_ERR_SHAPE, "rounds must be in [1, 2^24] and blocks in [1, 65536]");
    if (!operands || !sink)
        return fail(DGP_ERR_NULL, "NULL buffer");
    if (!aligned16(operands))
        return fail(DGP_ERR_ALIGN, "operands must be 16-byte aligned");
    dgp_status st = check_device_arch();
    if (st != DGP_OK)
        return st;
    return hip_status(launch_probe_mfma_peak(which, rounds, blocks, operands, sink, (hipStream_t)stream), "probe launch");
}

}  // extern "C"
