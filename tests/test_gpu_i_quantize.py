"""GPU tests of the operators that write a product's operand: quantisation of
activations and weights, the norm and the gated activation, against 64-bit
references (operand_common.py)."""
import pytest
import torch

import dense_gemm_packer_amd as dgp
from operand_common import (BLOCK, EPS, MODES, TYPES, check_operand, code_values, dequantize, pow2, to_grid)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rows(m, k, dtype, seed, spread=4.0):
    """Rows with sizes over several binades, zeros and a block of zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g, dtype=torch.float64)
    x *= torch.exp2(spread * torch.randn(m, k // 32, generator=g, dtype=torch.float64)).repeat_interleave(32, 1)
    x[:, ::17] = 0
    x[m // 2, :32] = 0
    x[m // 3, :128] = 0
    return torch.clamp(x, -3e4, 3e4).to(dtype)


# ------------------------------------------------------------ quantize

@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", ["tensor", "block128", "mx128", "mx32"])
@pytest.mark.parametrize("m,k", [(1, 256), (3, 512), (37, 1280), (130, 7168)])
def test_quantize(x_type, mode, m, k):
    x = rows(m, k, TYPES[x_type], m + k)
    Q, S = dgp.quantize(x.to(DEV), MODES[mode])
    check_operand(Q, S, x, mode)


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("m,k", [(511, 128), (512, 128), (513, 128), (8, 8192), (9, 8192)])
def test_quantize_tensor_around_the_one_launch_limit(x_type, m, k):
    wide = rows(m, k + 256, TYPES[x_type], m)
    for x in (wide[:, :k], wide[:, :k].contiguous()):
        check_operand(*dgp.quantize(x.to(DEV) if x.is_contiguous() else wide.to(DEV)[:, :k], dgp.SCALE_TENSOR), x, "tensor")


@pytest.mark.parametrize("mode", ["tensor", "block128", "mx128"])
def test_quantize_odd_block_count(mode):
    x = rows(7, 128 * 9, torch.bfloat16, 3)
    check_operand(*dgp.quantize(x.to(DEV), MODES[mode]), x, mode)


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", ["tensor", "block128", "mx128", "mx32"])
def test_quantize_strided_rows(x_type, mode):
    wide = rows(19, 1024, TYPES[x_type], 5).to(DEV)
    x = wide[:, 256:768]
    Q, S = dgp.quantize(x, MODES[mode])
    Qd, Sd = dgp.quantize(x.contiguous(), MODES[mode])
    assert torch.equal(Q.view(torch.uint8), Qd.view(torch.uint8)) and torch.equal(S, Sd)
    check_operand(Q, S, x.cpu(), mode)


def test_quantize_given_scale_saturates():
    x = torch.tensor([0.0, 1.0, -2.0, 447.9, 448.0, 460.0, 1e30, -1e30, float("inf"), -float("inf"), 2.0 ** -9,
                      2.0 ** -10, 3 * 2.0 ** -11], dtype=torch.float32)
    x = torch.cat([x, torch.zeros(128 - x.numel())]).view(1, 128)
    s = torch.ones(1, device=DEV)
    Q, S = dgp.quantize(x.to(DEV), dgp.SCALE_TENSOR, scale=s)
    assert S is s
    want = to_grid(torch.clamp(x.double(), -1e38, 1e38), "e4m3")
    assert torch.equal(code_values(Q, "tensor"), want)
    x[0, 5] = float("nan")
    got = code_values(dgp.quantize(x.to(DEV), dgp.SCALE_TENSOR, scale=s)[0], "tensor")
    assert torch.isnan(got[0, 5]) and int(torch.isnan(got).sum()) == 1


@pytest.mark.parametrize("grid,mode", [("e4m3", "mx128"), ("e2m1", "mx32")])
def test_every_bf16_rounds_to_nearest_even(grid, mode):
    """All finite bf16 values, each in a block whose largest value fixes the
    scale at 1: nearest grid value, ties to even, saturation beyond the top."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    top = 256.0 if grid == "e4m3" else 4.0          # scale 1 exactly (2^8 / 2^8, 2^2 / 2^2)
    vals = bits[torch.isfinite(bits) & (bits.abs().float() <= (448.0 if grid == "e4m3" else 7.9))]
    b = BLOCK[mode]
    per = b - 1
    n = -(-vals.numel() // per)
    x = torch.zeros(n, b, dtype=torch.bfloat16)
    x[:, 0] = top
    pad = torch.zeros(n * per, dtype=torch.bfloat16)
    pad[: vals.numel()] = vals
    x[:, 1:] = pad.view(n, per)
    if mode == "mx32":
        extra = (-n) % 8
        x = torch.cat([x, x[:extra]]).view(-1, 256)
    Q, S = dgp.quantize(x.to(DEV), MODES[mode])
    assert bool((S.cpu() == 127).all())
    assert torch.equal(code_values(Q, mode), to_grid(x.double(), grid))


@pytest.mark.parametrize("mode", ["mx128", "mx32"])
def test_e8m0_borders(mode):
    """Largest values on both sides of every border of the scale's exponent."""
    b = BLOCK[mode]
    borders = [448.0, 448.0 * 0.5, 512.0, 256.0, 6.0, 4.0, 7.999, 8.0, 1.0, 2.0 ** -100, 2.0 ** -117, 2.0 ** -118,
               2.0 ** -119, 2.0 ** -125, 2.0 ** -126, 2.0 ** -140, 2.0 ** -149, 3.0e38, 0.0]
    vals = []
    for v in borders:
        f = torch.tensor(v, dtype=torch.float32)
        vals += [f, torch.nextafter(f, torch.tensor(float("inf"))), torch.nextafter(f, torch.tensor(0.0))]
    x = torch.zeros(len(vals), 256, dtype=torch.float32)
    for i, v in enumerate(vals):
        x[i, :] = v * 0.37
        x[i, ::b] = -v if i % 2 else v
    Q, S = dgp.quantize(x.to(DEV), MODES[mode])
    check_operand(Q, S, x, mode)


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", ["block128", "mx128", "mx32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_block_gets_a_nan_scale(x_type, mode, bad):
    x = rows(4, 512, TYPES[x_type], 8)
    x[2, 200] = bad
    Q, S = dgp.quantize(x.to(DEV), MODES[mode])
    b = BLOCK[mode]
    s = S.cpu()
    isnan = torch.isnan(s) if mode == "block128" else s == 255
    want = torch.zeros_like(isnan)
    want[2, 200 // b] = True
    assert torch.equal(isnan, want)
    codes = code_values(Q, mode)
    blk = codes[2, 200 // b * b: (200 // b + 1) * b]
    assert bool((blk == 0).all()) if mode == "mx32" else bool(torch.isnan(blk).all())
    keep = [0, 1, 3]
    check_operand(Q.view(torch.uint8).cpu()[keep].view(Q.dtype), s[keep], x[keep], mode)


@pytest.mark.parametrize("m", [40, 300])     # one launch, and two
@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
def test_nonfinite_tensor_gets_a_nan_scale(bad, m):
    x = rows(m, 512, torch.bfloat16, 9)
    x[m - 3, 400] = bad
    Q, S = dgp.quantize(x.to(DEV), dgp.SCALE_TENSOR)
    assert bool(torch.isnan(S).all()) and bool(torch.isnan(Q.cpu().double()).all())


@pytest.mark.parametrize("mode", ["tensor", "block128", "mx128", "mx32"])
def test_all_zero_and_tiny(mode):
    for x in (torch.zeros(2, 256), torch.full((2, 256), 2.0 ** -149), torch.full((2, 256), -1e-40)):
        Q, S = dgp.quantize(x.to(DEV), MODES[mode])
        check_operand(Q, S, x, mode)


def test_empty_is_a_no_op():
    for mode in ("block128", "mx32"):
        Q, S = dgp.quantize(torch.empty(0, 256, device=DEV), MODES[mode])
        assert Q.shape[0] == 0 and S.shape[0] == 0


# ---------------------------------------------------------- quantize_b

@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", ["tensor", "block128", "mx128", "mx32"])
@pytest.mark.parametrize("shape", [(128, 256), (384, 1280), (3, 128, 512), (5, 256, 256)])
def test_quantize_b(x_type, mode, shape):
    w = rows(shape[-2] * (shape[0] if len(shape) == 3 else 1), shape[-1], TYPES[x_type], 11).view(shape)
    Bs, sB = dgp.quantize_b(w.to(DEV), MODES[mode])
    E, N, K = ([1] + list(shape))[-3:] if len(shape) == 2 else shape
    flat = Bs.view(E * N, -1)
    codes = dgp.unshuffle_b(flat).view(E, N, -1)
    for e in range(E):
        y = w.view(E, N, K)[e]
        if mode == "block128":
            s = torch.clamp(y.double().abs().view(N // 128, 128, K // 128, 128).amax((1, 3)) / 448, min=2.0 ** -126)
            got = sB.view(E, N // 128, K // 128)[e].cpu().double()
            assert bool(((got - s).abs() <= s * EPS).all())
            full = got.repeat_interleave(128, 0).repeat_interleave(128, 1)
            v = y.double() / full
            from operand_common import grid_step
            bound = grid_step(v, "e4m3") / 2 + 2 * EPS * v.abs()
            assert bool(((codes[e].cpu().double() - v).abs() <= bound).all())
        else:
            check_operand(codes[e], sB.view(E, -1)[e] if mode == "tensor" else sB.view(E, N, -1)[e], y, mode)


def test_quantize_b_narrow_weight():
    """Sixteen rows: fewer operand blocks than one workgroup makes."""
    w = rows(16, 128, torch.float32, 12)
    Bs, sB = dgp.quantize_b(w.to(DEV), dgp.SCALE_MX128)
    check_operand(dgp.unshuffle_b(Bs), sB, w, "mx128")


# ------------------------------------------------------------- the norm

def norm_reference(x, r, w, eps):
    h = x.double() if r is None else x.double() + r.double()
    return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()


# fp32 error of the norm, relative: the sum of squares adds at most 8 C terms
# per thread in sequence (C <= 4 pieces in registers; more where the row is
# read twice), then 4 + 2 + waves steps, every term positive, so its error is
# at most (terms in sequence + steps) half steps; half of that reaches the
# root, plus the quotient, the root, its reciprocal and two products, and h's
# own rounding, which counts twice (in the sum and in the product).
def norm_delta(k):
    return ((8 * max(4, k // 8192) + 6 + 16 + 4) / 2 + 6) * EPS


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("m,k,res,w32", [(1, 7168, True, False), (5, 256, True, True), (9, 512, False, False),
                                         (6, 2048, True, False), (700, 2304, False, True), (3, 16384, True, True),
                                         (2, 40960, True, False)])
def test_rmsnorm(x_type, mode, m, k, res, w32):
    dt = TYPES[x_type]
    x = rows(m, k, dt, 21, spread=1.0)
    r = rows(m, k, dt, 22, spread=1.0) if res else None
    g = torch.Generator().manual_seed(23)
    w = (1 + 0.2 * torch.randn(k, generator=g)).to(torch.float32 if w32 else dt)
    scale = torch.full((1,), 0.05, device=DEV) if mode == "tensor" else None
    got = dgp.rmsnorm_quantize(x.to(DEV), w.to(DEV), MODES[mode], residual=None if r is None else r.to(DEV),
                               eps=1e-5, scale=scale)
    h, y = norm_reference(x, r, w, 1e-5)
    check_operand(got[0], got[1], y, mode, norm_delta(k), scale)
    if res:
        half = torch.finfo(dt).eps / 2
        assert bool(((got[2].cpu().double() - h).abs() <= h.abs() * (half + EPS) + 2.0 ** -133).all() if dt != torch.float16
                    else ((got[2].cpu().double() - h).abs() <= h.abs() * (half + EPS) + 2.0 ** -25).all())
    else:
        assert len(got) == 2


@pytest.mark.parametrize("mode", ["none", "mx128"])
@pytest.mark.parametrize("m,k", [(3, 512), (5, 640), (8193, 1024), (9, 2048), (7, 4096), (1030, 3968), (384, 4224),
                                 (385, 8192), (2, 8320)])
def test_rmsnorm_row_splits(mode, m, k):
    """Every split of a row over threads and pieces, full and with threads left over."""
    x, r = (rows(m, k, torch.bfloat16, s, spread=1.0) for s in (27, 28))
    w = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(29))).bfloat16()
    Q, S, H = dgp.rmsnorm_quantize(x.to(DEV), w.to(DEV), MODES[mode], residual=r.to(DEV), eps=1e-5)
    h, y = norm_reference(x, r, w, 1e-5)
    check_operand(Q, S, y, mode, norm_delta(k))
    assert bool(((H.cpu().double() - h).abs() <= h.abs() * (2.0 ** -8 + EPS) + 2.0 ** -133).all())


@pytest.mark.parametrize("k", [256, 1024, 7168, 40960])
def test_rmsnorm_in_place_and_strided(k):
    m = 4
    x = rows(m, 2 * k, torch.bfloat16, 31, spread=1.0).to(DEV)[:, k:]
    r = rows(m, k, torch.bfloat16, 32, spread=1.0).to(DEV)
    w = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    Q, S, H = dgp.rmsnorm_quantize(x, w, dgp.SCALE_MX128, residual=r)
    r2 = r.clone()
    Q2, S2, H2 = dgp.rmsnorm_quantize(x.contiguous(), w, dgp.SCALE_MX128, residual=r2, residual_out=r2)
    assert H2 is r2
    assert torch.equal(H, H2) and torch.equal(S, S2) and torch.equal(Q.view(torch.uint8), Q2.view(torch.uint8))


def test_rmsnorm_zero_row_and_eps():
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    x[1] = 1e-20
    w = torch.ones(256, dtype=torch.bfloat16)
    Q, _ = dgp.rmsnorm_quantize(x.to(DEV), w.to(DEV), dgp.SCALE_NONE, eps=1e-6)
    check_operand(Q, None, norm_reference(x, None, w, 1e-6)[1], "none", norm_delta(256))
    Q, S = dgp.rmsnorm_quantize(torch.zeros(1, 256, device=DEV), torch.ones(256, device=DEV), dgp.SCALE_MX32, eps=0.0)
    assert bool((S == 255).all())     # 0 / 0


# ---------------------------------------------------- the gated activation

@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("m,k", [(1, 256), (13, 768), (65, 2048)])
def test_swiglu(x_type, mode, m, k):
    dt = TYPES[x_type]
    x = torch.clamp(rows(m, 2 * k, dt, 41, spread=1.5), min=-80.0)
    g, u = x[:, :k].double(), x[:, k:].double()
    xd = x.to(DEV)
    scale = torch.full((1,), 0.3, device=DEV) if mode == "tensor" else None
    Q, S = dgp.swiglu_quantize(xd[:, :k], xd[:, k:], MODES[mode], scale=scale)
    y = g * torch.sigmoid(g) * u
    # exp: the product with log2 e rounds the exponent |g| log2 e by half a
    # step, which is ln 2 times as much of the result; 1 ulp for exp2, the sum,
    # 1 ulp for the reciprocal, two products.
    delta = g.abs() * EPS * 2 + 8 * EPS
    check_operand(Q, S, y, mode, delta, scale)


def test_swiglu_far_gates():
    g = torch.tensor([-1e4, -200.0, -100.0, -89.0, 89.0, 200.0, 3e4, 0.0] * 32, dtype=torch.float32).view(1, 256)
    u = torch.full((1, 256), 2.0)
    Q, _ = dgp.swiglu_quantize(g.to(DEV), u.to(DEV), dgp.SCALE_NONE)
    want = g.double() * torch.sigmoid(g.double()) * 2
    got = Q.cpu().double()
    assert bool(torch.isfinite(got).all())
    assert bool(((got - want).abs() <= want.abs() * (2.0 ** -8 + 2e-5) + 1e-36).all())


# ----------------------------------------------------- together, streams

@pytest.mark.parametrize("mode", ["tensor", "block128", "mx128", "mx32"])
@pytest.mark.parametrize("m", [1, 16, 200])
def test_quantised_product(mode, m):
    """quantize and quantize_b feed gemm_preshuffle as they are."""
    n, k = 256, 1024
    a = rows(m, k, torch.bfloat16, 51, spread=1.0)
    b = rows(n, k, torch.float32, 52, spread=1.0)
    A, sA = dgp.quantize(a.to(DEV), MODES[mode])
    Bs, sB = dgp.quantize_b(b.to(DEV), MODES[mode])
    C = dgp.gemm_preshuffle(A, Bs, sA, sB, MODES[mode]).cpu().double()
    Bv = dgp.unshuffle_b(Bs)
    if mode == "block128":
        bd = Bv.cpu().double() * sB.cpu().double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    else:
        bd = dequantize(Bv, sB, mode)
    ad = dequantize(A, sA, mode)
    want = ad @ bd.t()
    bound = 2.0 ** -8 * want.abs() + (k + 8) * EPS * (ad.abs() @ bd.abs().t())
    assert bool(((C - want).abs() <= bound).all())


def test_on_a_side_stream_and_captured():
    x = rows(64, 1024, torch.bfloat16, 61).to(DEV)
    r = rows(64, 1024, torch.bfloat16, 62).to(DEV)
    w = torch.ones(1024, dtype=torch.bfloat16, device=DEV)
    want_q = dgp.quantize(x, dgp.SCALE_TENSOR)
    want_n = dgp.rmsnorm_quantize(x, w, dgp.SCALE_BLOCK128, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got_q = dgp.quantize(x, dgp.SCALE_TENSOR, stream=side)
    side.synchronize()
    assert torch.equal(got_q[0].view(torch.uint8), want_q[0].view(torch.uint8)) and torch.equal(got_q[1], want_q[1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cap_q = dgp.quantize(x, dgp.SCALE_TENSOR)
        cap_n = dgp.rmsnorm_quantize(x, w, dgp.SCALE_BLOCK128, residual=r)
    for seed in (63, 64, 65):
        x.copy_(rows(64, 1024, torch.bfloat16, seed))
        want_q = dgp.quantize(x, dgp.SCALE_TENSOR)
        want_n = dgp.rmsnorm_quantize(x, w, dgp.SCALE_BLOCK128, residual=r)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(cap_q + cap_n, want_q + want_n):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


def test_rows_behind_the_output_are_left(request):
    """Outputs given as the first rows of larger buffers: nothing past them is written."""
    x = rows(5, 256, torch.bfloat16, 71).to(DEV)
    Q = torch.full((9, 256), 7, dtype=torch.uint8, device=DEV)
    S = torch.full((9, 2), 9, dtype=torch.uint8, device=DEV)
    dgp.quantize(x, dgp.SCALE_MX128, out=Q[:5].view(torch.float8_e4m3fn), scales=S[:5])
    assert bool((Q[5:] == 7).all()) and bool((S[5:] == 9).all())
    check_operand(Q[:5].view(torch.float8_e4m3fn), S[:5], x.cpu(), "mx128")
