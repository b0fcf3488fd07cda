"""64-bit references of the operand-writing operators, and the comparison of
codes and scales with them.

A code is right when it is within half a grid step of the value it rounds,
widened by the relative error `delta` that the fp32 arithmetic before the
rounding may have made (each test derives its delta); where delta is 0 the
code must be the nearest grid value, ties to even."""
import torch

import dense_gemm_packer_amd as dgp

GRID = {"e4m3": (3, -6, 448.0), "e2m1": (1, 0, 6.0)}
EPS = 2.0 ** -24            # half a step of fp32, relative
MODES = {"none": dgp.SCALE_NONE, "tensor": dgp.SCALE_TENSOR, "block128": dgp.SCALE_BLOCK128,
         "mx128": dgp.SCALE_MX128, "mx32": dgp.SCALE_MX32}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"block128": 128, "mx128": 128, "mx32": 32}


def pow2(e):
    return torch.ldexp(torch.ones((), dtype=torch.float64), e)


def grid_step(v, grid):
    mant, low, _ = GRID[grid]
    e = torch.clamp(torch.frexp(v)[1] - 1, min=low)
    return pow2(e - mant)


def to_grid(v, grid):
    """Nearest grid value, ties to even, saturating."""
    step, top = grid_step(v, grid), GRID[grid][2]
    return torch.clamp(torch.round(v / step) * step, -top, top)


def unpack_e2m1(codes):
    """Packed E2M1 (uint8 view) -> values, element 2j from the low nibble."""
    c = codes.cpu().view(torch.uint8)
    n = torch.stack((c & 15, c >> 4), dim=-1).flatten(-2).long()
    half = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    return torch.cat((half, -half))[n]


def code_values(Q, mode):
    return unpack_e2m1(Q) if mode == "mx32" else Q.cpu().double()


def e8m0_of(amax, mode):
    """E8M0 byte of a block with largest magnitude amax (64 bits, finite)."""
    e = torch.frexp(amax)[1] - 1
    if mode == "mx32":
        e = e - 2
    else:
        e = e - 8 + (amax > 448.0 * pow2(e - 8)).to(e.dtype)
    return torch.where(amax > 0, torch.clamp(e + 127, min=0), 0).to(torch.int64)


def block_amax(y, mode):
    b = BLOCK[mode]
    return y.abs().unflatten(-1, (y.shape[-1] // b, b)).amax(-1)


def check_operand(Q, S, y, mode, delta=0.0, scale=None):
    """Q, S (as the library wrote them) against the 64-bit values y [M][K]
    whose fp32 versions are within a relative delta (a number or a tensor)."""
    y = y.double()
    if mode == "none":
        got = Q.cpu().double()
        assert Q.dtype == torch.bfloat16 and got.shape == y.shape
        bound = y.abs() * (2.0 ** -8 + delta) + 2.0 ** -133   # half a step of bf16, of its subnormals at the end
        assert bool(((got - y).abs() <= bound).all())
        return
    grid = "e2m1" if mode == "mx32" else "e4m3"
    got = code_values(Q, mode)
    assert got.shape == y.shape
    dmax = delta if isinstance(delta, float) else float(torch.as_tensor(delta).max())
    if mode == "tensor":
        if scale is None:
            s = torch.clamp(y.abs().max() / 448, min=2.0 ** -126)
            assert abs(float(S.cpu().double()) - s) <= s * (dmax + EPS)
            scale = S
        full = scale.cpu().double()
        extra = 2 * EPS                                        # 1/s and the product
    elif mode == "block128":
        s = torch.clamp(block_amax(y, mode) / 448, min=2.0 ** -126)
        assert tuple(S.shape) == tuple(s.shape) and S.dtype == torch.float32
        assert bool(((S.cpu().double() - s).abs() <= s * (dmax + EPS)).all())
        full = S.cpu().double().repeat_interleave(128, -1)
        extra = 2 * EPS
    else:
        amax = block_amax(y, mode)
        e = S.cpu().to(torch.int64)
        assert tuple(S.shape) == tuple(amax.shape) and S.dtype == torch.uint8
        lo, hi = e8m0_of(amax * (1 - dmax), mode), e8m0_of(amax * (1 + dmax), mode)
        assert bool(((e >= lo) & (e <= hi)).all())
        full = pow2(e - 127).repeat_interleave(BLOCK[mode], -1)
        extra = 0.0                                            # a power of two: exact
    v = y / full
    top = GRID[grid][2]
    tol = torch.as_tensor(delta, dtype=torch.float64) + extra
    if float(tol.max()) == 0.0:
        assert bool((got == to_grid(v, grid)).all())
        return
    clipped = torch.clamp(v, -top, top)
    bound = grid_step(clipped, grid) / 2 + tol * clipped.abs()
    # (a value a hair above a power of two may have rounded on the finer grid below it, and the reverse)
    assert bool(((got - clipped).abs() <= bound * (1 + 1e-9)).all())


def dequantize(Q, S, mode):
    """64-bit values of an operand."""
    v = code_values(Q, mode)
    if mode == "none":
        return v
    if mode == "tensor":
        return v * S.cpu().double()
    if mode == "block128":
        return v * S.cpu().double().repeat_interleave(128, -1)
    return v * pow2(S.cpu().to(torch.int64) - 127).repeat_interleave(BLOCK[mode], -1)
