"""64-bit references of the layer norm and of the gradients, the error that the
kernels' fp32 arithmetic may have made by then, and inputs.

Every error is a sum of half steps of fp32 (EPS, relative) over the operations
on the way, with a sum of n values counted as `chain(n)` roundings of each of
its terms."""
import torch

import dense_gemm_packer_amd as dgp
from operand_common import BLOCK, EPS, GRID, block_amax, code_values, e8m0_of, grid_step, pow2

GRAD_MODES = {"none": dgp.SCALE_NONE, "tensor": dgp.SCALE_TENSOR, "block128": dgp.SCALE_BLOCK128, "mx128": dgp.SCALE_MX128}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def chain(k):
    """Roundings of a term in a sum over a row of k: a thread's own pieces (at
    most 16 terms, in rows beyond 8192 k / 1024), the lanes and the waves (at most 22)."""
    return max(16, k / 1024) + 24


def rows_chain(m):
    """Roundings of a term in a sum over m rows: a workgroup's own rows (of
    256), the rows side by side (at most 16), every 32nd part (8), the 32 sums of these."""
    return m / 64 + 64


def kept(x, mode, dev):
    """x [M][K] as the forward pass keeps it, on the device, and the 64-bit values that it stands for."""
    x = x.to(dev)
    if mode == "none":
        return x, None, x.cpu().double()
    Q, S = dgp.quantize(x, GRAD_MODES[mode])
    return Q, S, kept_values(Q, S, mode)


def kept_values(Q, S, mode):
    v = Q.cpu().double()
    if mode == "none":
        return v
    if mode == "tensor":
        return v * S.cpu().double()
    s = S.cpu().double() if mode == "block128" else pow2(S.cpu().to(torch.int64) - 127)
    return v * s.repeat_interleave(128, -1)


def activations(m, k, dtype, seed, mean=0.0, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g, dtype=torch.float64)
    x *= torch.exp2(spread * torch.randn(m, 1, generator=g, dtype=torch.float64))
    x[:, ::37] *= 12
    return (x + mean).to(dtype)


# ------------------------------------------------------------ the layer norm

def mean64(v):
    return v.mean(-1, keepdim=True)


def norm_statistics(x, eps, layer):
    """(xhat, rstd, error of xhat) of 64-bit rows whose fp32 versions are within half a step."""
    k = x.shape[-1]
    d = x - mean64(x) if layer else x
    rstd = 1 / torch.sqrt(mean64(d * d) + eps)
    xh = d * rstd
    # a row's values to half a step of |x|; the mean, subtracted twice; rstd, half of the error of
    # a sum of squares (two roundings a term, and the row's own error) and five operations
    err = EPS * (x.abs() * rstd + 4 * xh.abs() + (chain(k) * mean64(xh.abs()) if layer else 0))
    lost = EPS * (chain(k) + 8) + mean64(xh.abs() * err)
    return xh, rstd, err + xh.abs() * lost


def layernorm_reference(x, r, w, b, eps):
    """(h, y, error of y)."""
    h = x.double() if r is None else x.double() + r.double()
    xh, _, err = norm_statistics(h, eps, True)
    y = xh * w.double()
    err = err * w.double().abs() + 2 * EPS * y.abs()
    if b is not None:
        y = y + b.double()
        err = err + EPS * y.abs()
    return h, y, err


def check_near(got, want, err, dtype):
    """Within the error before the rounding and half a step of the type."""
    assert got.dtype == dtype and tuple(got.shape) == tuple(want.shape)
    g = got.cpu().double()
    bound = (want.abs() + err) * HALF[dtype] + err + TINY[dtype]
    bad = ~((g - want).abs() <= bound)
    assert not bool(bad.any()), (int(bad.sum()), float(((g - want).abs() / bound).max()))


def check_operand_near(Q, S, y, err, mode, scale=None):
    """Codes and scales of values that are within `err` of y before the rounding."""
    if mode == "none":
        check_near(Q, y, err, torch.bfloat16)
        return
    grid = "e2m1" if mode == "mx32" else "e4m3"
    got, top = code_values(Q, mode), GRID[grid][2]
    assert got.shape == y.shape
    if mode == "tensor":
        full = scale.cpu().double()
    elif mode == "block128":
        amax, most = block_amax(y, mode), block_amax(err, mode)
        s = torch.clamp(amax / 448, min=2.0 ** -126)
        assert tuple(S.shape) == tuple(s.shape) and S.dtype == torch.float32
        assert bool(((S.cpu().double() - s).abs() <= most / 448 + s * 2 * EPS).all())
        full = S.cpu().double().repeat_interleave(128, -1)
    else:
        amax, most = block_amax(y, mode), block_amax(err, mode)
        e = S.cpu().to(torch.int64)
        assert tuple(S.shape) == tuple(amax.shape) and S.dtype == torch.uint8
        assert bool(((e >= e8m0_of(torch.clamp(amax - most, min=0), mode)) & (e <= e8m0_of(amax + most, mode))).all())
        full = pow2(e - 127).repeat_interleave(BLOCK[mode], -1)
    v, lost = torch.clamp(y / full, -top, top), err / full + 2 * EPS * (y / full).abs()
    # (a value past a power of two by its error rounds on the coarser grid there)
    bound = grid_step(torch.clamp(v.abs() + lost, max=top), grid) / 2 + lost
    assert bool(((got - v).abs() <= bound * (1 + 1e-9)).all())


# -------------------------------------------------------------- gradients

def norm_backward_reference(dy, x, w, r, eps, layer):
    """dict of (value, error before the rounding) for dx, dw and (layer) db."""
    m, k = x.shape
    dy, w = dy.double(), w.double()
    xh, rstd, ex = norm_statistics(x, eps, layer)
    g = dy * w
    c = mean64(g * xh)
    mg = mean64(g) if layer else 0.0
    dx = rstd * (g - mg - xh * c)
    n = chain(k) + 4
    # c: each term's product, the sum, xhat's error and (through the mean taken from g) g's own mean
    ec = EPS * n * mean64(g.abs() * xh.abs()) + mean64(g.abs() * ex)
    if layer:
        ec = ec + EPS * n * mean64(g.abs()) * mean64(xh.abs())
    eg = EPS * 2 * g.abs() + (EPS * n * mean64(g.abs()) if layer else 0.0)
    err = rstd * (eg + xh.abs() * ec + ex * c.abs() + EPS * 4 * (g.abs() + (mg.abs() if layer else 0) + (xh * c).abs()))
    # rstd's own error (half of a sum of squares' and the row's, five operations)
    err = err + dx.abs() * (EPS * (chain(k) + 8) + mean64(xh.abs() * ex))
    if r is not None:
        dx = dx + r.double()
        err = err + EPS * dx.abs()
    out = {"dx": (dx, err)}
    terms = dy.abs() * (ex + 2 * EPS * xh.abs())
    out["dw"] = ((dy * xh).sum(0), terms.sum(0) + EPS * rows_chain(m) * (dy * xh).abs().sum(0))
    if layer:
        out["db"] = (dy.sum(0), EPS * rows_chain(m) * dy.abs().sum(0))
    return out


def swiglu_backward_reference(dy, gate, up):
    """([dg | du], error): exp(-g) is exp2 of one fp32 product, 2 |g| half steps and 4 more of its
    own; 1 / (1 + e) and the products a half or a whole step each (the reciprocal: 2)."""
    dy, s = dy.double(), torch.sigmoid(gate)
    t = torch.sigmoid(-gate)
    n = 2 * gate.abs() + 16
    dg, du = dy * up * s * (1 + gate * t), dy * gate * s
    err = torch.cat([EPS * n * (dy * up * s).abs() * (1 + (gate * t).abs()), EPS * n * du.abs()], -1)
    return torch.cat([dg, du], -1), err
