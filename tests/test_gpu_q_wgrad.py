"""GPU tests of a weight's gradient: exact inputs (small whole numbers, scales
with few bits) whose sums fit fp32, so that every result is known bit for bit;
real inputs against 64 bits; groups, row lists and what must stay untouched."""
import pytest
import torch

import dense_gemm_packer_amd as dgp
from gradient_common import GRAD_MODES, kept_values
from operand_common import EPS, pow2

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
OUTS = {"f32": torch.float32, "bf16": torch.bfloat16}


def whole(mode, rows, k, seed):
    """x as an operand, of whole numbers up to 8 times a scale, and its 64-bit values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-8, 9, (rows, k), generator=g).float()
    if mode == "none":
        return x.bfloat16().to(DEV), None, x.double()
    Q = x.to(torch.float8_e4m3fn)
    if mode == "tensor":
        S = torch.tensor([0.75])
    elif mode == "block128":      # 1, 1.5, .75 times a power of two: exact in bf16
        S = torch.tensor([1.0, 1.5, 0.75])[torch.randint(0, 3, (rows, k // 128), generator=g)]
        S = S * torch.exp2(torch.randint(-2, 2, S.shape, generator=g).float())
    else:
        S = torch.randint(124, 129, (rows, k // 128), generator=g).to(torch.uint8)
    return Q.to(DEV), S.to(DEV), kept_values(Q, S, mode)


def grads(m, n, seed):
    g = torch.Generator().manual_seed(seed)
    d = torch.randint(-4, 5, (m, n), generator=g).float()
    return d.bfloat16().to(DEV), d.double()


def equal(got, want):
    """`want` fits fp32; bf16 results are rounded once."""
    assert bool((want.float().double() == want).all())
    assert tuple(got.shape) == tuple(want.shape)
    return torch.equal(got.cpu(), want.float().to(got.dtype))


@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("out", list(OUTS))
@pytest.mark.parametrize("m,n,k", [(1, 16, 128), (2, 48, 256), (31, 128, 128), (33, 144, 384), (64, 256, 256), (100, 272, 640),
                                   (257, 1024, 128), (1000, 512, 512), (4097, 144, 256)])
def test_exact(mode, out, m, n, k):
    X, S, xv = whole(mode, m, k, m + k)
    dY, d = grads(m, n, n)
    assert equal(dgp.gemm_wgrad(dY, X, S, GRAD_MODES[mode], out_dtype=OUTS[out]), d.t() @ xv)


@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("out", list(OUTS))
@pytest.mark.parametrize("m,n,k", [(1, 4096, 3968), (97, 4112, 4096), (320, 3600, 4480), (4101, 2112, 2048), (9000, 1040, 1152)])
def test_exact_large_tiles(mode, out, m, n, k):
    """Enough 256 x 256 tiles for the whole GPU, or made enough by parts of the rows."""
    X, S, xv = whole(mode, m, k, m)
    dY, d = grads(m, n, 5)
    want = (d.float().to(DEV).t() @ xv.float().to(DEV)).cpu().double()     # (whole numbers of eighths: exact in any order)
    assert equal(dgp.gemm_wgrad(dY, X, S, GRAD_MODES[mode], out_dtype=OUTS[out]), want)


def test_bf16_k_of_64():
    X, S, xv = whole("none", 70, 192, 1)
    dY, d = grads(70, 80, 2)
    assert equal(dgp.gemm_wgrad(dY, X), d.t() @ xv)


def grouped_case(mode, counts, n, k, gather, tail, seed):
    g = torch.Generator().manual_seed(seed)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    m = int(off[-1]) + tail
    x_rows = max(1, m // 3) if gather else m
    X, S, xv = whole(mode, x_rows, k, seed)
    dY, d = grads(m, n, seed + 1)
    rows = torch.randint(0, x_rows, (m,), generator=g).to(torch.int32) if gather else None
    xr = xv[rows.long()] if gather else xv
    want = torch.stack([d[a:b].t() @ xr[a:b] for a, b in zip(off[:-1].tolist(), off[1:].tolist())])
    return dict(dC=dY, X=X, sX=S, scale_mode=GRAD_MODES[mode], offsets=off.to(DEV),
                rows=None if rows is None else rows.to(DEV)), want


@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", list(OUTS))
@pytest.mark.parametrize("counts,n,k", [([5], 16, 128), ([0, 3, 0, 40, 1, 0], 144, 256), ([33, 32, 31, 64, 65], 128, 384),
                                        ([200, 0, 7, 400], 272, 640)])
def test_groups(mode, gather, out, counts, n, k):
    kw, want = grouped_case(mode, counts, n, k, gather, 9, sum(counts))
    assert equal(dgp.gemm_wgrad(**kw, out_dtype=OUTS[out]), want)


@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("gather", [False, True])
def test_groups_large_tiles(mode, gather):
    kw, want = grouped_case(mode, [37, 0, 130, 1] * 8, 768, 640, gather, 3, 4)
    assert equal(dgp.gemm_wgrad(**kw), want)


@pytest.mark.parametrize("gather", [False, True])
def test_rows_that_count_for_nothing(gather):
    """Rows behind the last group, the other groups' rows and rows of X that no list names hold NaN."""
    kw, want = grouped_case("none", [7, 45, 3], 48, 256, gather, 70, 8)
    for g, (a, b) in enumerate(((0, 7), (7, 52), (52, 55))):
        dY, X = kw["dC"].clone(), kw["X"].clone()
        keep = torch.zeros(dY.shape[0], dtype=torch.bool, device=DEV)
        keep[a:b] = True
        dY[~keep] = float("nan")
        used = torch.zeros(X.shape[0], dtype=torch.bool, device=DEV)
        used[kw["rows"][a:b].long() if gather else torch.arange(a, b, device=DEV)] = True
        X[~used] = float("nan")
        assert equal(dgp.gemm_wgrad(**{**kw, "dC": dY, "X": X})[g], want[g])


def test_row_lists_out_of_range():
    """A row that X does not have counts as zeros."""
    kw, _ = grouped_case("mx128", [40, 20], 32, 128, True, 0, 3)
    rows = kw["rows"].clone()
    bad = torch.zeros_like(rows, dtype=torch.bool)
    bad[::7] = True
    rows[::14], rows[7::14] = -1, kw["X"].shape[0]
    rows[28] = 2 ** 31 - 1
    dY = kw["dC"].clone()
    dY[bad] = 0
    assert torch.equal(dgp.gemm_wgrad(**{**kw, "rows": rows}), dgp.gemm_wgrad(**{**kw, "dC": dY}))


def test_offsets_that_break_the_rule():
    """Wrong rows, but only rows of dC: what lies around it holds NaN."""
    big = torch.full((300, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    big[100:200] = 1
    X = torch.ones(100, 128, dtype=torch.bfloat16, device=DEV)
    for off in ([-50, 10, 400], [90, 20, 100], [2 ** 31 - 1, -2 ** 31, 7], [100, 100, 100]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        got = dgp.gemm_wgrad(big[100:200], X, offsets=o)
        assert bool(torch.isfinite(got).all()) and float(got.max()) <= 100
    first = dgp.gemm_wgrad(big[100:200], X, offsets=torch.tensor([-50, 10, 400], dtype=torch.int32, device=DEV))
    assert bool((first[0] == 10).all()) and bool((first[1] == 90).all())


@pytest.mark.parametrize("m", [0, 50])
def test_no_rows(m):
    dY, _ = grads(m, 32, 1)
    X, S, _ = whole("tensor", m, 128, 2)
    if m:
        S = torch.full((1,), float("nan"), device=DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    out = torch.full((3, 32, 128), 5.0, device=DEV)
    assert dgp.gemm_wgrad(dY, X, S, dgp.SCALE_TENSOR, offsets=off, out=out) is out and not bool(out.any())
    if m == 0:
        assert not bool(dgp.gemm_wgrad(dY, X, S, dgp.SCALE_TENSOR).any())
    out = torch.full((3, 32, 128), 5.0, device=DEV)
    dgp.gemm_wgrad(dY, X, S, dgp.SCALE_TENSOR, offsets=off, out=out, accumulate=True)
    assert bool((out == 5).all())


@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("m,n,k", [(50, 144, 256), (3000, 128, 256), (40, 4096, 4096)])
def test_accumulate(mode, m, n, k):
    X, S, xv = whole(mode, m, k, 3)
    dY, d = grads(m, n, 4)
    out = torch.randint(-100, 100, (n, k), generator=torch.Generator().manual_seed(5)).float().to(DEV)
    want = out.cpu().double() + (d.float().to(DEV).t() @ xv.float().to(DEV)).cpu().double()
    assert dgp.gemm_wgrad(dY, X, S, GRAD_MODES[mode], out=out, accumulate=True) is out
    assert equal(out, want)


def test_strided_gradient():
    """dC a part of wider rows; what lies beside it holds NaN."""
    wide = torch.full((130, 480), float("nan"), dtype=torch.bfloat16, device=DEV)
    dY, d = grads(130, 144, 6)
    wide[:, 64:208] = dY
    X, S, xv = whole("mx128", 130, 256, 7)
    assert equal(dgp.gemm_wgrad(wide[:, 64:208], X, S, dgp.SCALE_MX128), d.t() @ xv)


def test_scales_at_any_byte():
    X, S, xv = whole("mx128", 65, 384, 9)
    dY, d = grads(65, 64, 10)
    for shift in (1, 2, 3):
        buf = torch.zeros(S.numel() + 8, dtype=torch.uint8, device=DEV)
        s = buf[shift:shift + S.numel()].view(S.shape)
        s.copy_(S)
        assert equal(dgp.gemm_wgrad(dY, X, s, dgp.SCALE_MX128), d.t() @ xv)


@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("out", list(OUTS))
@pytest.mark.parametrize("m,n,k", [(700, 144, 384), (130, 4096, 4096)])
def test_real_values(mode, out, m, n, k):
    """fp32 sums: at most m roundings of each term; x to bf16 (2^-8) or to 2^-17 with block
    scales; the output's own half step."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(m, k, generator=g, device=DEV) * torch.exp(torch.randn(m, 1, generator=g, device=DEV))
    X, S = (x.bfloat16(), None) if mode == "none" else dgp.quantize(x, GRAD_MODES[mode])
    dY = (1e-3 * torch.randn(m, n, generator=g, device=DEV)).bfloat16()
    got = dgp.gemm_wgrad(dY, X, S, GRAD_MODES[mode], out_dtype=OUTS[out]).double()
    xv = kept_values(X, S, mode).to(DEV)
    want, size = dY.double().t() @ xv, dY.double().abs().t() @ xv.abs()
    lost = EPS * (m + 8)
    if mode == "block128":
        lost += 2.0 ** -8 if out == "bf16" else 2.0 ** -17 + EPS
    bound = size * lost
    if out == "bf16":
        bound = bound + (want.abs() + bound) * 2.0 ** -8
    assert bool(((got - want).abs() <= bound).all())


@pytest.mark.parametrize("e", [0, 1, 100, 254])
def test_scale_range(e):
    """E8M0 scales over the whole range: exact wherever x and the sum are normal numbers."""
    Q = torch.tensor([448.0, 1.0, 2.0 ** -6, 2.0 ** -9, -3.5, 0.0, 30.0, -0.0625] * 16).to(torch.float8_e4m3fn).view(1, 128)
    S = torch.full((1, 1), e, dtype=torch.uint8)
    d = torch.full((1, 16), 2.0 ** -20 if e > 200 else 2.0 ** 20, dtype=torch.bfloat16)
    got = dgp.gemm_wgrad(d.to(DEV), Q.to(DEV), S.to(DEV), dgp.SCALE_MX128).cpu().double()
    x = Q.double() * pow2(torch.tensor(e - 127))
    want = (d.double().t() @ x)
    normal = (x.abs() >= 2.0 ** -126) & (x.abs() < 2.0 ** 128)
    assert torch.equal(got[:, normal[0]], want[:, normal[0]])
    small = (x.abs() < 2.0 ** -126)[0]
    assert bool(((got - want)[:, small].abs() <= d.double()[0, 0] * 2.0 ** -126).all())


def test_nan_scale():
    X, S, xv = whole("mx128", 40, 256, 12)
    dY, d = grads(40, 32, 13)
    dY[17] = 1
    S[17, 1] = 255
    got = dgp.gemm_wgrad(dY, X, S, dgp.SCALE_MX128)
    assert bool(torch.isnan(got[:, 128:]).all()) and bool(torch.isfinite(got[:, :128]).all())
