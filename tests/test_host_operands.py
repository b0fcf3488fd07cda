"""Host-side refusals of the operators that write a product's operand and of
the grouped product: every bad argument is turned down with its documented
status before any HIP call (only invalid calls are made, so no device is
touched), and the binding's own checks raise before a launch."""
import ctypes
import os

import pytest
import torch

OK, NULL, SHAPE, ALIGN, DTYPE, SCALE, SPLITK, WS, CONFIG, ARCH, HIP = range(11)
BF16, FP8, FP4, F16, F32 = range(5)
NONE, TENSOR, BLOCK, MX, MX32 = range(5)
P = 0x10000          # aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def dgp():
    import dense_gemm_packer_amd as d
    if not os.path.exists(d.LIB_PATH):
        from dense_gemm_packer_amd import build
        build.build()
    return d


@pytest.fixture(scope="module")
def L(dgp):
    return dgp.lib()


def quantize(L, X=P, ldx=256, xt=BF16, Q=P, S=P, scale=None, M=4, K=256, mode=BLOCK, ws=None, wsb=0):
    return L.dgp_quantize(X, ldx, xt, Q, S, scale, M, K, mode, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=FP8), DTYPE), (dict(xt=FP4), DTYPE), (dict(xt=7), DTYPE),
    (dict(mode=NONE), SCALE), (dict(mode=5), SCALE), (dict(mode=-1), SCALE),
    (dict(M=-1), SHAPE), (dict(K=-128), SHAPE), (dict(K=64, ldx=64), SHAPE), (dict(K=129, ldx=256), SHAPE),
    (dict(mode=MX32, K=128), SHAPE), (dict(ldx=128), SHAPE), (dict(M=1 << 31), SHAPE),
    (dict(K=1 << 24, ldx=1 << 24), SHAPE),
    (dict(X=None), NULL), (dict(Q=None), NULL), (dict(S=None), NULL), (dict(S=None, mode=MX), NULL),
    (dict(X=P + 8), ALIGN), (dict(Q=P + 4), ALIGN), (dict(ldx=257), ALIGN), (dict(ldx=260, xt=BF16), ALIGN),
    (dict(S=P + 2), ALIGN), (dict(scale=P), SCALE), (dict(scale=P + 2, mode=TENSOR), ALIGN),
    (dict(mode=TENSOR), WS), (dict(mode=TENSOR, ws=P, wsb=1023), WS), (dict(mode=TENSOR, ws=P + 2, wsb=4096), ALIGN),
])
def test_quantize_refusals(L, kw, status):
    assert quantize(L, **kw) == status
    assert L.dgp_last_error()


def test_no_op_sizes(L):
    assert quantize(L, M=0) == OK and quantize(L, K=0, ldx=0) == OK
    assert L.dgp_quantize_b(None, BF16, None, None, 0, 128, 128, BLOCK, None, 0, None) == OK
    assert L.dgp_rmsnorm_quantize(None, 0, None, 0, BF16, None, BF16, 1e-6, None, None, None, None, 0, 128, BLOCK, None) == OK
    assert L.dgp_swiglu_quantize(None, 0, None, 0, BF16, None, None, None, 0, 128, BLOCK, None) == OK


def test_workspace_bytes(L, dgp):
    assert L.dgp_quantize_workspace_bytes(1, TENSOR) == 1024
    assert L.dgp_quantize_workspace_bytes(3, TENSOR) == 3072
    for mode in (BLOCK, MX, MX32):
        assert L.dgp_quantize_workspace_bytes(3, mode) == 0


def quantize_b(L, B=P, xt=BF16, Bs=P, sB=P, E=1, N=128, K=256, mode=BLOCK, ws=None, wsb=0):
    return L.dgp_quantize_b(B, xt, Bs, sB, E, N, K, mode, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=FP8), DTYPE), (dict(mode=NONE), SCALE), (dict(E=-1), SHAPE), (dict(E=65536), SHAPE), (dict(N=-16), SHAPE),
    (dict(N=24, mode=MX), SHAPE), (dict(N=64), SHAPE), (dict(K=192), SHAPE), (dict(K=128, mode=MX32), SHAPE),
    (dict(E=60000, N=1 << 16, mode=MX), SHAPE), (dict(B=None), NULL), (dict(Bs=None), NULL), (dict(sB=None), NULL),
    (dict(B=P + 2), ALIGN), (dict(Bs=P + 8), ALIGN), (dict(sB=P + 1), ALIGN),
    (dict(mode=TENSOR), WS), (dict(mode=TENSOR, E=2, ws=P, wsb=1024), WS),
])
def test_quantize_b_refusals(L, kw, status):
    assert quantize_b(L, **kw) == status


def norm(L, X=P, ldx=256, R=None, ldr=0, xt=BF16, W=P, wt=BF16, eps=1e-6, Q=P, S=P, scale=None, H=None, M=4, K=256,
         mode=BLOCK):
    return L.dgp_rmsnorm_quantize(X, ldx, R, ldr, xt, W, wt, eps, Q, S, scale, H, M, K, mode, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=FP4), DTYPE), (dict(wt=F16), DTYPE), (dict(xt=F32, wt=BF16), DTYPE), (dict(mode=6), SCALE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(K=96, ldx=96), SHAPE), (dict(K=32, ldx=32, mode=NONE), SHAPE),
    (dict(X=None), NULL), (dict(W=None), NULL), (dict(Q=None), NULL), (dict(S=None), NULL),
    (dict(mode=TENSOR), NULL), (dict(scale=P), SCALE), (dict(R=P, ldr=128), SHAPE), (dict(R=P + 2, ldr=256), ALIGN),
    (dict(W=P + 2), ALIGN), (dict(H=P + 8), ALIGN), (dict(R=P, ldr=257), ALIGN),
])
def test_rmsnorm_refusals(L, kw, status):
    assert norm(L, **kw) == status


def swiglu(L, G=P, ldg=512, U=P, ldu=512, xt=BF16, Q=P, S=P, scale=None, M=4, K=256, mode=BLOCK):
    return L.dgp_swiglu_quantize(G, ldg, U, ldu, xt, Q, S, scale, M, K, mode, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=9), DTYPE), (dict(mode=-1), SCALE), (dict(K=320, ldg=640, ldu=640), SHAPE), (dict(ldg=128), SHAPE),
    (dict(ldu=255), SHAPE), (dict(G=None), NULL), (dict(U=None), NULL), (dict(Q=None), NULL), (dict(S=None), NULL),
    (dict(mode=TENSOR), NULL), (dict(G=P + 4), ALIGN), (dict(ldu=513), ALIGN), (dict(mode=NONE, scale=P), SCALE),
])
def test_swiglu_refusals(L, kw, status):
    assert swiglu(L, **kw) == status


def test_binding_refuses_host_tensors(dgp):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dgp.quantize(x, dgp.SCALE_BLOCK128)
    with pytest.raises(ValueError):
        dgp.quantize_b(x, dgp.SCALE_BLOCK128)
    with pytest.raises(ValueError):
        dgp.rmsnorm_quantize(x, x[0], dgp.SCALE_BLOCK128)
    with pytest.raises(ValueError):
        dgp.swiglu_quantize(x, x, dgp.SCALE_BLOCK128)


class Fake:
    """Stands for a device tensor in the binding's shape checks."""

    def __init__(self, t, device="cuda:0"):
        self.t, self.is_cuda, self.device = t, True, torch.device(device)

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_shape_checks(dgp):
    bf = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="2-D"):
        dgp._rows(Fake(bf[0]), "X")
    with pytest.raises(ValueError, match="contiguous"):
        dgp._rows(Fake(bf.t()), "X")
    with pytest.raises(ValueError, match="overlap"):
        dgp._rows(Fake(bf[:1].expand(4, 256)), "X")
    with pytest.raises(ValueError, match="must be"):
        dgp._rows(Fake(bf), "residual", torch.Size((3, 256)), Fake(bf))
    with pytest.raises(ValueError, match="float16"):
        dgp._rows(Fake(bf.half()), "residual", bf.shape, Fake(bf))
    assert dgp._rows(Fake(bf[:, :128]), "X") == 256 and dgp._rows(Fake(bf[:1, :128]), "X") == 128
    X = Fake(bf)
    for kw in (dict(scale=Fake(torch.ones(2)), mode=dgp.SCALE_TENSOR), dict(scale=Fake(torch.ones(1).double()), mode=dgp.SCALE_TENSOR),
               dict(out=Fake(bf), mode=dgp.SCALE_MX128), dict(scales=Fake(torch.ones(4, 2)), mode=dgp.SCALE_MX128),
               dict(scales=Fake(torch.ones(4, 2)), mode=dgp.SCALE_NONE),
               dict(scales=Fake(torch.ones(4, 2), "cuda:1"), mode=dgp.SCALE_BLOCK128)):
        mode = kw.pop("mode")
        with pytest.raises(ValueError):
            dgp._operand_out(X, 4, 256, mode, kw.get("scale"), kw.get("out"), kw.get("scales"), None)
    with pytest.raises(dgp.DgpError) as e:
        dgp._operand_out(X, 4, 256, dgp.SCALE_MX128, Fake(torch.ones(1)), None, None, None)
    assert e.value.status == SCALE
    with pytest.raises(dgp.DgpError):
        dgp._mode(dgp.SCALE_NONE, False)
    with pytest.raises(dgp.DgpError):
        dgp._mode(17, True)
    with pytest.raises(TypeError):
        dgp.input_code(bf.double())


def grouped(L, A=P, a_rows=64, Bs=P, C=P, M=64, N=128, K=256, E=4, offsets=P, rows=None, dtype=FP8, mode=MX, sA=P, sB=P,
            cfg=None):
    return L.dgp_gemm_preshuffle_grouped(A, a_rows, Bs, C, M, N, K, E, offsets, rows, dtype, mode, sA, sB, cfg, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F16), DTYPE), (dict(dtype=F32), DTYPE), (dict(mode=NONE), SCALE), (dict(dtype=BF16), SCALE),
    (dict(dtype=FP4, mode=MX), SCALE), (dict(M=-1), SHAPE), (dict(N=120), SHAPE), (dict(K=0), SHAPE), (dict(K=192), SHAPE),
    (dict(mode=BLOCK, N=64), SHAPE), (dict(E=-1), SHAPE), (dict(E=65536), SHAPE), (dict(a_rows=-1), SHAPE),
    (dict(a_rows=63), SHAPE), (dict(rows=P, a_rows=0), SHAPE), (dict(rows=P, a_rows=1 << 25), SHAPE),
    (dict(A=None), NULL), (dict(Bs=None), NULL), (dict(C=None), NULL), (dict(offsets=None), NULL), (dict(sA=None), NULL),
    (dict(A=P + 8), ALIGN), (dict(C=P + 4), ALIGN), (dict(offsets=P + 2), ALIGN), (dict(rows=P + 1), ALIGN),
    (dict(sA=P + 2, mode=BLOCK), ALIGN),
    (dict(M=1 << 29, a_rows=1 << 29, N=1 << 20), SHAPE),
])
def test_grouped_refusals(L, kw, status):
    assert grouped(L, **kw) == status


def test_grouped_configurations(L, dgp):
    for cfg in (dict(tile_m=64, tile_n=32, tile_k=128), dict(tile_m=128, tile_n=128, tile_k=128), dict(tile_m=1, tile_n=16), dict(tile_m=16, tile_n=32, waves_m=2),
                dict(tile_m=256, tile_n=256, tile_k=128, schedule=3), dict(tile_m=256, tile_n=256, tile_k=64)):
        c = dgp.Config(**cfg)
        assert grouped(L, cfg=ctypes.byref(c)) == CONFIG, cfg
    assert grouped(L, M=0, A=None, Bs=None, C=None, offsets=None) == OK
    assert grouped(L, E=0, A=None, Bs=None, C=None, offsets=None) == OK


def test_grouped_binding_checks(dgp):
    A = torch.zeros(6, 256, dtype=torch.bfloat16)
    Bs = torch.zeros(3, 32, 256, dtype=torch.bfloat16)
    off = torch.zeros(4, dtype=torch.int32)
    rows = torch.zeros(9, dtype=torch.int32)
    ok = lambda **kw: dgp.check_grouped_operands(**{**dict(A=A, Bs=Bs, offsets=off, sA=None, sB=None,  # noqa: E731
                                                          mode=dgp.SCALE_NONE, rows=None, out=None), **kw})
    ok()
    ok(rows=rows, out=torch.zeros(9, 32, dtype=torch.bfloat16))
    for kw in (dict(A=A[0]), dict(Bs=Bs[0]), dict(Bs=Bs.half()), dict(Bs=Bs[:, :, :128]), dict(offsets=off[:3]),
               dict(offsets=off.long()), dict(rows=rows.long()), dict(rows=rows.view(3, 3)),
               dict(out=torch.zeros(6, 32)), dict(rows=rows, out=torch.zeros(6, 32, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            ok(**kw)
    f8 = dict(A=A.to(torch.float8_e4m3fn), Bs=Bs.to(torch.float8_e4m3fn), mode=dgp.SCALE_TENSOR)
    ok(**f8, sA=torch.ones(1), sB=torch.ones(3))
    with pytest.raises(ValueError):
        ok(**f8, sA=torch.ones(1), sB=torch.ones(1))
    with pytest.raises(ValueError):
        ok(**{**f8, "mode": dgp.SCALE_MX128}, sA=torch.ones(12), sB=torch.ones(192))
