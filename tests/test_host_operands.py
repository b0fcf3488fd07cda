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


# The binding's own checks, in the order they are made; host tensors that pass
# them all are refused last.

def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "device tensor"), (dict(X=bf(256)), ValueError, "2-D"), (dict(X=bf(256, 4).t()), ValueError, "contiguous"),
    (dict(X=bf(1, 256).expand(4, 256)), ValueError, "overlap"), (dict(X=bf(4, 256).double()), TypeError, "input type"),
    (dict(X=None), TypeError, "must be a tensor"), (dict(X=[1, 2]), TypeError, "must be a tensor"),
    (dict(scale_mode="x"), TypeError, None), (dict(out=bf(4, 256)), ValueError, "out must be"),
    (dict(out=torch.zeros(4, 128, dtype=torch.float8_e4m3fn)), ValueError, "out must be"),
    (dict(out=torch.zeros(256, 4, dtype=torch.float8_e4m3fn).t()), ValueError, "contiguous"),
    (dict(scales=torch.zeros(4, 2)), ValueError, "scales must be"),
    (dict(scales=torch.zeros(4, dtype=torch.uint8)), ValueError, "scales must be"),
    (dict(scale=torch.ones(1)), ValueError, "SCALE_TENSOR only"),
    (dict(scale_mode=1, scale=torch.ones(2)), ValueError, "one value"),
    (dict(scale_mode=1, scale=torch.ones(1).double()), ValueError, "scale must be"),
    (dict(scale_mode=1, scale=torch.ones(1), scales=torch.ones(1)), ValueError, "no scales to write"),
    (dict(scale_mode=4, out=torch.zeros(4, 128, dtype=torch.uint8)), ValueError, "out must be"),
    (dict(stream="s"), ValueError, "device tensor"),
])
def test_quantize_binding_checks(dgp, kw, error, match):
    with pytest.raises(error, match=match):
        dgp.quantize(**{**dict(X=bf(4, 256), scale_mode=MX), **kw})


@pytest.mark.parametrize("mode", [NONE, 5, -1, 17])
def test_modes_an_operator_does_not_write(dgp, mode):
    for f in (lambda: dgp.quantize(bf(4, 256), mode), lambda: dgp.quantize_b(bf(128, 256), mode)):
        with pytest.raises(dgp.DgpError) as e:
            f()
        assert e.value.status == SCALE
    if mode != NONE:
        for f in (lambda: dgp.rmsnorm_quantize(bf(4, 256), bf(256), mode), lambda: dgp.swiglu_quantize(bf(4, 256), bf(4, 256), mode)):
            with pytest.raises(dgp.DgpError):
                f()


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "device tensor"), (dict(B=bf(256)), ValueError, "2-D or 3-D"), (dict(B=bf(2, 2, 128, 256)), ValueError, "2-D or 3-D"),
    (dict(B=bf(256, 128).t()), ValueError, "contiguous"), (dict(B=bf(128, 256).long()), TypeError, "input type"),
    (dict(out=torch.zeros(128, 256, dtype=torch.uint8)), ValueError, "out must be"),
    (dict(scales=torch.zeros(128, 1, dtype=torch.uint8)), ValueError, "scales must be"),
    (dict(B=bf(3, 128, 256), scales=torch.zeros(128, 2, dtype=torch.uint8)), ValueError, "scales must be"),
])
def test_quantize_b_binding_checks(dgp, kw, error, match):
    with pytest.raises(error, match=match):
        dgp.quantize_b(**{**dict(B=bf(128, 256), scale_mode=MX), **kw})


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "device tensor"), (dict(weight=bf(128)), ValueError, "weight must hold"),
    (dict(weight=bf(1, 256)), ValueError, "weight must hold"), (dict(weight=bf(256).half()), ValueError, "weight must hold"),
    (dict(weight=bf(512)[::2]), ValueError, "contiguous"), (dict(residual=bf(3, 256)), ValueError, "residual must be"),
    (dict(residual=bf(4, 256).half()), ValueError, "residual is"), (dict(residual_out=bf(4, 256)), ValueError, "needs a residual"),
    (dict(residual=bf(4, 256), residual_out=bf(4, 256).float()), ValueError, "residual_out must be"),
    (dict(eps="x"), TypeError, None), (dict(scale_mode=NONE, scales=torch.ones(4, 2)), ValueError, "writes no scales"),
    (dict(weight=torch.zeros(256)), ValueError, "device tensor"),
])
def test_rmsnorm_binding_checks(dgp, kw, error, match):
    with pytest.raises(error, match=match):
        dgp.rmsnorm_quantize(**{**dict(X=bf(4, 256), weight=bf(256), scale_mode=BLOCK), **kw})


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "device tensor"), (dict(up=bf(4, 128)), ValueError, "up must be"),
    (dict(up=bf(4, 256).float()), ValueError, "up is"), (dict(gate=bf(4, 512)[:, :256]), ValueError, "device tensor"),
    (dict(up=bf(256, 4).t()), ValueError, "contiguous"),
])
def test_swiglu_binding_checks(dgp, kw, error, match):
    with pytest.raises(error, match=match):
        dgp.swiglu_quantize(**{**dict(gate=bf(4, 256), up=bf(4, 256), scale_mode=BLOCK), **kw})


def test_binding_follows_the_active_library(dgp):
    """Inside lds_poison_build the native module calls that library."""
    dgp._native()
    with dgp.lds_poison_build() as poison:
        dgp._native()
        assert dgp._bound is poison
    dgp._native()
    assert dgp._bound is dgp.lib()


Z = 0x40000000       # a second one, far from the first


@pytest.mark.parametrize("kw", [
    dict(), dict(Q=P + 2032), dict(Q=Z, S=P + 2044), dict(Q=Z, S=Z + 4096, X=Z + 496, M=2, ldx=1024),
])
def test_quantize_refuses_overlap(L, kw):
    """Q or S inside X's rows, from its first byte to its last."""
    assert quantize(L, **kw) == SHAPE and b"overlap" in L.dgp_last_error()


def test_quantize_b_refuses_overlap(L):
    assert quantize_b(L, Bs=P, sB=Z) == SHAPE and quantize_b(L, Bs=Z, sB=P + 16) == SHAPE
    assert quantize_b(L, Bs=Z, sB=P - 4) == SHAPE    # (two values)
    assert b"overlap" in L.dgp_last_error()


@pytest.mark.parametrize("kw", [
    dict(Q=P), dict(S=P + 64), dict(R=P + 0x8000, ldr=256, Q=P + 0x8000), dict(H=P + 512), dict(H=P, ldx=512),
    dict(H=P, ldx=512, M=1, Q=P), dict(R=P + 0x8000, ldr=512, H=P + 0x8000), dict(H=Z + 512), dict(H=P, Q=P, mode=NONE),
    dict(Q=P, mode=NONE, xt=F16, wt=F16), dict(Q=P + 512, mode=NONE),
])
def test_rmsnorm_refuses_overlap(L, kw):
    """A shifted or differently strided output, the scales, or Q over the residual output."""
    base = dict(X=P, W=Z + 0x100000, Q=Z, S=Z + 0x10000)
    assert norm(L, **{**base, **kw}) == SHAPE and b"overlap" in L.dgp_last_error()


@pytest.mark.parametrize("kw", [dict(Q=P), dict(Q=P, ldg=256, ldu=256, U=P + 512 * 4, M=5, mode=NONE), dict(S=P + 1024), dict(Q=P, mode=NONE)])
def test_swiglu_refuses_overlap(L, kw):
    base = dict(G=P, U=P + 512, Q=Z, S=Z + 0x10000)
    assert swiglu(L, **{**base, **kw}) == SHAPE and b"overlap" in L.dgp_last_error()


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
    # too many threads for one launch; too many tiles for the search's sums
    small = ctypes.byref(dgp.Config(tile_m=16, tile_n=16))
    assert grouped(L, M=1 << 22, a_rows=1 << 22, N=1 << 14, cfg=small) == SHAPE
    assert grouped(L, M=1 << 29, a_rows=1 << 29, N=16, E=64, cfg=small) == SHAPE
    assert b"tiles" in L.dgp_last_error()
    assert grouped(L, M=0, A=None, Bs=None, C=None, offsets=None) == OK
    assert grouped(L, E=0, A=None, Bs=None, C=None, offsets=None) == OK


F8 = torch.float8_e4m3fn
f8 = dict(A=torch.zeros(6, 256, dtype=F8), Bs=torch.zeros(3, 32, 256, dtype=F8))


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "device tensor"),
    (dict(rows=torch.zeros(9, dtype=torch.int32), out=bf(9, 32)), ValueError, "device tensor"),
    (dict(A=bf(256)), ValueError, "2-D"), (dict(Bs=bf(32, 256)), ValueError, "3-D"), (dict(A=bf(6, 256).float()), TypeError, "element type"),
    (dict(Bs=bf(3, 32, 256).half()), ValueError, "one element type"), (dict(Bs=bf(3, 32, 128)), ValueError, "elements per row"),
    (dict(A=bf(256, 6).t()), ValueError, "contiguous"), (dict(offsets=torch.zeros(3, dtype=torch.int32)), ValueError, "offsets must be"),
    (dict(offsets=torch.zeros(4, dtype=torch.int64)), ValueError, "offsets must be"),
    (dict(offsets=torch.zeros(8, dtype=torch.int32)[::2]), ValueError, "contiguous"),
    (dict(rows=torch.zeros(9)), ValueError, "rows must be"), (dict(rows=torch.zeros(3, 3, dtype=torch.int32)), ValueError, "rows must be"),
    (dict(out=torch.zeros(6, 32)), ValueError, "out must be"),
    (dict(rows=torch.zeros(9, dtype=torch.int32), out=bf(6, 32)), ValueError, "out must be"),
    (dict(**f8, scale_mode=TENSOR, sA=torch.ones(1), sB=torch.ones(3)), ValueError, "device tensor"),
    (dict(**f8, scale_mode=TENSOR, sA=torch.ones(1), sB=torch.ones(1)), ValueError, "sB must hold 3"),
    (dict(**f8, scale_mode=TENSOR, sA=torch.ones(6), sB=torch.ones(3)), ValueError, "sA must hold 1"),
    (dict(**f8, scale_mode=MX, sA=torch.ones(12), sB=torch.ones(192)), ValueError, "sA must hold 12"),
    (dict(**f8, scale_mode=MX, sA=torch.ones(12, dtype=torch.uint8), sB=torch.ones(64, dtype=torch.uint8)), ValueError, "sB must hold 192"),
    (dict(**f8, sA=torch.ones(1), sB=torch.ones(3)), ValueError, "ambiguous"),
])
def test_grouped_binding_checks(dgp, kw, error, match):
    base = dict(A=bf(6, 256), Bs=bf(3, 32, 256), offsets=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(error, match=match):
        dgp.gemm_preshuffle_grouped(**{**base, **kw})
