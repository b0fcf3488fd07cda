"""Host-side refusals of the layer norm and of the gradients: every bad argument
is turned down with its documented status before any HIP call (only invalid
calls and no-ops are made, so no device is touched), and the binding's own
checks raise before a launch."""
import pytest
import torch

import test_host_operands as ops
from test_host_operands import (ALIGN, BF16, BLOCK, DTYPE, F16, F32, FP4, FP8, MX, MX32, NONE, NULL, OK, SCALE, SHAPE, TENSOR,
                                WS, L, bf, dgp)  # noqa: F401 (fixtures)

Y, X, S, W, R, D, DW, DB, T, U = (0x40000000 + i * 0x10000000 for i in range(10))   # far apart, never dereferenced


def refused(L, status):
    return status == SHAPE and b"overlap" in L.dgp_last_error()


# ------------------------------------------------------------ the layer norm

def layernorm(L, X=X, ldx=256, R=None, ldr=0, xt=BF16, W=W, B=None, wt=BF16, eps=1e-5, Q=D, S=S, scale=None, H=None, M=4,
              K=256, mode=BLOCK):
    return L.dgp_layernorm_quantize(X, ldx, R, ldr, xt, W, B, wt, eps, Q, S, scale, H, M, K, mode, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=FP4), DTYPE), (dict(wt=F16), DTYPE), (dict(xt=F32, wt=BF16), DTYPE), (dict(mode=6), SCALE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(K=96, ldx=96), SHAPE), (dict(K=32, ldx=32, mode=NONE), SHAPE), (dict(M=-1), SHAPE), (dict(ldx=128), SHAPE),
    (dict(X=None), NULL), (dict(W=None), NULL), (dict(Q=None), NULL), (dict(S=None), NULL),
    (dict(mode=TENSOR), NULL), (dict(scale=T), SCALE), (dict(R=R, ldr=128), SHAPE), (dict(R=R + 2, ldr=256), ALIGN),
    (dict(W=W + 2), ALIGN), (dict(H=DB + 8), ALIGN), (dict(R=R, ldr=257), ALIGN), (dict(B=DB + 4), ALIGN),
])
def test_layernorm_refusals(L, kw, status):
    assert layernorm(L, **kw) == status


@pytest.mark.parametrize("kw", [
    dict(B=D), dict(B=D + 4 * 256 - 16), dict(B=D - 496), dict(B=D - 1008, wt=F32), dict(B=S - 496), dict(B=S + 16),
    dict(R=R, ldr=256, H=DB, B=DB + 4 * 512 - 16), dict(W=D), dict(Q=X), dict(S=X + 64), dict(S=D + 4 * 256 - 4),
])
def test_layernorm_refuses_overlap(L, kw):
    assert refused(L, layernorm(L, **kw))


# -------------------------------------------------------------- the norms back

def norm_back(L, layer=True, Y=Y, ldy=256, type=BF16, X=X, ldx=256, S=None, mode=NONE, W=W, wt=BF16, R=None, ldr=0, eps=1e-5,
              D=D, dW=DW, dB=DB, M=4, K=256, ws=T, wsb=1 << 40):
    if layer:
        return L.dgp_layernorm_backward(Y, ldy, type, X, ldx, S, mode, W, wt, R, ldr, eps, D, dW, dB, M, K, ws, wsb, None)
    return L.dgp_rmsnorm_backward(Y, ldy, type, X, ldx, S, mode, W, wt, R, ldr, eps, D, dW, M, K, ws, wsb, None)


both = pytest.mark.parametrize("layer", [True, False])


@both
@pytest.mark.parametrize("kw,status", [
    (dict(type=FP8), DTYPE), (dict(type=FP4), DTYPE), (dict(type=-1), DTYPE), (dict(wt=F16), DTYPE), (dict(type=F32), DTYPE),
    (dict(mode=MX32), SCALE), (dict(mode=-1), SCALE), (dict(mode=9), SCALE),
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=-64), SHAPE), (dict(K=96), SHAPE), (dict(K=192, mode=MX, S=S), SHAPE),
    (dict(K=1 << 23, ldy=1 << 23, ldx=1 << 23), SHAPE), (dict(eps=-1e-9), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(eps=float("inf")), SHAPE),
    (dict(ldy=192), SHAPE), (dict(ldx=128), SHAPE), (dict(R=R, ldr=255), SHAPE),
    (dict(Y=None), NULL), (dict(X=None), NULL), (dict(W=None), NULL), (dict(D=None), NULL), (dict(dW=None), NULL),
    (dict(mode=TENSOR), NULL), (dict(mode=BLOCK), NULL), (dict(mode=MX), NULL),
    (dict(Y=Y + 8), ALIGN), (dict(ldy=260), ALIGN), (dict(X=X + 2), ALIGN), (dict(ldx=257), ALIGN), (dict(ldx=264, mode=MX, S=S), ALIGN),
    (dict(R=R + 4, ldr=256), ALIGN), (dict(W=W + 2), ALIGN), (dict(D=D + 8), ALIGN), (dict(dW=DW + 4), ALIGN),
    (dict(mode=BLOCK, S=S + 2), ALIGN), (dict(mode=TENSOR, S=S + 1), ALIGN), (dict(ws=T + 4), ALIGN),
    (dict(ws=None, M=100), WS), (dict(wsb=16, M=100), WS),       # (4 rows of 256 are one workgroup's: none needed)
])
def test_norm_backward_refusals(L, layer, kw, status):
    assert norm_back(L, layer, **kw) == status
    assert L.dgp_last_error()


def test_layernorm_backward_bias_gradient_alignment(L):
    assert norm_back(L, dB=DB + 8) == ALIGN


@both
def test_norm_backward_no_columns(L, layer):
    assert norm_back(L, layer, K=0, Y=None, X=None, W=None, D=None, dW=None, dB=None, ws=None, wsb=0) == OK


@both
def test_norm_backward_workspace(L, layer):
    """Exactly the documented number is enough, a byte less is not, and it grows with neither past a machine's worth of rows."""
    bytes_of = L.dgp_norm_backward_workspace_bytes
    assert bytes_of(0, 256, layer) == bytes_of(4, 0, layer) == bytes_of(-1, 256, layer) == 0
    for m, k in ((40, 256), (5000, 2048), (100000, 8192), (3, 16448)):
        need = bytes_of(m, k, layer)
        assert need > 0 and norm_back(L, layer, M=m, K=k, ldy=k, ldx=k, wsb=need - 1) == WS
    assert bytes_of(1 << 20, 8192, layer) == bytes_of(1 << 22, 8192, layer) <= 2 * 256 * 2 * 8192 * 4


@both
def test_norm_backward_workspace_of_any_size(L, layer):
    """The query takes what the operator would refuse: lengths that are no multiple of 64, down to one element."""
    for k in (1, 7, 8, 9, 63, 65, 511, 513, 8191, 8193):
        for m in (1, 2, 127, 1 << 30):
            assert 0 <= L.dgp_norm_backward_workspace_bytes(m, k, layer) <= (256 * 2 * k + 4 * m) * 4


@both
@pytest.mark.parametrize("kw", [
    # dX over a shifted or strided dY, R or X, over codes, the weight or the scales
    dict(D=Y + 512), dict(D=Y, ldy=512), dict(D=X + 512), dict(D=X, ldx=512), dict(D=R + 16, R=R, ldr=256), dict(D=R, R=R, ldr=512),
    dict(D=X, S=S, mode=TENSOR), dict(D=W), dict(D=W - 4 * 512 + 16), dict(D=S, S=S, mode=TENSOR), dict(D=S - 2032, S=S, mode=BLOCK),
    dict(D=S - 2032, S=S, mode=MX),
    # rows that are read twice
    dict(D=Y, K=8256, ldy=8256, ldx=8256), dict(D=X, K=8256, ldy=8256, ldx=8256),
    # the sums and the workspace over inputs and each other
    dict(dW=Y + 2032), dict(dW=X), dict(dW=R, R=R, ldr=256), dict(dW=W), dict(dW=D + 2032), dict(dW=S, S=S, mode=MX), dict(dW=T, M=100),
    dict(M=100, ws=Y), dict(M=100, ws=X + 16), dict(M=100, ws=W), dict(M=100, ws=D), dict(M=100, ws=DW + 1008), dict(M=100, ws=R, R=R, ldr=256), dict(M=100, ws=S, S=S, mode=BLOCK),
])
def test_norm_backward_refuses_overlap(L, layer, kw):
    assert refused(L, norm_back(L, layer, **kw))


@pytest.mark.parametrize("kw", [dict(dB=DW + 1008), dict(dB=DW, M=0), dict(dB=Y), dict(dB=X + 2032), dict(dB=D), dict(dB=W), dict(dB=T, M=100)])
def test_layernorm_bias_gradient_overlap(L, kw):
    assert refused(L, norm_back(L, **kw))


# ------------------------------------------------- the gated activation back

def swiglu_back(L, Y=Y, ldy=256, type=BF16, G=X, ldg=256, U=U, ldu=256, SG=None, ldsg=2, SU=None, ldsu=2, mode=NONE, D=D, M=4,
                K=256):
    return L.dgp_swiglu_backward(Y, ldy, type, G, ldg, U, ldu, SG, ldsg, SU, ldsu, mode, D, M, K, None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=FP8), DTYPE), (dict(mode=MX32), SCALE), (dict(mode=-2), SCALE), (dict(M=-1), SHAPE), (dict(K=-64), SHAPE),
    (dict(K=96), SHAPE), (dict(K=64, mode=MX), SHAPE), (dict(K=1 << 23), SHAPE), (dict(M=1 << 30), SHAPE),
    (dict(ldy=128), SHAPE), (dict(ldg=128), SHAPE), (dict(ldu=128), SHAPE),
    (dict(mode=MX, SG=S, SU=S, ldsg=1), SHAPE), (dict(mode=BLOCK, SG=S, SU=S, ldsu=1), SHAPE),
    (dict(Y=None), NULL), (dict(G=None), NULL), (dict(U=None), NULL), (dict(D=None), NULL), (dict(mode=MX, SG=S), NULL),
    (dict(mode=TENSOR, SU=S), NULL),
    (dict(Y=Y + 2), ALIGN), (dict(G=X + 4), ALIGN), (dict(U=U + 8), ALIGN), (dict(ldu=260), ALIGN), (dict(D=D + 8), ALIGN),
    (dict(mode=BLOCK, SG=S + 2, SU=S), ALIGN), (dict(mode=TENSOR, SG=S, SU=S + 2), ALIGN),
])
def test_swiglu_backward_refusals(L, kw, status):
    assert swiglu_back(L, **kw) == status


def test_swiglu_backward_no_ops(L):
    assert swiglu_back(L, M=0, Y=None, G=None, U=None, D=None) == OK and swiglu_back(L, K=0, Y=None, G=None, U=None, D=None) == OK


@pytest.mark.parametrize("kw", [
    dict(D=Y), dict(D=Y + 2032), dict(D=X), dict(D=U), dict(D=X, U=X + 512), dict(D=X, U=X + 512, ldg=512, ldu=1024),
    dict(D=X, U=X + 1024, ldg=512, ldu=512), dict(D=X + 16, U=X + 528, ldg=512, ldu=512), dict(D=X, U=X + 256, ldg=512, ldu=512, mode=MX, SG=S, SU=S),
    dict(D=S - 4080, SG=S, SU=R, mode=MX), dict(D=S - 4080, SG=R, SU=S, mode=BLOCK), dict(D=S, SG=S, SU=S, mode=TENSOR),
])
def test_swiglu_backward_refuses_overlap(L, kw):
    assert refused(L, swiglu_back(L, **kw))


# --------------------------------------------------------- a weight's gradient

def wgrad(L, dC=Y, ldc=128, X=X, x_rows=64, dtype=FP8, S=S, mode=MX, dB=D, ot=F32, acc=0, M=64, N=128, K=256, E=1, offsets=None,
          rows=None, ws=None, wsb=0):
    return L.dgp_gemm_wgrad(dC, ldc, X, x_rows, dtype, S, mode, dB, ot, acc, M, N, K, E, offsets, rows, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=FP4), DTYPE), (dict(dtype=F16), DTYPE), (dict(dtype=F32), DTYPE), (dict(ot=F16), DTYPE), (dict(ot=FP8), DTYPE),
    (dict(acc=2), DTYPE), (dict(acc=1, ot=BF16), DTYPE), (dict(mode=MX32), SCALE), (dict(mode=NONE), SCALE), (dict(dtype=BF16), SCALE),
    (dict(mode=-1), SCALE), (dict(M=-1), SHAPE), (dict(N=-16), SHAPE), (dict(K=-128), SHAPE), (dict(E=-1), SHAPE), (dict(E=65536), SHAPE),
    (dict(N=120), SHAPE), (dict(K=192), SHAPE), (dict(K=96, dtype=BF16, mode=NONE), SHAPE), (dict(N=(1 << 22) + 16), SHAPE),
    (dict(K=(1 << 22) + 128), SHAPE), (dict(M=1 << 30, x_rows=1 << 30), SHAPE), (dict(x_rows=63), SHAPE), (dict(x_rows=-1), SHAPE),
    (dict(ldc=112), SHAPE), (dict(ldc=(1 << 25) + 8), SHAPE), (dict(offsets=T, rows=U, x_rows=0), SHAPE),
    (dict(offsets=T, rows=U, x_rows=1 << 25), SHAPE), (dict(N=1 << 22, K=1 << 22, ldc=1 << 22, E=65535, offsets=T), SHAPE),
    (dict(E=2), NULL), (dict(rows=U), NULL), (dict(dB=None), NULL), (dict(dC=None), NULL), (dict(X=None), NULL), (dict(S=None), NULL),
    (dict(dC=Y + 8), ALIGN), (dict(ldc=132), ALIGN), (dict(X=X + 4), ALIGN), (dict(dB=D + 8), ALIGN), (dict(offsets=T + 2), ALIGN),
    (dict(offsets=T, rows=U + 1), ALIGN), (dict(S=S + 2, mode=BLOCK), ALIGN), (dict(S=S + 1, mode=TENSOR), ALIGN), (dict(ws=T + 8), ALIGN),
])
def test_wgrad_refusals(L, kw, status):
    assert wgrad(L, **kw) == status
    assert L.dgp_last_error()


def test_wgrad_no_ops(L):
    for kw in (dict(N=0), dict(K=0), dict(E=0)):
        assert wgrad(L, dC=None, X=None, S=None, dB=None, **kw) == OK


def test_wgrad_workspace(L):
    f = L.dgp_wgrad_workspace_bytes
    assert f(0, 128, 256, 1) == f(64, 0, 256, 1) == f(64, 128, 0, 1) == f(64, 128, 256, 0) == f(-1, 128, 256, 1) == 0
    assert f(64, 128, 256, 1) == 0                       # few rows: one part
    need = f(8192, 128, 256, 1)
    assert need > 0 and need % (128 * 256 * 4) == 0      # several parts, each fp32
    big = dict(M=8192, x_rows=8192)
    assert wgrad(L, **big) == WS and wgrad(L, ws=T, wsb=need - 1, **big) == WS
    for m, n, k, e in ((1 << 29, 1 << 22, 1 << 22, 65535), (1 << 30, 16, 64, 1), (1, 1 << 22, 1 << 22, 1)):
        assert f(m, n, k, e) <= 16 * e * n * k * 4       # (and nothing overflows on the way)


@pytest.mark.parametrize("kw", [
    dict(dB=Y), dict(dB=Y + (63 * 128 + 128) * 2 - 16), dict(dB=Y - 128 * 256 * 4 + 16), dict(dB=X), dict(dB=X + 64 * 256 - 16), dict(dB=S),
    dict(dB=S - 128 * 256 * 4 + 16), dict(dB=S, mode=TENSOR), dict(offsets=D), dict(offsets=D + 128 * 256 * 4 - 4), dict(offsets=T, rows=D),
    dict(M=8192, x_rows=8192, ws=Y, wsb=1 << 30), dict(M=8192, x_rows=8192, ws=X, wsb=1 << 30), dict(M=8192, x_rows=8192, ws=S, wsb=1 << 30),
    dict(M=8192, x_rows=8192, ws=D, wsb=1 << 30), dict(M=8192, x_rows=8192, ws=T, offsets=T, wsb=1 << 30),
])
def test_wgrad_refuses_overlap(L, kw):
    assert refused(L, wgrad(L, **kw))


# The binding's own checks; host tensors that pass them all are refused last.

F8 = torch.float8_e4m3fn


def codes(*shape):
    return torch.zeros(*shape, dtype=F8)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "device tensor"), (dict(weight=bf(128)), ValueError, "weight must hold"),
    (dict(bias=bf(128)), ValueError, "bias must hold"), (dict(bias=torch.zeros(256)), ValueError, "bias"),
    (dict(weight=torch.zeros(256), bias=bf(256)), ValueError, "bias"), (dict(bias=bf(512)[::2]), ValueError, "contiguous"),
    (dict(residual=bf(3, 256)), ValueError, "residual must be"), (dict(residual_out=bf(4, 256)), ValueError, "needs a residual"),
    (dict(X=bf(256)), ValueError, "2-D"), (dict(eps="x"), TypeError, None),
])
def test_layernorm_binding_checks(dgp, kw, error, match):
    with pytest.raises(error, match=match):
        dgp.layernorm_quantize(**{**dict(X=bf(4, 256), weight=bf(256), bias=bf(256), scale_mode=BLOCK), **kw})


NORM_BACK = [
    (dict(), ValueError, "device tensor"), (dict(dY=bf(256)), ValueError, "2-D"), (dict(dY=None), TypeError, "must be a tensor"),
    (dict(dY=bf(4, 256).double()), TypeError, "input type"), (dict(X=bf(3, 256)), ValueError, "X must be"),
    (dict(X=bf(4, 256).float()), ValueError, "X must be"), (dict(X=codes(4, 256)), ValueError, "X must be"),
    (dict(scales=u8(4, 2)), ValueError, "no scales"), (dict(scale_mode=MX), ValueError, "X must be"),
    (dict(scale_mode=MX, X=codes(4, 256)), ValueError, "scales are needed"),
    (dict(scale_mode=MX, X=codes(4, 256), scales=torch.zeros(4, 2)), ValueError, "scales must be"),
    (dict(scale_mode=MX, X=codes(4, 256), scales=u8(4, 4)[:, :2]), ValueError, "contiguous"),
    (dict(scale_mode=BLOCK, X=codes(4, 256), scales=torch.zeros(4, 1)), ValueError, "scales must be"),
    (dict(scale_mode=TENSOR, X=codes(4, 256), scales=torch.zeros(2)), ValueError, "one float32"),
    (dict(weight=bf(128)), ValueError, "weight must hold"), (dict(weight=bf(256).half()), ValueError, "weight must hold"),
    (dict(residual_grad=bf(4, 128)), ValueError, "residual_grad must be"), (dict(residual_grad=bf(4, 256).half()), ValueError, "residual_grad is"),
    (dict(dx=bf(4, 128)), ValueError, "dx must be"), (dict(dx=bf(256, 4).t()), ValueError, "contiguous"),
    (dict(dweight=bf(256)), ValueError, "dweight must be"), (dict(dweight=torch.zeros(1, 256)), ValueError, "dweight must be"),
    (dict(eps="x"), TypeError, None), (dict(scale_mode="x"), TypeError, None),
]


@pytest.mark.parametrize("kw,error,match", NORM_BACK)
@pytest.mark.parametrize("name", ["layernorm_backward", "rmsnorm_backward"])
def test_norm_backward_binding_checks(dgp, name, kw, error, match):
    with pytest.raises(error, match=match):
        getattr(dgp, name)(**{**dict(dY=bf(4, 256), X=bf(4, 256), weight=bf(256)), **kw})


def test_layernorm_backward_bias_gradient_check(dgp):
    with pytest.raises(ValueError, match="dbias must be"):
        dgp.layernorm_backward(bf(4, 256), bf(4, 256), bf(256), dbias=bf(256))


@pytest.mark.parametrize("mode", [MX32, 5, -1, 17])
def test_modes_that_no_gradient_reads(dgp, mode):
    for f in (lambda: dgp.layernorm_backward(bf(4, 256), u8(4, 128), bf(256), mode, u8(4, 8)),
              lambda: dgp.rmsnorm_backward(bf(4, 256), u8(4, 128), bf(256), mode, u8(4, 8)),
              lambda: dgp.swiglu_backward(bf(4, 256), u8(4, 128), u8(4, 128), mode, u8(4, 8), u8(4, 8)),
              lambda: dgp.gemm_wgrad(bf(4, 256), u8(4, 128), u8(4, 8), mode)):
        with pytest.raises(dgp.DgpError) as e:
            f()
        assert e.value.status == SCALE


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "device tensor"), (dict(up=bf(4, 128)), ValueError, "up must be"), (dict(gate=bf(5, 256)), ValueError, "gate must be"),
    (dict(up=bf(4, 256).half()), ValueError, "up must be"), (dict(gate_scales=u8(4, 2)), ValueError, "no scales"),
    (dict(scale_mode=MX, gate=codes(4, 256), up=codes(4, 256), gate_scales=u8(4, 2)), ValueError, "up_scales are needed"),
    (dict(scale_mode=MX, gate=codes(4, 256), up=codes(4, 256), gate_scales=u8(4, 1), up_scales=u8(4, 2)), ValueError, "gate_scales must be"),
    (dict(scale_mode=BLOCK, gate=codes(4, 256), up=codes(4, 256), gate_scales=torch.zeros(2, 4).t(), up_scales=torch.zeros(4, 2)),
     ValueError, "contiguous"),
    (dict(scale_mode=TENSOR, gate=codes(4, 256), up=codes(4, 256), gate_scales=torch.ones(1), up_scales=torch.ones(2)), ValueError, "one float32"),
    (dict(out=bf(4, 256)), ValueError, "out must be"), (dict(out=bf(4, 512).float()), ValueError, "out must be"),
    (dict(gate=bf(4, 512)[:, :256], up=bf(4, 512)[:, 256:]), ValueError, "device tensor"),
])
def test_swiglu_backward_binding_checks(dgp, kw, error, match):
    with pytest.raises(error, match=match):
        dgp.swiglu_backward(**{**dict(dY=bf(4, 256), gate=bf(4, 256), up=bf(4, 256)), **kw})


i32 = dict(dtype=torch.int32)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "device tensor"), (dict(dC=bf(32)), ValueError, "2-D"), (dict(dC=bf(6, 32).float()), ValueError, "bfloat16"),
    (dict(X=bf(5, 256)), ValueError, "X has 5 rows"), (dict(X=bf(256)), ValueError, "X must be a 2-D"), (dict(X=bf(6, 256).half()), ValueError, "X must be a 2-D"),
    (dict(X=bf(256, 6).t()), ValueError, "contiguous"), (dict(sX=torch.ones(1)), ValueError, "no scales"),
    (dict(scale_mode=TENSOR), ValueError, "X must be a 2-D"),
    (dict(scale_mode=TENSOR, X=codes(6, 256), sX=torch.ones(2)), ValueError, "sX must hold 1"), (dict(scale_mode=MX, X=codes(6, 256), sX=u8(6, 1)), ValueError, "sX must hold 12"),
    (dict(scale_mode=MX, X=codes(6, 256), sX=torch.zeros(12)), ValueError, "sX must hold 12"),
    (dict(scale_mode=BLOCK, X=codes(6, 256), sX=u8(12)), ValueError, "sX must hold 12"),
    (dict(offsets=torch.zeros(4)), ValueError, "offsets must be"), (dict(offsets=torch.zeros(2, 2, **i32)), ValueError, "offsets must be"),
    (dict(offsets=torch.zeros(0, **i32)), ValueError, "offsets must be"), (dict(offsets=torch.zeros(8, **i32)[::2]), ValueError, "contiguous"),
    (dict(rows=torch.zeros(6, **i32)), ValueError, "rows needs offsets"),
    (dict(offsets=torch.zeros(4, **i32), rows=torch.zeros(5, **i32)), ValueError, "rows must be"),
    (dict(offsets=torch.zeros(4, **i32), rows=torch.zeros(6)), ValueError, "rows must be"),
    (dict(offsets=torch.zeros(4, **i32), rows=torch.zeros(6, **i32), X=bf(2, 256)), ValueError, "device tensor"),
    (dict(out=bf(32, 128)), ValueError, "out must be"), (dict(out=torch.zeros(1, 32, 256)), ValueError, "out must be"),
    (dict(offsets=torch.zeros(4, **i32), out=torch.zeros(32, 256)), ValueError, "out must be"),
    (dict(accumulate=True), ValueError, "accumulate needs out"),
    (dict(accumulate=True, out=bf(32, 256)), (TypeError, ValueError), None), (dict(out_dtype=torch.float16), (TypeError, ValueError), None),
])
def test_wgrad_binding_checks(dgp, kw, error, match):
    with pytest.raises(error, match=match):
        dgp.gemm_wgrad(**{**dict(dC=bf(6, 32), X=bf(6, 256)), **kw})
