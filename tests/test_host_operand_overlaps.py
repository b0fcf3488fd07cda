"""Host-side refusals of operands that overlap: what a launch would write is
compared with everything it reads before any HIP call (only invalid calls are
made, so no device is touched)."""
import pytest

import test_host_operands as ops
from test_host_operands import L, dgp  # noqa: F401 (fixtures)

X, Q, S, W, H, R = (0x40000000 + i * 0x1000000 for i in range(6))   # far apart, never dereferenced


def refused(L, status):
    return status == ops.SHAPE and b"overlap" in L.dgp_last_error()


@pytest.mark.parametrize("at", [0, 4, 2044])
@pytest.mark.parametrize("m,ldx", [(4, 256), (2, 768)])
def test_measured_tensor_scale_inside_the_input(L, at, m, ldx):
    """The one scale that dgp_quantize measures, from X's first byte to its last
    (4 rows of 512 bytes; 2 rows, the second from byte 1536 on)."""
    assert refused(L, ops.quantize(L, X=X, Q=Q, S=X + at, M=m, ldx=ldx, mode=ops.TENSOR, ws=W, wsb=1024))


# The norm's weight (256 bf16 values: 512 bytes; fp32: 1024) is read by every row.

@pytest.mark.parametrize("kw", [
    dict(W=Q), dict(W=Q + 4 * 256 - 16), dict(W=Q - 496), dict(W=Q - 1008, wt=ops.F32), dict(W=S - 496), dict(W=S + 16),
    dict(W=S, mode=ops.MX), dict(W=S + 16, mode=ops.MX32), dict(W=Q + 4 * 128 - 16, mode=ops.MX32),
    dict(W=Q, mode=ops.NONE), dict(W=Q + 4 * 512 - 16, mode=ops.NONE), dict(W=H, R=R, ldr=256, H=H),
    dict(W=H - 496, R=R, ldr=256, H=H), dict(W=H + 4 * 512 - 16, R=R, ldr=256, H=H), dict(W=Q, M=1),
])
def test_norm_output_over_the_weight(L, kw):
    assert refused(L, ops.norm(L, **{**dict(X=X, Q=Q, S=S, W=W), **kw}))


# A given per-tensor scale (4 bytes) is read by every workgroup.

@pytest.mark.parametrize("at", [0, 512, 1020])
def test_codes_over_a_given_scale(L, at):
    tensor = dict(Q=Q, S=None, scale=Q + at, mode=ops.TENSOR)
    assert refused(L, ops.quantize(L, X=X, **tensor))
    assert refused(L, ops.norm(L, X=X, W=W, **tensor))
    assert refused(L, ops.swiglu(L, G=X, U=X + 512, **tensor))


def test_residual_stream_over_a_given_scale(L):
    assert refused(L, ops.norm(L, X=X, W=W, R=R, ldr=256, H=H, Q=Q, S=None, scale=H + 2044, mode=ops.TENSOR))


# Outputs on each other.

@pytest.mark.parametrize("kw", [
    dict(S=Q), dict(S=Q + 4 * 256 - 4), dict(S=Q - 28), dict(S=Q, mode=ops.MX), dict(S=Q - 7, mode=ops.MX),
    dict(S=Q + 4 * 128 - 1, mode=ops.MX32), dict(S=Q - 31, mode=ops.MX32),
])
def test_scales_over_codes(L, kw):
    """4 rows of 256: 1024 bytes of e4m3 codes and 8 fp32 or 8 E8M0 scales, or
    512 bytes of E2M1 codes and 32 scales."""
    kw = {**dict(Q=Q, S=S), **kw}
    assert refused(L, ops.quantize(L, X=X, **kw))
    assert refused(L, ops.norm(L, X=X, W=W, **kw))
    assert refused(L, ops.swiglu(L, G=X, U=X + 512, **kw))


@pytest.mark.parametrize("at", [0, 1020])
def test_measured_tensor_scale_over_codes(L, at):
    assert refused(L, ops.quantize(L, X=X, Q=Q, S=Q + at, mode=ops.TENSOR, ws=W, wsb=1024))


@pytest.mark.parametrize("kw", [dict(S=H), dict(S=H - 28), dict(S=H + 2044), dict(S=H + 2047, mode=ops.MX)])
def test_scales_over_the_residual_stream(L, kw):
    assert refused(L, ops.norm(L, **{**dict(X=X, W=W, R=R, ldr=256, H=H, Q=Q), **kw}))


@pytest.mark.parametrize("kw", [
    dict(sB=Q), dict(sB=Q + 3 * 128 * 256 - 4), dict(sB=Q - 20), dict(sB=Q - 3 * 256 + 1, mode=ops.MX),
    dict(sB=Q + 3 * 128 * 128 - 1, mode=ops.MX32), dict(sB=Q - 8, mode=ops.TENSOR, ws=W, wsb=4096),
])
def test_weight_scales_over_weight_codes(L, kw):
    """3 weights of 128 x 256."""
    assert refused(L, ops.quantize_b(L, **{**dict(B=X, Bs=Q, E=3), **kw}))
