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
