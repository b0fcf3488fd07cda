"""Host-side refusals of operands that overlap: what a launch would write is
compared with everything it reads before any HIP call (only invalid calls are
made, so no device is touched)."""
import pytest

import test_host_operands as ops
from test_host_operands import L, dgp  # noqa: F401 (fixtures)

X, Q, S, W = (0x40000000 + i * 0x1000000 for i in range(4))   # far apart, never dereferenced


def refused(L, status):
    return status == ops.SHAPE and b"overlap" in L.dgp_last_error()


@pytest.mark.parametrize("at", [0, 4, 2044])
@pytest.mark.parametrize("m,ldx", [(4, 256), (2, 768)])
def test_measured_tensor_scale_inside_the_input(L, at, m, ldx):
    """The one scale that dgp_quantize measures, from X's first byte to its last
    (4 rows of 512 bytes; 2 rows, the second from byte 1536 on)."""
    assert refused(L, ops.quantize(L, X=X, Q=Q, S=X + at, M=m, ldx=ldx, mode=ops.TENSOR, ws=W, wsb=1024))
