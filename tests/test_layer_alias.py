"""Which of a gradient's matrices may share memory.  No GPU work: where the
checks pass, an injected launch failure ends the call."""
import pytest

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from matrix_orthogonalizing_optimizer_shape_gb300 import layer as L
from test_layer_args import FAKE, M, grad_args, lib  # noqa: F401

DY, W, X, NEW = FAKE, FAKE + 4096, FAKE + 8192, FAKE + 32768


@pytest.mark.parametrize("dx,dw,ok", [
    (NEW, True, True), (DY, True, False), (W, True, False), (X, True, False),
    (DY, False, False), (W, False, False),
    (X, False, True),  # x is read for dw only
])
def test_dx_may_take_the_place_of_an_unread_x(lib, monkeypatch, dx, dw, ok):  # noqa: F811
    monkeypatch.setenv("DION3_INJECT", "launch_fail")
    a = grad_args(dx=M(data=dx), dw=M(data=FAKE + 16384) if dw else L._Matrix())
    got = lib.dion3_linear_backward(a, None, 0, None)
    assert (got, b"injected" in lib.dion3_last_error()) == ((d3.ERR_CUDA, True) if ok else (d3.ERR_INVALID_ARG, False))
