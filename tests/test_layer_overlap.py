"""Results of the layer operators that share some elements of what the call reads, without
being in its place.  No GPU work: where the checks pass, an injected launch failure ends
the call."""
import pytest

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from matrix_orthogonalizing_optimizer_shape_gb300 import layer as L
from test_layer_args import FAKE, M, grad_args, lib, linear_args  # noqa: F401

X, W, R, NEW = FAKE, FAKE + (1 << 20), FAKE + (2 << 20), FAKE + (3 << 20)


def norm(lib, residual=None, h=None, y=M(data=NEW)):  # noqa: F811
    return lib.dion3_rms_norm(4, 64, M(data=X), residual, W, d3.BF16, 1e-6, h, y, None, None, None)


def norm_backward(lib, dh=None, dx=M(data=NEW)):  # noqa: F811
    return lib.dion3_rms_norm_backward(4, 64, M(data=X), M(data=R), W, d3.BF16, W, dh, dx, None, 0, None, 0, None)


def linear(lib, **kw):  # noqa: F811
    return lib.dion3_linear(linear_args(**{"x": M(data=X), "w": M(data=W), "y": M(data=NEW), **kw}), None, 0, None)


def linear_backward(lib, **kw):  # noqa: F811
    kw = {"dy": M(data=X), "w": M(data=W), "x": M(data=R), "dx": M(data=NEW), "dw": M(data=NEW + (1 << 20)), **kw}
    ws = NEW + (2 << 20) if "act" in kw else None
    return lib.dion3_linear_backward(grad_args(**kw), ws, 1 << 20 if ws else 0, None)


@pytest.mark.parametrize("call,kw,names", [
    (norm, dict(h=M(data=X + 128)), "x and h"), (norm, dict(y=M(data=X + 2)), "x and y"),
    (norm, dict(y=M(data=X + 384)), "x and y"), (norm, dict(residual=M(data=R), h=M(data=R - 128)), "residual and h"),
    (norm, dict(h=M(data=R), y=M(data=R + 128)), "h and y"),
    (norm_backward, dict(dx=M(data=X + 128)), "dy and dx"), (norm_backward, dict(dx=M(data=R + 8)), "h and dx"),
    (norm_backward, dict(dh=M(data=NEW - 256)), "dh and dx"),
    (linear, dict(y=M(data=X + 128)), "x and y"), (linear, dict(residual=M(data=NEW + 128)), "residual and y"),
    (linear, dict(z=M(data=NEW + 2)), "y and z"), (linear, dict(z=M(data=X + 256)), "x and z"),
    (linear_backward, dict(dx=M(data=X + 128)), "dy and dx"), (linear_backward, dict(dx=M(data=R - 126)), "x and dx"),
])
def test_shared_elements_are_refused(lib, call, kw, names):  # noqa: F811
    assert call(lib, **kw) == d3.ERR_INVALID_ARG
    assert lib.dion3_last_error().decode() == f"{names} share memory"


@pytest.mark.parametrize("call,kw", [
    (norm, dict(h=M(data=X))), (norm, dict(residual=M(data=R), h=M(data=R))), (norm, dict(y=M(data=X))),
    (norm, dict(y=M(data=X + 512))), (norm_backward, dict(dx=M(data=X))), (norm_backward, dict(dh=M(data=NEW))),
    (norm_backward, {}), (linear, {}), (linear, dict(residual=M(data=NEW))), (linear, dict(y=M(data=X + 512))),
    (linear, dict(x=M(data=X, ld=128), y=M(data=X + 128, ld=128))), (linear_backward, {}),
    (linear_backward, dict(dx=M(data=R), dw=L._Matrix())), (linear_backward, dict(dx=M(data=R + 128), dw=L._Matrix())),
    # With an activation the products read dz, formed in the workspace before.
    (linear_backward, dict(act=1, z=M(data=W), dx=M(data=X + 128))),
    (linear_backward, dict(dy=M(data=X, ld=128), dx=M(data=X + 128, ld=128))),
])
def test_places_that_pass(lib, monkeypatch, call, kw):  # noqa: F811
    monkeypatch.setenv("DION3_INJECT", "launch_fail")
    assert call(lib, **kw) == d3.ERR_CUDA and b"injected" in lib.dion3_last_error(), lib.dion3_last_error()
