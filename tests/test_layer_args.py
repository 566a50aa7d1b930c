"""Host-side checks of the layer operators: sizes, refusals and their messages.
No call here launches GPU work."""
import ctypes
import os

import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from matrix_orthogonalizing_optimizer_shape_gb300 import layer as L

FAKE = 0x7F0000000000  # a 256-byte aligned address that no call here reads


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(d3.LIB_PATH):
        d3.build()
    return d3.load_library()


def M(ld=64, dtype=d3.BF16, data=FAKE):
    return L._Matrix(data, ld, dtype)


def P(ldc=64, lds=2, codes=FAKE, scales=FAKE):
    return L._Packed8(codes, ldc, scales, lds)


def linear_args(**kw):
    a = dict(tokens=4, in_features=64, out_features=64, act=0, x=M(data=FAKE), w=M(data=FAKE + 4096),
             y=M(data=FAKE + 8192), residual=L._Matrix(), z=L._Matrix(), z8=L._Packed8(), y8=L._Packed8(), bias=None,
             bias_dtype=0)
    a.update(kw)
    return L._LinearArgs(*a.values())


def grad_args(**kw):
    a = dict(tokens=4, in_features=64, out_features=64, act=0, accumulate=0, dy=M(), w=M(data=FAKE + 4096),
             x=M(data=FAKE + 8192), z=L._Matrix(), x8=L._Packed8(), z8=L._Packed8(), dx=L._Matrix(),
             dw=M(data=FAKE + 16384), db=None)
    a.update(kw)
    return L._LinearGradArgs(*a.values())


INV, UNS, WS = d3.ERR_INVALID_ARG, d3.ERR_UNSUPPORTED, d3.ERR_WORKSPACE


@pytest.mark.parametrize("kw,status,word", [
    (dict(tokens=-1), INV, b"rows"), (dict(in_features=0), INV, b"cols"), (dict(out_features=0), INV, b"cols"),
    (dict(in_features=1 << 25), UNS, b"larger"), (dict(act=4), INV, b"activation"), (dict(act=-1), INV, b"activation"),
    (dict(w=M(dtype=d3.F32)), UNS, b"fp32"), (dict(w=M(dtype=7)), INV, b"dtype"), (dict(x=M(dtype=d3.F16)), INV, b"x"),
    (dict(x=M(data=None)), INV, b"x is NULL"), (dict(y=M(ld=63, data=FAKE + 8192)), INV, b"y"),
    (dict(x=M(data=FAKE + 1)), INV, b"aligned"), (dict(z=M(dtype=d3.F32)), INV, b"z"),
    (dict(z8=P(ldc=63)), INV, b"z8"), (dict(y8=P(lds=1)), INV, b"y8"), (dict(z8=P(scales=None)), INV, b"z8"),
    (dict(bias=FAKE + 2, bias_dtype=d3.F32), INV, b"bias"), (dict(bias=FAKE, bias_dtype=9), INV, b"bias"),
    (dict(y=M(data=FAKE)), INV, b"y may not be x"), (dict(x=M(ld=65)), WS, b"NULL"),
    (dict(x=M(data=FAKE + 2)), WS, b"NULL"),
])
def test_linear_refuses(lib, kw, status, word):
    assert lib.dion3_linear(linear_args(**kw), None, 0, None) == status
    assert word in lib.dion3_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(tokens=-5), INV, b"rows"), (dict(act=9), INV, b"activation"), (dict(w=M(dtype=d3.F32)), UNS, b"fp32"),
    (dict(dw=M(dtype=5)), INV, b"dw"), (dict(x=L._Matrix()), INV, b"x is NULL"),
    (dict(x8=P()), INV, b"x and x8"), (dict(act=1), INV, b"z is NULL"), (dict(act=1, z=M(), z8=P()), INV, b"z and z8"),
    (dict(dx=M()), INV, b"dx may not be dy"), (dict(db=FAKE + 2), INV, b"db"), (dict(act=2, z=M()), WS, b"NULL"),
    (dict(x=L._Matrix(), x8=P(lds=1)), INV, b"x8"), (dict(dy=M(ld=60)), INV, b"dy"),
])
def test_linear_backward_refuses(lib, kw, status, word):
    assert lib.dion3_linear_backward(grad_args(**kw), None, 0, None) == status
    assert word in lib.dion3_last_error()


def test_workspace_checks(lib):
    a = grad_args(act=2, z=M())
    need = d3.linear_backward_workspace_size(4, 64, 64, dtype=torch.bfloat16)
    assert lib.dion3_linear_backward(a, FAKE, 64, None) == WS
    assert lib.dion3_linear_backward(a, FAKE + 16, need, None) == INV and b"256" in lib.dion3_last_error()
    assert lib.dion3_linear(None, None, 0, None) == INV and lib.dion3_linear_backward(None, None, 0, None) == INV
    out = ctypes.c_size_t(7)
    for fn in (lib.dion3_linear_workspace_size, lib.dion3_linear_backward_workspace_size):
        assert fn(4, 64, 64, d3.BF16, 0, None) == INV
        assert fn(4, 64, 0, d3.BF16, 0, ctypes.byref(out)) == INV
        assert fn(4, 64, 8, d3.F32, 0, ctypes.byref(out)) == UNS
    assert lib.dion3_rms_norm_backward_workspace_size(4, 1 << 20, ctypes.byref(out)) == UNS
    assert out.value == 7


def test_workspace_sizes(lib):
    bf = torch.bfloat16
    assert d3.linear_workspace_size(100, 64, 32, dtype=bf) == 0
    assert d3.linear_workspace_size(100, 65, 32, dtype=bf) >= 132 * 72 * 2
    assert d3.linear_workspace_size(100, 64, 32, dtype=bf, strided=True) >= 132 * 64 * 2
    assert d3.linear_workspace_size(0, 64, 32, dtype=bf) == 0
    big = d3.linear_backward_workspace_size(1 << 24, 4096, 4096, dtype=bf)  # past 32 bits
    assert big > 2 * (1 << 24) * 4096 * 2


@pytest.mark.parametrize("call,word", [
    (lambda l: l.dion3_pack8(2, 64, M(ld=32), P(), None), b"pitch"),
    (lambda l: l.dion3_pack8(2, 64, M(dtype=5), P(), None), b"dtype"),
    (lambda l: l.dion3_pack8(2, 64, M(), P(codes=None), None), b"NULL"),
    (lambda l: l.dion3_pack8(2, 64, None, P(), None), b"NULL"),
    (lambda l: l.dion3_unpack8(2, 64, P(lds=1), M(), None), b"pitches"),
    (lambda l: l.dion3_unpack8(-2, 64, P(), M(), None), b"rows"),
    (lambda l: l.dion3_rms_norm(2, 64, M(), None, None, d3.BF16, 1e-6, None, M(), None, None, None), b"weight"),
    (lambda l: l.dion3_rms_norm(2, 64, M(), None, FAKE, d3.BF16, 1e-6, None, None, None, None, None), b"neither"),
    (lambda l: l.dion3_rms_norm(2, 64, M(), None, FAKE, d3.BF16, -1.0, None, M(), None, None, None), b"eps"),
    (lambda l: l.dion3_rms_norm(2, 64, M(), None, FAKE, d3.BF16, float("nan"), None, M(), None, None, None), b"eps"),
    (lambda l: l.dion3_rms_norm(2, 64, M(), M(dtype=d3.F16), FAKE, d3.BF16, 0.0, None, M(), None, None, None), b"residual"),
    (lambda l: l.dion3_rms_norm(2, 64, M(), None, FAKE, d3.BF16, 0.0, None, M(), None, FAKE + 2, None), b"rstd"),
    (lambda l: l.dion3_rms_norm_backward(2, 64, M(), M(), FAKE, d3.BF16, None, None, M(), None, 0, None, 0, None), b"rstd"),
    (lambda l: l.dion3_rms_norm_backward(2, 64, M(), M(), FAKE, d3.BF16, FAKE, None, None, None, 0, None, 0, None), b"dx"),
    (lambda l: l.dion3_rms_norm_backward(2, 64, M(), M(dtype=d3.F32), FAKE, d3.BF16, FAKE, None, M(), None, 0, None, 0,
                                         None), b"h has dtype"),
])
def test_norm_and_blocks_refuse(lib, call, word):
    assert call(lib) == INV
    assert word in lib.dion3_last_error()


def test_norm_limits_and_workspace(lib):
    assert lib.dion3_rms_norm(2, 50000, M(ld=50000), None, FAKE, d3.BF16, 0.0, None, M(ld=50000), None, None, None) == UNS
    assert lib.dion3_rms_norm_backward(2, 64, M(), M(), FAKE, d3.BF16, FAKE, None, M(), FAKE, 0, None, 0, None) == WS


def test_injected_launch_failure(lib):
    os.environ["DION3_INJECT"] = "launch_fail"
    try:
        assert lib.dion3_linear(linear_args(), None, 0, None) == d3.ERR_CUDA
        assert lib.dion3_pack8(2, 64, M(), P(), None) == d3.ERR_CUDA
    finally:
        del os.environ["DION3_INJECT"]


def test_no_tokens_enqueue_nothing(lib):
    """Zero tokens pass with null bases and without a GPU (nothing is launched)."""
    none = L._Matrix(None, 64, d3.BF16)
    a = linear_args(tokens=0, x=none, y=none)
    assert lib.dion3_linear(a, None, 0, None) == d3.OK
    assert lib.dion3_pack8(0, 64, none, L._Packed8(), None) == d3.OK
    assert lib.dion3_linear_backward(grad_args(tokens=0, dy=none, x=none, accumulate=1), None, 0, None) == d3.OK


def test_binding_refuses_before_the_library():
    """CPU tensors, wrong shapes, types and layouts never reach the library."""
    z = torch.zeros
    cpu = z(4, 8)
    for call in (lambda: d3.pack8(cpu, None), lambda: d3.linear(cpu, cpu, cpu), lambda: d3.rms_norm(cpu, cpu[0], cpu),
                 lambda: d3.linear_backward(cpu, cpu, cpu, dx=cpu),
                 lambda: d3.Packed8(z(4, 8, dtype=torch.int8), z(4, 1, dtype=torch.uint8)),
                 lambda: d3.Packed8(cpu, cpu)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(d3.Dion3Error):
        d3.linear_workspace_size(4, 8, 8, dtype=torch.float64)


class Fake:
    """What the binding reads of a tensor, on no device."""
    is_cuda = True

    def __init__(self, shape, stride, dtype=torch.bfloat16):
        self.shape, self._s, self.dtype = shape, stride, dtype

    def stride(self, i=None):
        return self._s if i is None else self._s[i]

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return FAKE


def test_matrix_marshalling():
    assert L._mat("x", Fake((4, 8), (11, 1))) == (FAKE, 11, d3.BF16)
    assert L._mat("x", Fake((1, 8), (1, 1)))[1] == 8  # the stride of a single row says nothing
    assert L._mat("x", Fake((4, 1), (3, 9)))[1] == 3  # nor does that of a single column
    for bad in (Fake((4, 8), (1, 4)), Fake((4, 8), (4, 1)), Fake((4, 8), (0, 1)), Fake((8,), (1,)),
                Fake((4, 8), (8, 1), torch.int32)):
        with pytest.raises(ValueError):
            L._mat("x", bad)
    with pytest.raises(ValueError):
        L._mat("x", Fake((4, 8), (8, 1)), 4, 9)
    with pytest.raises(ValueError):
        L._vec("w", Fake((8,), (2,)), 8)
    with pytest.raises(ValueError):
        L._vec("w", Fake((8,), (1,)), 8, f32=True)
