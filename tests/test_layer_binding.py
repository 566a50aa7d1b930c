"""What the binding of the layer operators hands to the library: the addresses
and strides that the tensors have when a call is made.  No GPU work."""
import struct

import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from matrix_orthogonalizing_optimizer_shape_gb300 import layer as L


class Fake:
    """What the binding reads of a tensor, on no device."""
    is_cuda = True

    def __init__(self, shape, dtype, address, pitch=None, device=0):
        self.shape, self.dtype, self.address, self.device = torch.Size(shape), dtype, address, device
        self.pitch = shape[-1] if pitch is None else pitch

    def stride(self, i=None):
        s = (self.pitch, 1) if len(self.shape) == 2 else (1,)
        return s if i is None else s[i]

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return self.address

    def get_device(self):
        return self.device

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 4


@pytest.fixture
def calls(monkeypatch):
    """The arguments of the library's calls, which are not made."""
    made = []
    monkeypatch.setattr(L, "_fn", lambda name: lambda *a: made.append((name, a)) or 0)
    monkeypatch.setattr(L, "_device", lambda: 0, raising=False)
    L._load_torch()
    return made


def blocks(codes, scales):
    return d3.Packed8(Fake((4, 40), torch.int8, codes, 48), Fake((4, 2), torch.uint8, scales, 16))


def fields(data):
    return struct.unpack("@PqPq", data)


def test_blocks_follow_their_attributes(calls):
    p, out = blocks(0x1000, 0x2000), Fake((4, 40), torch.bfloat16, 0x8000)
    d3.unpack8(p, out, stream=1)
    p.codes, p.scales = Fake((4, 40), torch.int8, 0x3000, 64), Fake((4, 2), torch.uint8, 0x4000, 2)
    d3.unpack8(p, out, stream=1)
    p.codes.address = 0x5000  # the same tensor object with other storage
    d3.pack8(out, p, stream=1)
    d3.rms_norm(out, Fake((40,), torch.float32, 0x9000), y8=p, stream=1)
    assert [fields(a[2]) for _, a in calls[:2]] == [(0x1000, 48, 0x2000, 16), (0x3000, 64, 0x4000, 2)]
    assert fields(calls[2][1][3]) == (0x5000, 64, 0x4000, 2)
    assert fields(calls[3][1][9]) == (0x5000, 64, 0x4000, 2)


def test_blocks_follow_their_attributes_in_the_linear_layer(calls):
    x, w, y = Fake((4, 8), torch.bfloat16, 0x10), Fake((40, 8), torch.bfloat16, 0x20), Fake((4, 40), torch.bfloat16, 0x30)
    p = blocks(0x1000, 0x2000)
    p.codes, p.scales = Fake((4, 40), torch.int8, 0x3000, 64), Fake((4, 2), torch.uint8, 0x4000, 2)
    d3.linear(x, w, y, z=p, y8=p, stream=1)
    d3.linear_backward(y, x, w, dx=Fake((4, 8), torch.bfloat16, 0x40), act=d3.ACT_RELU, z=p, stream=1)
    d3.linear_backward(x, p, Fake((8, 40), torch.bfloat16, 0x50), dw=Fake((8, 40), torch.float32, 0x60), stream=1)
    got = L._LINEAR.unpack(calls[0][1][0])
    assert got[19:27] == (0x3000, 64, 0x4000, 2) * 2
    got = L._LINEAR_GRAD.unpack(calls[1][1][0])
    assert got[17:25] == (0, 0, 0, 0, 0x3000, 64, 0x4000, 2)
    got = L._LINEAR_GRAD.unpack(calls[2][1][0])
    assert got[17:25] == (0x3000, 64, 0x4000, 2, 0, 0, 0, 0)


@pytest.mark.parametrize("codes,scales", [
    (Fake((4, 40), torch.uint8, 1), None), (Fake((4, 41), torch.int8, 1), None), (Fake((4, 40), torch.int8, 1, 8), None),
    (Fake((160,), torch.int8, 1), None), (None, Fake((4, 3), torch.uint8, 1)), (None, Fake((4, 2), torch.int8, 1)),
    (None, Fake((3, 2), torch.uint8, 1))])
def test_replaced_blocks_are_checked(calls, codes, scales):
    p = blocks(0x1000, 0x2000)
    p.codes, p.scales = codes or p.codes, scales or p.scales
    with pytest.raises(ValueError):
        d3.unpack8(p, Fake((4, 40), torch.bfloat16, 0x8000), stream=1)
    assert not calls


def all_calls():
    """Every entry point with every tensor that it takes, as (call, names of the tensors)."""
    bf, f32 = torch.bfloat16, torch.float32

    def mat(rows, cols, dtype=bf):
        return lambda d: Fake((rows, cols), dtype, 0x100, device=d)

    def vec(n):
        return lambda d: Fake((n,), f32, 0x100, device=d)

    def pack(rows, cols):
        def make(d):
            return d3.Packed8(Fake((rows, cols), torch.int8, 0x100, device=d),
                              Fake((rows, -(-cols // 32)), torch.uint8, 0x100, device=d))
        return make
    big = vec(1 << 20)
    return [(d3.pack8, dict(x=mat(4, 40), out=pack(4, 40))), (d3.unpack8, dict(src=pack(4, 40), out=mat(4, 40))),
            (d3.rms_norm, dict(x=mat(4, 40), weight=vec(40), y=mat(4, 40), residual=mat(4, 40), h=mat(4, 40),
                               y8=pack(4, 40), rstd=vec(4))),
            (d3.rms_norm_backward, dict(dy=mat(4, 40), h=mat(4, 40), weight=vec(40), rstd=vec(4), dx=mat(4, 40),
                                        dh=mat(4, 40), dw=vec(40), ws=big)),
            (d3.linear, dict(x=mat(4, 8), w=mat(40, 8), y=mat(4, 40), bias=vec(40), residual=mat(4, 40), z=mat(4, 40),
                             y8=pack(4, 40), ws=big)),
            (d3.linear, dict(x=mat(4, 8), w=mat(40, 8), y=mat(4, 40), z=pack(4, 40))),
            (d3.linear_backward, dict(dy=mat(4, 40), x=mat(4, 8), w=mat(40, 8), dx=mat(4, 8), dw=mat(40, 8, f32),
                                      db=vec(40), z=mat(4, 40), ws=big)),
            (d3.linear_backward, dict(dy=mat(4, 40), x=pack(4, 8), w=mat(40, 8), dw=mat(40, 8, f32), z=pack(4, 40)))]


@pytest.mark.parametrize("case", range(8))
def test_tensors_on_another_device_are_refused(calls, monkeypatch, case):
    call, tensors = all_calls()[case]
    for stream in (None, 1):
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1, raising=False)
        call(**{k: t(0) for k, t in tensors.items()}, stream=stream)
        assert len(calls) == 1
        calls.clear()
        for other in tensors:  # one of them is on the other device, and all are while the first is current
            with pytest.raises(ValueError, match="device|cuda:1"):
                call(**{k: t(int(k == other)) for k, t in tensors.items()}, stream=stream)
        with pytest.raises(ValueError, match="cuda:1"):
            call(**{k: t(1) for k, t in tensors.items()}, stream=stream)
        assert not calls


def test_blocks_on_two_devices_are_refused(calls):
    with pytest.raises(ValueError, match="device"):
        d3.Packed8(Fake((4, 40), torch.int8, 1), Fake((4, 2), torch.uint8, 1, device=1))


@pytest.mark.gpu
def test_blocks_moved_to_the_host_and_back(cuda_lib):
    x = torch.randn(70, 100, device="cuda")
    p, out = d3.alloc_packed8(70, 100), torch.empty(70, 100, device="cuda")
    d3.pack8(x, p)
    want = torch.empty_like(out)
    d3.unpack8(p, want)
    old, kept = (p.codes, p.scales), (p.codes.cpu(), p.scales.cpu())
    p.codes, p.scales = (t.cuda() for t in kept)
    old[0].zero_(), old[1].zero_()
    d3.unpack8(p, out)
    assert torch.equal(out, want)
    d3.pack8(2 * x, p)
    assert bool((old[0] == 0).all()) and torch.equal(p.scales.cpu(), kept[1] + 1)
