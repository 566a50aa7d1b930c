"""Host-side checks of the model operators: sizes, refusals and their messages, and
what the binding hands to the library.  No call here launches GPU work."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from matrix_orthogonalizing_optimizer_shape_gb300 import layer as L
from matrix_orthogonalizing_optimizer_shape_gb300 import model as G
from test_layer_args import FAKE, M, lib  # noqa: F401

INV, UNS, WS = d3.ERR_INVALID_ARG, d3.ERR_UNSUPPORTED, d3.ERR_WORKSPACE
A, B, C, D, E = (FAKE + (i << 20) for i in range(1, 6))
NAN, INF = float("nan"), float("inf")


def ref(m):
    return None if m is None else ctypes.byref(m)


def embedding(lib, **kw):  # noqa: F811
    a = dict(tokens=4, vocab=9, cols=64, ids=FAKE, id_bytes=8, table=M(data=A), scale=1.0, y=M(data=B))
    a.update(kw)
    a["table"], a["y"] = ref(a["table"]), ref(a["y"])
    return lib.dion3_embedding(*a.values(), None)


def embedding_backward(lib, **kw):  # noqa: F811
    a = dict(tokens=4, vocab=9, cols=64, dy=M(data=A), ids=FAKE, id_bytes=8, scale=1.0, dtable=M(data=B), accumulate=0,
             ws=C, ws_bytes=1 << 20)
    a.update(kw)
    a["dy"], a["dtable"] = ref(a["dy"]), ref(a["dtable"])
    return lib.dion3_embedding_backward(*a.values(), None)


def recurrence(lib, **kw):  # noqa: F811
    a = dict(tokens=4, channels=64, z=M(data=A), x=M(data=B), offsets=FAKE, sequences=2, first=None, h=M(data=C), last=None)
    a.update(kw)
    for k in "zxh":
        a[k] = ref(a[k])
    return lib.dion3_recurrence(*a.values(), None)


def recurrence_backward(lib, **kw):  # noqa: F811
    a = dict(tokens=4, channels=64, dh=M(data=A), z=M(data=B), x=M(data=C), h=M(data=D), offsets=FAKE, sequences=2,
             first=None, dlast=None, dz=M(data=E), dx=M(data=E + 65536), dfirst=None)
    a.update(kw)
    for k in ("dh", "z", "x", "h", "dz", "dx"):
        a[k] = ref(a[k])
    return lib.dion3_recurrence_backward(*a.values(), None)


def log_probs(lib, **kw):  # noqa: F811
    a = dict(rows=4, vocab=64, logits=M(data=A), scale=1.0, targets=FAKE, target_bytes=8, logp=B, entropy=None, stats=None,
             top=0, top_values=None, top_ids=None)
    a.update(kw)
    a["logits"] = ref(a["logits"])
    return lib.dion3_log_probs(*a.values(), None)


def log_probs_backward(lib, **kw):  # noqa: F811
    a = dict(rows=4, vocab=64, logits=M(data=A), scale=1.0, targets=FAKE, target_bytes=8, stats=B, dlogp=C, dentropy=None,
             dlogits=M(data=D))
    a.update(kw)
    a["logits"], a["dlogits"] = ref(a["logits"]), ref(a["dlogits"])
    return lib.dion3_log_probs_backward(*a.values(), None)


def T(data=A, rows=1, cols=64, ld=64, dtype=d3.BF16):
    return struct.pack("@" + G._TENSOR, data, rows, cols, ld, dtype)


def clip(lib, ts=(T(),), out=None, max_norm=1.0, norm=B, ws=C, ws_bytes=1 << 20, n=None):  # noqa: F811
    join = lambda v: None if v is None else b"".join(v)  # noqa: E731
    return lib.dion3_clip_grad_norm(join(ts), join(out), len(ts or ()) if n is None else n, max_norm, norm, ws, ws_bytes,
                                    None)


@pytest.mark.parametrize("call,kw,status,word", [
    (embedding, dict(tokens=-1), INV, b"rows"), (embedding, dict(cols=0), INV, b"cols"),
    (embedding, dict(cols=1 << 21), UNS, b"larger"), (embedding, dict(vocab=-1), INV, b"rows"),
    (embedding, dict(id_bytes=2), INV, b"4 or 8"), (embedding, dict(ids=None), INV, b"ids is NULL"),
    (embedding, dict(ids=FAKE + 4), INV, b"ids is not aligned"), (embedding, dict(table=None), INV, b"table is NULL"),
    (embedding, dict(table=M(dtype=7)), INV, b"dtype"), (embedding, dict(y=M(data=None)), INV, b"y is NULL"),
    (embedding, dict(y=M(ld=63)), INV, b"pitch"), (embedding, dict(y=M(data=A)), INV, b"y may not be table"),
    (embedding, dict(scale=NAN), INV, b"scale"), (embedding, dict(scale=INF), INV, b"scale"),
    (embedding_backward, dict(tokens=-1), INV, b"rows"), (embedding_backward, dict(tokens=1 << 28), UNS, b"tokens"),
    (embedding_backward, dict(vocab=(1 << 24) + 1), UNS, b"vocabulary"),
    (embedding_backward, dict(dy=M(data=B)), INV, b"dtable may not be dy"),
    (embedding_backward, dict(dtable=M(data=B + 1)), INV, b"aligned"), (embedding_backward, dict(dy=None), INV, b"dy"),
    (embedding_backward, dict(ws=None), WS, b"NULL"), (embedding_backward, dict(ws_bytes=64), WS, b"small"),
    (embedding_backward, dict(ws=C + 8), INV, b"256"), (embedding_backward, dict(scale=NAN), INV, b"scale"),
    (recurrence, dict(tokens=-1), INV, b"rows"), (recurrence, dict(channels=1 << 20, z=M(ld=1 << 20)), UNS, b"larger"),
    (recurrence, dict(sequences=-1), INV, b"sequences"), (recurrence, dict(sequences=1 << 28), UNS, b"sequences"),
    (recurrence, dict(offsets=None), INV, b"offsets is NULL"), (recurrence, dict(offsets=FAKE + 2), INV, b"offsets"),
    (recurrence, dict(x=M(dtype=d3.F16)), INV, b"x has dtype"), (recurrence, dict(h=None), INV, b"h is NULL"),
    (recurrence, dict(z=M(dtype=3)), INV, b"dtype"), (recurrence, dict(first=FAKE + 2), INV, b"first"),
    (recurrence, dict(last=FAKE + 1), INV, b"last"), (recurrence, dict(h=M(data=A, ld=80)), INV, b"needs its pitch"),
    (recurrence_backward, dict(tokens=-1), INV, b"rows"), (recurrence_backward, dict(h=None), INV, b"h is NULL"),
    (recurrence_backward, dict(dz=M(data=D)), INV, b"may not be h"), (recurrence_backward, dict(dx=M(data=D)), INV, b"may not be h"),
    (recurrence_backward, dict(dx=M(data=E)), INV, b"one another"), (recurrence_backward, dict(dz=M(data=A, ld=66)), INV, b"pitch"),
    (recurrence_backward, dict(first=E, dfirst=E), INV, b"dfirst may not be first"),
    (recurrence_backward, dict(dlast=FAKE + 2), INV, b"dlast"), (recurrence_backward, dict(sequences=0, offsets=None), INV, b"offsets"),
    (log_probs, dict(rows=-1), INV, b"rows"), (log_probs, dict(rows=1 << 22), UNS, b"rows"),
    (log_probs, dict(vocab=1 << 22, logits=M(ld=1 << 22)), UNS, b"larger"), (log_probs, dict(vocab=0), INV, b"cols"),
    (log_probs, dict(scale=0.0), INV, b"scale"), (log_probs, dict(scale=-1.0), INV, b"scale"),
    (log_probs, dict(scale=NAN), INV, b"scale"), (log_probs, dict(scale=INF), INV, b"scale"),
    (log_probs, dict(targets=None), INV, b"without targets"), (log_probs, dict(target_bytes=1), INV, b"4 or 8"),
    (log_probs, dict(targets=FAKE + 4), INV, b"aligned"), (log_probs, dict(logp=FAKE + 2), INV, b"logp"),
    (log_probs, dict(top=33), INV, b"top"), (log_probs, dict(top=-1), INV, b"top"),
    (log_probs, dict(vocab=5, top=6), INV, b"top"), (log_probs, dict(top_ids=FAKE + 2), INV, b"top_ids"),
    (log_probs, dict(logits=None), INV, b"logits"), (log_probs, dict(stats=FAKE + 3), INV, b"stats"),
    (log_probs_backward, dict(stats=None), INV, b"stats is NULL"), (log_probs_backward, dict(targets=None), INV, b"without targets"),
    (log_probs_backward, dict(dlogits=M(data=D, dtype=d3.F32)), INV, b"dlogits has dtype"),
    (log_probs_backward, dict(dlogits=M(data=A, ld=65)), INV, b"needs its pitch"),
    (log_probs_backward, dict(scale=0.0), INV, b"scale"), (log_probs_backward, dict(dentropy=FAKE + 1), INV, b"dentropy"),
    (clip, dict(n=-1), INV, b"n must"), (clip, dict(ts=None, n=2), INV, b"tensors is NULL"),
    (clip, dict(max_norm=-1.0), INV, b"max_norm"), (clip, dict(max_norm=NAN), INV, b"max_norm"),
    (clip, dict(norm=B + 2), INV, b"norm"), (clip, dict(ws=None), WS, b"NULL"), (clip, dict(ws_bytes=100), WS, b"small"),
    (clip, dict(ts=(T(dtype=4),)), INV, b"tensors[0]: unknown dtype"), (clip, dict(ts=(T(), T(data=0))), INV, b"tensors[1] is NULL"),
    (clip, dict(ts=(T(rows=3, ld=63),)), INV, b"pitch"), (clip, dict(ts=(T(data=A + 1),)), INV, b"aligned"),
    (clip, dict(ts=(T(rows=-1),)), INV, b"negative"), (clip, dict(ts=(T(rows=1 << 31),)), UNS, b"larger"),
    (clip, dict(out=(T(data=D, cols=63),)), INV, b"not of the size"), (clip, dict(out=(T(data=D, dtype=9),)), INV, b"out[0]"),
    (clip, dict(ts=(T(), T())), INV, b"tensors 0 and 1 share"), (clip, dict(ts=(T(), T(data=A + 126))), INV, b"share"),
    (clip, dict(ts=(T(),), out=(T(data=A + 2),)), INV, b"share"),
    (clip, dict(ts=(T(), T(data=B)), out=(T(data=B), T(data=D))), INV, b"share"),
    (clip, dict(ts=(T(),), out=(T(dtype=d3.F32),)), INV, b"share"),
    (clip, dict(ts=(T(rows=9, cols=32, ld=96), T(data=A + 62, rows=9, cols=32, ld=96))), INV, b"share"),
    (clip, dict(ts=(T(rows=9, cols=32, ld=96), T(data=A + 64, rows=9, cols=32, ld=98))), INV, b"share"),
])
def test_refusals(lib, call, kw, status, word):  # noqa: F811
    assert call(lib, **kw) == status, lib.dion3_last_error()
    assert word in lib.dion3_last_error()


def test_valid_calls_reach_the_launch(lib, monkeypatch):  # noqa: F811
    """What the checks let pass, up to an injected launch failure."""
    monkeypatch.setenv("DION3_INJECT", "launch_fail")
    cols = lambda i, n=32: T(data=A + 2 * i, rows=9, cols=n, ld=96)  # noqa: E731
    for call, kw in (
            (embedding, {}), (embedding, dict(vocab=0, table=M(data=None))), (embedding, dict(y=M(data=B, dtype=d3.F32))),
            (embedding_backward, {}), (embedding_backward, dict(tokens=0, dy=M(data=None), ids=None, ws=None, ws_bytes=0)),
            (recurrence, {}), (recurrence, dict(offsets=None, sequences=1)), (recurrence, dict(h=M(data=A))),
            (recurrence, dict(h=M(data=B), first=D, last=D)),
            (recurrence_backward, {}), (recurrence_backward, dict(dz=M(data=B), dx=M(data=A))),
            (recurrence_backward, dict(dlast=FAKE, dfirst=FAKE)),
            (log_probs, {}), (log_probs, dict(targets=None, logp=None)), (log_probs, dict(top=32, top_ids=D)),
            (log_probs_backward, {}), (log_probs_backward, dict(dlogits=M(data=A))),
            (log_probs_backward, dict(targets=None, dlogp=None)),
            (clip, {}), (clip, dict(ts=())), (clip, dict(max_norm=INF)), (clip, dict(norm=None)), (clip, dict(out=(T(),))),
            (clip, dict(ts=(T(), T(data=A + 128)))), (clip, dict(ts=(cols(64), cols(0), cols(32)))),
            (clip, dict(ts=(T(rows=0, data=0), T()))), (clip, dict(out=(T(data=A + 128),)))):
        assert call(lib, **kw) == d3.ERR_CUDA and b"injected" in lib.dion3_last_error(), (call, kw, lib.dion3_last_error())


def test_nothing_to_do(lib):  # noqa: F811
    """Calls without work pass with null bases and without a GPU."""
    none = M(data=None)
    assert embedding(lib, tokens=0, y=none, ids=None) == d3.OK
    assert embedding_backward(lib, tokens=0, dy=none, ids=None, ws=None, ws_bytes=0, accumulate=1) == d3.OK
    assert embedding_backward(lib, vocab=0, dtable=none) == d3.OK
    assert recurrence(lib, tokens=0, z=none, x=none, h=none) == d3.OK
    assert recurrence(lib, sequences=0) == d3.OK
    assert recurrence_backward(lib, tokens=0, dh=none, z=none, x=none, h=none, dz=none, dx=none) == d3.OK
    assert log_probs(lib, rows=0, logits=none, targets=None) == d3.OK
    assert log_probs_backward(lib, rows=0, logits=none, stats=None, dlogits=none) == d3.OK


def test_workspace_sizes(lib):  # noqa: F811
    assert d3.embedding_backward_workspace_size(0, 10, 8) == 0
    n = d3.embedding_backward_workspace_size(1 << 26, 1000, 4096)  # past 32 bits
    assert n > 8 * (1 << 26) + 2 * (1 << 17) * 4096 * 4
    assert 0 < d3.grad_norm_workspace_size() <= 65536
    assert lib.dion3_embedding_backward_workspace_size(4, 9, 8, None) == INV
    assert lib.dion3_grad_norm_workspace_size(None) == INV
    assert lib.dion3_grad_norm(T(), 1, None, C, 1 << 20, None) == INV and b"norm is NULL" in lib.dion3_last_error()


def test_binding_refuses_before_the_library():
    """CPU tensors, wrong shapes and types never reach the library."""
    z, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    v = torch.zeros(4)
    for call in (lambda: d3.embedding(i, z, z), lambda: d3.embedding_backward(z, i, z), lambda: d3.recurrence(z, z, z),
                 lambda: d3.recurrence_backward(z, z, z, z, z, z), lambda: d3.log_probs(z, i, v),
                 lambda: d3.log_probs_backward(z, i, v, z), lambda: d3.grad_norm([z], v[:1]),
                 lambda: d3.clip_grad_norm([z], 1.0), lambda: d3.clip_grad_norm([z], 1.0, out=[])):
        with pytest.raises(ValueError):
            call()


class Fake:
    """What the binding reads of a tensor, on no device."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.bfloat16, stride=None, device=0, address=FAKE):
        self.shape, self.dtype, self.device, self.address = torch.Size(shape), dtype, device, address
        self._s = stride or tuple(int(torch.Size(shape[i + 1:]).numel()) for i in range(len(shape)))

    def stride(self):
        return self._s

    def is_contiguous(self):
        return self._s == tuple(int(self.shape[i + 1:].numel()) for i in range(len(self.shape)))

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 4

    def data_ptr(self):
        return self.address

    def get_device(self):
        return self.device


@pytest.fixture
def calls(monkeypatch):
    """The arguments of the library's calls, which are not made."""
    made = []
    monkeypatch.setattr(L, "_fn", lambda name: lambda *a: made.append((name, a)) or 0)
    monkeypatch.setattr(L, "_device", lambda: 0)
    L._load_torch()
    return made


def test_binding_marshals_what_tensors_have(calls):
    f32, i32, i64 = torch.float32, torch.int32, torch.int64
    z, off, s = Fake((6, 8), stride=(24, 1)), Fake((3,), i32, address=A), Fake((2, 8), f32, address=B)
    d3.recurrence(z, z, z, offsets=off, first=s, last=s, stream=1)
    assert calls[-1][1][:2] == (6, 8) and calls[-1][1][4:7] == (A, 2, B) and calls[-1][1][8] == B
    d3.recurrence(z, z, z, stream=1)
    assert calls[-1][1][4:7] == (None, 1, None)
    d3.log_probs(Fake((6, 50)), Fake((6,), i64), Fake((6,), f32), top_ids=Fake((6, 4), i32, address=C), stream=1)
    assert calls[-1][1][5] == 8 and calls[-1][1][9:12] == (4, None, C)
    d3.embedding(Fake((6,), i32), Fake((9, 8)), Fake((6, 8)), scale=2.0, stream=1)
    assert calls[-1][1][:5] == (6, 9, 8, FAKE, 4)
    d3.clip_grad_norm([Fake((2, 3, 4)), Fake((5, 6), f32, (7, 1), address=A), Fake(())], 1.0, Fake((), f32), stream=1)
    got = struct.unpack("@" + G._TENSOR * 3, calls[-1][1][0])
    assert got == (FAKE, 1, 24, 24, d3.BF16, A, 5, 6, 7, d3.F32, FAKE, 1, 1, 1, d3.BF16) and calls[-1][1][1] is None
    d3.clip_grad_norm([Fake((5, 6), f32, (7, 1), address=A), Fake((4,))], 1.0, out=[Fake((5, 6)), Fake((4,), address=B)], stream=1)
    assert struct.unpack("@" + G._TENSOR * 2, calls[-1][1][0]) == (A, 5, 6, 7, d3.F32, FAKE, 1, 4, 4, d3.BF16)
    assert struct.unpack("@" + G._TENSOR * 2, calls[-1][1][1]) == (FAKE, 5, 6, 6, d3.BF16, B, 1, 4, 4, d3.BF16)


def test_binding_refuses_layouts_types_and_other_devices(calls):
    f32, i32, i64 = torch.float32, torch.int32, torch.int64
    z, t = Fake((6, 8)), Fake((6,), i64)
    for call in (
            lambda: d3.embedding(Fake((6,), torch.int16), z, z), lambda: d3.embedding(Fake((5,), i64), z, z),
            lambda: d3.embedding(Fake((6,), i64, (2,)), z, z), lambda: d3.embedding(t, Fake((9, 7)), z),
            lambda: d3.embedding(Fake((6,), i64, device=1), z, z), lambda: d3.embedding(t, Fake((9, 8), device=1), z),
            lambda: d3.recurrence(z, z, z, offsets=Fake((3,), i64)), lambda: d3.recurrence(z, z, z, offsets=Fake((0,), i32)),
            lambda: d3.recurrence(z, z, z, first=Fake((1, 8))), lambda: d3.recurrence(z, z, z, first=Fake((2, 8), f32)),
            lambda: d3.recurrence(z, z, z, offsets=Fake((3,), i32), last=Fake((2, 8), f32, (9, 1))),
            lambda: d3.recurrence(z, Fake((6, 8), stride=(1, 6)), z), lambda: d3.recurrence(z, z, Fake((6, 8), device=2)),
            lambda: d3.log_probs(z, t, Fake((6,))), lambda: d3.log_probs(z, t, Fake((6, 1), f32)),
            lambda: d3.log_probs(z, top_ids=Fake((6, 4), i64)), lambda: d3.log_probs(z, stats=Fake((6, 2), f32)),
            lambda: d3.log_probs(z, top_ids=Fake((6, 4), i32), top_values=Fake((6, 3), f32)),
            lambda: d3.log_probs_backward(z, t, Fake((6, 3), f32), Fake((6, 9))),
            lambda: d3.clip_grad_norm([z, Fake((3,), i32)], 1.0), lambda: d3.clip_grad_norm([z, Fake((3,), device=1)], 1.0),
            lambda: d3.clip_grad_norm([Fake((2, 3, 4), stride=(24, 4, 1))], 1.0),
            lambda: d3.clip_grad_norm([z], 1.0, out=[Fake((8, 6))]), lambda: d3.clip_grad_norm([z], 1.0, Fake((2,), f32)),
            lambda: d3.grad_norm([z], Fake((1,)))):
        with pytest.raises(ValueError):
            call()
    assert not calls




def test_clipping_refuses_strided_tensors_without_a_device(calls):
    """Rows of a CPU matrix into rows of another: dense ones are refused on another way."""
    class Host(Fake):
        is_cuda = False

    t, o = Host((5, 6), stride=(7, 1), device=-1), Host((5, 6), stride=(9, 1), device=-1, address=A)
    for out in (None, [o], [Fake((5, 6))]):
        with pytest.raises(ValueError, match="not a CUDA tensor"):
            d3.clip_grad_norm([t], 1.0, out=out, stream=1)
    with pytest.raises(ValueError):
        d3.clip_grad_norm([Fake((5, 6), stride=(7, 1))], 1.0, out=[o], stream=1)
    assert not calls


def test_rows_and_columns_of_one_matrix_are_apart(lib, monkeypatch):  # noqa: F811
    """Against the sets of elements: matrices of one base pitch, its multiples and single rows."""
    monkeypatch.setenv("DION3_INJECT", "launch_fail")
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(4000):
        ts, sets = [], []
        for _ in range(2):
            rows, cols, start = int(rng.integers(1, 5)), int(rng.integers(1, 8)), int(rng.integers(0, 40))
            ld = 8 * int(rng.integers(1, 4))
            ts.append(T(data=A + 2 * start, rows=rows, cols=cols, ld=ld))
            sets.append({start + r * ld + c for r in range(rows) for c in range(cols)})
        status, meet = clip(lib, ts=tuple(ts)), bool(sets[0] & sets[1])
        if meet:
            assert status == INV and b"share" in lib.dion3_last_error(), (ts, sets)
        seen.add((meet, status))
    assert seen == {(True, INV), (False, d3.ERR_CUDA), (False, INV)}  # (wrapping around a pitch may be refused)
    view = lambda i, rows, cols, ld: T(data=A + 2 * i, rows=rows, cols=cols, ld=ld)  # noqa: E731
    for ts in ((view(0, 9, 32, 96), view(4 * 96 + 32, 1, 64, 64)),    # columns, and a single row of the others
               (view(0, 5, 96, 192), view(96, 5, 96, 192)),           # every other row
               (view(0, 5, 32, 192), view(32, 9, 64, 96)),            # every other row of some columns, all of others
               (view(32, 1, 64, 64), view(0, 9, 32, 96))):
        assert clip(lib, ts=ts) == d3.ERR_CUDA, lib.dion3_last_error()
