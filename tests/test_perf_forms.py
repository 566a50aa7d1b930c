"""The plain forms of perf/more_operators.py: a pass leaves its inputs as they were, so
that every pass on one state gives the same bits, and agrees with the 64-bit form.  They
run on the CPU: whatever asks for "cuda" gets it there."""
import importlib.util
import math
import os
import random

import pytest
import torch
from torch.overrides import TorchFunctionMode

from _layer_ref import TINY, U

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")


class OnCpu(TorchFunctionMode):
    def __torch_function__(self, func, types, args=(), kwargs=None):
        kwargs = dict(kwargs or {})
        if kwargs.get("device") == "cuda":
            kwargs["device"] = "cpu"
        return func(*args, **kwargs)


@pytest.fixture
def forms(monkeypatch):
    spec = importlib.util.spec_from_file_location("more_operators", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    real = torch.Generator
    monkeypatch.setattr(torch, "Generator", lambda device="cpu": real())
    with OnCpu():
        yield m


def tensors(v, name=""):
    """Every tensor of a state, a result or a list in one, by its place."""
    if isinstance(v, torch.Tensor):
        return {name: v}
    items = v.items() if isinstance(v, dict) else enumerate(v) if isinstance(v, (list, tuple)) else ()
    return {k: t for i, e in items for k, t in tensors(e, f"{name}/{i}").items()}


def cases():
    """One case of every operator, element type and choice."""
    for dtype in ("f32", "bf16", "f16"):
        for table in ("f32", dtype):
            for op in ("embed", "embed_grad"):
                yield dict(op=op, table=table, dtype=dtype, tokens=90, vocab=1000, cols=65, scale=64.0)
        for op in ("scan", "scan_grad"):
            for sequences in (1, 20, 70):
                for states in (True, False):
                    yield dict(op=op, dtype=dtype, tokens=70, channels=65, sequences=sequences, states=states)
        for entropy in (True, False):
            c = dict(dtype=dtype, tokens=9, vocab=1001, entropy=entropy, scale=1.25, masked=entropy)
            yield dict(c, op="logp", top=5 if entropy else 0)
            yield dict(c, op="logp_grad")
        yield dict(op="clip", dtype=dtype, layers=1, d=64, ffn=70)


@pytest.mark.parametrize("case", list(cases()), ids=lambda c: "-".join(str(v) for v in c.values()))
def test_passes_on_one_state_agree(forms, case):
    state = forms.prepare(case, 5)
    before = {k: t.clone() for k, t in tensors(state).items()}
    first = {k: t.clone() for k, t in tensors(forms.run(state)).items()}
    for _ in range(2):
        again = tensors(forms.run(state))
        assert all(torch.equal(again[k], t) for k, t in first.items())
    assert all(torch.equal(t, before[k]) for k, t in tensors(state).items())
    # A result is rounded once (u) after 32-bit steps: seven doublings of a scan or a sum of
    # at most 1001 terms in lanes and pairs (20 deep), and gates or exponentials of some
    # units each, are within 64 units of 2^-24 of what the terms' sizes add up to, 2^-18.
    for k, want in tensors(forms.exact(case, 5)).items():
        got, want = first[k], want.double()
        kind = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[got.dtype]
        there = torch.isfinite(want)
        assert torch.equal(there, torch.isfinite(got)), k
        off, size = float((got.double() - want)[there].norm()), float(want[there].norm())
        assert off <= (1.001 * U[kind] + 2.0 ** -18) * size + TINY[kind] * math.sqrt(got.numel()), k


def test_drawn_cases_are_of_the_operators(forms):
    rng = random.Random(3)
    ops = {c["op"] for c in forms.listed()}
    assert {forms.draw(rng)["op"] for _ in range(200)} == ops
