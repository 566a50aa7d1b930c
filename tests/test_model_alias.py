"""Which arguments of the model operators may share memory.  No GPU work: where the
checks pass, an injected launch failure ends the call."""
import numpy as np
import pytest

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from test_layer_args import FAKE, M, lib  # noqa: F401
from test_model_args import (A, B, C, D, E, INV, embedding, embedding_backward, log_probs, log_probs_backward, recurrence,
                             recurrence_backward)


@pytest.fixture
def status(lib, monkeypatch):  # noqa: F811
    """What a call answers: "passes", or the two arguments that it refuses."""
    monkeypatch.setenv("DION3_INJECT", "launch_fail")

    def of(call, **kw):
        got, text = call(lib, **kw), lib.dion3_last_error().decode()
        if got == d3.ERR_CUDA and "injected" in text:
            return "passes"
        assert got == INV, text
        return text

    return of


@pytest.mark.parametrize("call,kw,names", [
    # One row behind, one element behind, a part of the rows.
    (recurrence, dict(h=M(data=A + 128)), "z and h"), (recurrence, dict(h=M(data=B - 2)), "x and h"),
    (recurrence, dict(h=M(data=A + 3 * 128)), "z and h"), (recurrence, dict(first=D, last=D + 4), "first and last"),
    (recurrence, dict(first=A + 500, last=C + 256), "h and last"), (recurrence, dict(last=A), "z and last"),
    (recurrence, dict(first=C), "first and h"),
    (recurrence_backward, dict(dx=M(data=E + 2)), "dz and dx"), (recurrence_backward, dict(dz=M(data=D + 128)), "h and dz"),
    (recurrence_backward, dict(dz=M(data=A + 128)), "dh and dz"), (recurrence_backward, dict(dx=M(data=B - 126)), "z and dx"),
    (recurrence_backward, dict(dx=M(data=C + 256)), "x and dx"), (recurrence_backward, dict(dfirst=E), "dz and dfirst"),
    (recurrence_backward, dict(first=FAKE, dfirst=FAKE + 256), "first and dfirst"),
    (recurrence_backward, dict(dlast=FAKE, dfirst=FAKE + 256), "dlast and dfirst"),
    (recurrence_backward, dict(first=E), "first and dz"),
    (log_probs_backward, dict(dlogits=M(data=A + 128)), "logits and dlogits"),
    (log_probs_backward, dict(dlogits=M(data=A - 4)), "logits and dlogits"),
    (log_probs_backward, dict(stats=D), "stats and dlogits"), (log_probs_backward, dict(dlogp=D + 8), "dlogp and dlogits"),
    (log_probs_backward, dict(dentropy=D), "dentropy and dlogits"), (log_probs_backward, dict(targets=D), "targets and dlogits"),
    (log_probs, dict(stats=A), "logits and stats"), (log_probs, dict(logp=A + 508), "logits and logp"),
    (log_probs, dict(entropy=B), "logp and entropy"), (log_probs, dict(top=2, top_values=C, top_ids=C + 28), "top_values and top_ids"),
    (embedding, dict(y=M(data=A + 128)), "table and y"), (embedding, dict(ids=B), "ids and y"),
    (embedding_backward, dict(dtable=M(data=A + 256)), "dy and dtable"), (embedding_backward, dict(ids=B + 128), "ids and dtable"),
    (embedding_backward, dict(dtable=M(data=C)), "dtable and workspace"), (embedding_backward, dict(dy=M(data=C)), "dy and workspace"),
])
def test_shared_memory_is_refused(status, call, kw, names):
    assert status(call, **kw) == f"{names} share memory"


@pytest.mark.parametrize("call,kw", [
    # The places that results may take, and what lies beside without meeting.
    (recurrence, dict(h=M(data=A))), (recurrence, dict(h=M(data=B))), (recurrence, dict(x=M(data=A), h=M(data=A))),
    (recurrence, dict(h=M(data=A + 512))), (recurrence, dict(h=M(data=A - 512))), (recurrence, dict(first=D, last=D)),
    (recurrence, dict(z=M(ld=192), x=M(data=FAKE + 128, ld=192), h=M(data=FAKE + 256, ld=192))),
    (recurrence, dict(tokens=1, z=M(data=A, ld=64), h=M(data=A + 128))),
    (recurrence_backward, dict(dz=M(data=A), dx=M(data=B))), (recurrence_backward, dict(dz=M(data=C), dx=M(data=A))),
    (recurrence_backward, dict(dz=M(data=E, ld=128), dx=M(data=E + 128, ld=128))),
    (recurrence_backward, dict(z=M(data=C), dz=M(data=C))), (recurrence_backward, dict(dlast=FAKE + 4096, dfirst=FAKE + 4096)),
    (recurrence_backward, dict(x=M(data=D), z=M(data=D))),
    (log_probs_backward, dict(dlogits=M(data=A))), (log_probs_backward, dict(logits=M(ld=128), dlogits=M(data=FAKE + 128, ld=128), targets=D)),
    (log_probs, dict(entropy=B + 16, stats=B + 32)), (embedding, dict(y=M(data=A + 9 * 128))),
    (embedding, dict(table=M(ld=128), y=M(data=FAKE + 128, ld=128), ids=D)), (embedding_backward, dict(dtable=M(data=A + 512))),
])
def test_places_that_results_may_take(status, call, kw):
    assert status(call, **kw) == "passes"


def test_against_the_sets_of_elements(status):
    """Random matrices of one buffer: what shares an element is refused unless it is the
    same place, and rows that begin and end within one pitch are told apart exactly."""
    rng, seen = np.random.default_rng(1), set()
    for _ in range(3000):
        rows, cols, ld = (int(rng.integers(1, n)) for n in (6, 9, 4))
        ld *= 8
        start = [int(v) for v in rng.integers(0, 60, 2)]
        if rng.random() < 0.1:
            start[1] = start[0]
        a, b = ({s + r * ld + c for r in range(rows) for c in range(cols)} for s in start)
        got = status(recurrence, tokens=rows, channels=cols, z=M(data=D + 2 * start[0], ld=ld), h=M(data=D + 2 * start[1], ld=ld))
        meets, same = bool(a & b), start[0] == start[1]
        wraps = any(s % ld + cols > ld for s in (start[0] - min(start), start[1] - min(start)))
        if same or not (meets or wraps):
            assert got == "passes", (rows, cols, ld, start)
        elif meets:
            assert got == "z and h share memory", (rows, cols, ld, start)
        seen.add((meets, same, got))
    assert len(seen) >= 3


@pytest.mark.parametrize("call,kw,meets", [
    # Dense results in the gaps between the rows of a matrix with a pitch: row values, states, whole matrices.
    (log_probs, dict(logits=M(ld=192), targets=D, logp=FAKE + 128), False),
    (log_probs, dict(logits=M(ld=192), targets=D, logp=FAKE + 128, stats=FAKE + 144), False),
    (log_probs, dict(logits=M(ld=192), targets=D, logp=FAKE + 384 - 12), True),
    (log_probs, dict(logits=M(ld=192), targets=D, logp=FAKE + 384 - 16), False),
    (recurrence, dict(z=M(data=A, ld=1024), last=A + 128), False), (recurrence, dict(z=M(data=A, ld=1024), last=A + 2048 - 508), True),
    (recurrence, dict(z=M(data=A, ld=1024), h=M(data=A + 128)), False), (recurrence, dict(z=M(data=A, ld=1024), h=M(data=A + 126)), True),
    (recurrence, dict(z=M(data=A, ld=1024), h=M(data=A + 2048 - 512)), False),
    (recurrence, dict(z=M(data=A, ld=1024), h=M(data=A + 2048 - 510)), True),
    (embedding, dict(y=M(data=A - 512)), False), (embedding, dict(y=M(data=A - 510)), True),
])
def test_dense_results_between_rows(status, call, kw, meets):
    assert ("share memory" in status(call, **kw)) == meets
