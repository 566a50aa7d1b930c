"""Sizes that 32 bits do not hold never reach the library, which would see their low bits:
2^32 + 6 rows as 6.  No GPU work."""
import struct

import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from matrix_orthogonalizing_optimizer_shape_gb300 import layer as L
from matrix_orthogonalizing_optimizer_shape_gb300 import model as G
from test_model_args import FAKE, Fake, calls  # noqa: F401

BIG = 2 ** 32 + 6
I64, I32, F32 = torch.int64, torch.int32, torch.float32


class Blocks:
    """What the binding reads of a Packed8."""

    def __init__(self, rows, cols):
        self.codes, self.scales = Fake((rows, cols), torch.int8), Fake((rows, -(-cols // 32)), torch.uint8)


@pytest.mark.parametrize("call", [
    lambda: d3.embedding(Fake((BIG,), I64), Fake((9, 8)), Fake((BIG, 8))),
    lambda: d3.embedding(Fake((6,), I64), Fake((BIG, 8)), Fake((6, 8))),
    lambda: d3.embedding(Fake((6,), I64), Fake((9, BIG)), Fake((6, BIG))),
    lambda: d3.embedding_backward(Fake((BIG, 8)), Fake((BIG,), I64), Fake((9, 8))),
    lambda: d3.embedding_backward(Fake((6, 8)), Fake((6,), I64), Fake((BIG, 8))),
    lambda: d3.recurrence(*[Fake((BIG, 8))] * 3), lambda: d3.recurrence(*[Fake((6, BIG))] * 3),
    lambda: d3.recurrence(*[Fake((6, 8))] * 3, offsets=Fake((BIG,), I32)),
    lambda: d3.recurrence_backward(*[Fake((BIG, 8))] * 6), lambda: d3.recurrence_backward(*[Fake((6, BIG))] * 6),
    lambda: d3.recurrence_backward(*[Fake((6, 8))] * 6, offsets=Fake((2 ** 31 + 2,), I32)),
    lambda: d3.log_probs(Fake((BIG, 8)), Fake((BIG,), I64), Fake((BIG,), F32)), lambda: d3.log_probs(Fake((6, BIG))),
    lambda: d3.log_probs_backward(Fake((BIG, 8)), None, Fake((BIG, 3), F32), Fake((BIG, 8))),
    lambda: d3.log_probs_backward(Fake((6, 2 ** 31)), None, Fake((6, 3), F32), Fake((6, 2 ** 31))),
    lambda: d3.rms_norm(Fake((BIG, 8)), Fake((8,)), Fake((BIG, 8))), lambda: d3.rms_norm(Fake((6, BIG)), Fake((BIG,)), Fake((6, BIG))),
    lambda: d3.rms_norm_backward(Fake((BIG, 8)), Fake((BIG, 8)), Fake((8,)), Fake((BIG,), F32), Fake((BIG, 8))),
    lambda: d3.linear(Fake((BIG, 8)), Fake((9, 8)), Fake((BIG, 9))), lambda: d3.linear(Fake((6, 8)), Fake((BIG, 8)), Fake((6, BIG))),
    lambda: d3.linear_backward(Fake((BIG, 9)), Fake((BIG, 8)), Fake((9, 8)), dw=Fake((9, 8))),
    lambda: d3.pack8(Fake((BIG, 32)), Blocks(BIG, 32)), lambda: d3.unpack8(Blocks(BIG, 32), Fake((BIG, 32))),
    lambda: d3.embedding_backward_workspace_size(BIG, 9, 8), lambda: d3.embedding_backward_workspace_size(4, BIG, 8),
    lambda: d3.embedding_backward_workspace_size(4, 9, BIG), lambda: d3.rms_norm_backward_workspace_size(BIG, 8),
    lambda: d3.linear_workspace_size(BIG, 8, 8, dtype=torch.bfloat16),
    lambda: d3.linear_backward_workspace_size(4, BIG, 8, dtype=torch.bfloat16),
])
def test_refused(calls, call):  # noqa: F811
    with pytest.raises(ValueError, match="larger than any operator takes"):
        call()
    assert not calls


def test_tensors_that_are_clipped_name_their_sizes_in_64_bits(calls):  # noqa: F811
    d3.clip_grad_norm([Fake((4, BIG), stride=(2 * BIG, 1)), Fake((BIG,))], 1.0, stream=1)
    got = struct.unpack("@" + G._TENSOR * 2, calls[-1][1][0])
    assert got == (FAKE, 4, BIG, 2 * BIG, d3.BF16, FAKE, 1, BIG, BIG, d3.BF16)


def test_the_largest_size_is_named(calls):  # noqa: F811
    d3.recurrence(*[Fake((L._MOST, 8))] * 3, stream=1)
    assert calls[-1][1][:2] == (2 ** 31 - 1, 8)
