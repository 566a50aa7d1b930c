"""Clipping of a small set in one launch of a cluster and in the launches of any set: the
same bits.  More tensors than the cluster takes, most of them empty, go the second way."""
import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes", [[(1, 1)], [(64, 64), (1, 4096), (33, 1000)], [(128, 513), (513, 128)] * 3, [(4, 65536)]])
def test_both_ways_give_the_same_bits(cuda_lib, dtype, sizes):
    rng = np.random.default_rng(len(sizes))
    ws = d3.alloc_workspace(d3.grad_norm_workspace_size())
    # Whole numbers: their squares' sums are exact in any order.
    ts = [torch.from_numpy(rng.integers(-8, 9, s)).to(dtype).cuda() for s in sizes]
    empty = [torch.empty(0, dtype=dtype, device="cuda") for _ in range(20)]
    total = sum(float(t.double().square().sum()) for t in ts)
    for max_norm in (0.0, 0.5, 1e9):
        got = []
        for more in ([], empty):
            new, norm = [torch.full_like(t, 7) for t in ts], torch.zeros(1, device="cuda")
            d3.clip_grad_norm(ts + more, max_norm, norm, out=new + more, ws=ws)
            place = [t.clone() for t in ts]
            d3.clip_grad_norm(place + more, max_norm, ws=ws)
            assert all(torch.equal(a, b) for a, b in zip(new, place))
            got.append((new, norm))
        assert all(torch.equal(a, b) for a, b in zip(got[0][0], got[1][0])) and torch.equal(got[0][1], got[1][1])
        assert float(got[0][1]) == float(np.float32(np.sqrt(total)))
