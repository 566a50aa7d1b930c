"""32-bit weight gradients over many tokens: the tensor cores' sums stop at 4096
tokens in every kernel that the product can take, so the error does not grow."""
import pytest
import torch

import matrix_orthogonalizing_optimizer_shape_gb300 as d3
from test_gpu_layer_norm import out, untouched

pytestmark = pytest.mark.gpu

#: Tokens of a piece, and the most CTAs that share the tokens.
PIECE, SHARES = 4096, 8
DTYPES = [torch.bfloat16, torch.float16]


def operands(t, k, n, dtype):
    """Positive rows (an accumulator that truncates loses one way) that repeat every piece."""
    g = torch.Generator(device="cuda").manual_seed(k + n)
    rows = torch.arange(t, device="cuda") % PIECE
    return [torch.randn(PIECE, c, generator=g, device="cuda").abs_().to(dtype)[rows] for c in (k, n)]


def gradient(x, dy, dw, **kw):
    (t, k), n = x.shape, dy.shape[1]
    ws = d3.alloc_workspace(d3.linear_backward_workspace_size(t, k, n, dtype=x.dtype))
    d3.linear_backward(dy, x, torch.zeros(n, k, dtype=x.dtype, device="cuda"), dw=dw, ws=ws, **kw)
    d3.device_status()
    return dw


# tokens, in, out: 128- and 64-wide tiles over 4 and 8 CTAs, at odd widths too; pairs 256 and 128 wide
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,n", [(262144, 1024, 1024), (524288, 256, 256), (524288, 136, 72), (524288, 65, 7),
                                   (131072, 2304, 2560), (131072, 2048, 1024)])
def test_error_does_not_grow_with_the_tokens(cuda_lib, t, k, n, dtype):
    """Every sum of whole pieces is made of the same partial sums, so a longer one is a shorter one's multiple but for
    the roundings of adding them: 2^-24 of a partial result for each, of which one share is at most t / PIECE long."""
    short = PIECE * SHARES
    x, dy = operands(t, k, n, dtype)
    for pad in (0, 1):
        one = gradient(x[:short], dy[:short], out(n, k, "f32", pad)[0]).double()
        dw, buf = out(n, k, "f32", pad)
        many = gradient(x, dy, dw).double()
        tol = 2.0 ** -24 * (t // PIECE + short // PIECE + 2 * SHARES)
        off = float((many / (one * (t // short)) - 1).abs().max())
        assert off <= tol and untouched(dw, buf), (off, tol)
        gradient(x, dy, dw, accumulate=True)
        off = float((dw.double() / (many * 2) - 1).abs().max())
        assert off <= tol and untouched(dw, buf), (off, tol)


# one piece a CTA, one slab of 64 tokens more, a ragged last slab; pieces that end inside a pair's tile
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,n", [(32768, 256, 256), (33280, 256, 256), (65473, 256, 200), (524301, 136, 72),
                                   (8256, 2304, 2560), (12289, 1024, 2048), (20000, 1024, 1024)])
def test_sums_of_ragged_pieces(cuda_lib, t, k, n, dtype):
    """Against 64 bits.  The i-th of a piece's 256 additions to an accumulator adds 16 products; each of the 17 terms
    loses at most 2^-23 of i / 256 of the piece, which grows evenly (to 5 %); pieces and shares add with 2^-24."""
    x, dy = operands(t, k, n, dtype)
    want = torch.zeros(n, k, dtype=torch.float64, device="cuda")
    for i in range(0, t, 65536):
        want += dy[i:i + 65536].double().t() @ x[i:i + 65536].double()
    joined = -(-t // PIECE) + SHARES + 1
    tol = 1.05 * 17 * (PIECE // 16 + 1) / 2 * 2.0 ** -23 + joined * 2.0 ** -24
    for pad in (0, 1):
        dw, buf = out(n, k, "f32", pad)
        gradient(x, dy, dw)
        off = float((dw.double() / want - 1).abs().max())
        assert off <= tol and untouched(dw, buf), (off, tol)
        first = dw.clone()
        gradient(x, dy, dw)
        assert torch.equal(dw, first), "the same bits every call"
