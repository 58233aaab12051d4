"""Experts' linears over a part of the rows: offsets that start behind the first row, as a slice of
all experts' offsets has them.  What no expert has is zero in an output that the call makes, in front as behind."""
import numpy as np
import pytest
import torch

from . import block_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from int8_mixed_precision_rowwise_amd import training as T  # noqa: E402

bf, i32, nan = torch.bfloat16, torch.int32, float("nan")


def randn(seed, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(bf).cuda()


def leave_nan(*shapes):
    """Blocks of these sizes that hold NaN go back to the allocator, which gives them to the next calls."""
    blocks = [torch.full(s, nan, dtype=bf, device="cuda") for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del blocks


# rows in front, of each expert, behind; N, K: few rows, small tiles and big tiles
PARTS = [(5, [3, 0, 9], 4, 40, 72), (20, [0, 0], 0, 40, 72), (130, [70, 0, 300], 40, 136, 264), (300, [0, 0], 7, 136, 264),
         (700, [1400, 0, 600, 3000, 0, 260], 90, 2056, 2056)]


@pytest.mark.parametrize("front,counts,behind,N,K", PARTS)
@pytest.mark.parametrize("gather", [False, True])
def test_rows_in_front_of_the_first_expert(front, counts, behind, N, K, gather):
    E, used = len(counts), sum(counts)
    R, tokens = front + used + behind, 50
    offsets = torch.tensor(np.cumsum([front, *counts]), dtype=i32, device="cuda")
    W, dY = randn(2, E, N, K, std=0.02), randn(3, R, N)
    X = randn(1, tokens if gather else R, K)
    rows = ((torch.arange(R, dtype=i32) * 7) % tokens).cuda() if gather else None
    x = ref.to64(X)[rows.cpu().numpy()] if gather else ref.to64(X)
    q = i8.quantize_block_weight(W)
    leave_nan((R, N), (R, K))
    Y = i8.expert_linear_fwd(X, *q, offsets, rows)
    dX, dW = i8.expert_linear_bwd(dY, X, *q, offsets, rows)
    out = slice(front, front + used)
    for t in (Y, dX):
        rest = torch.cat((t[:front], t[front + used:]))
        assert not bool(rest.isnan().any()) and not bool(rest.any())
    a, w, dy = front, ref.to64(W), ref.to64(dY)
    for e, n in enumerate(counts):
        at, a = slice(a, a + n), a + n
        ref.close(Y[at], *ref.forward(x[at], w[e]), f"Y of expert {e}")
        ref.close(dX[at], *ref.grad_input(dy[at], w[e]), f"dX of expert {e}")
        ref.close(dW[e], *ref.grad_weight(dy[at], x[at]), f"dW of expert {e}")
    # given outputs keep them
    gy, gx = torch.full((R, N), 7.0, dtype=bf, device="cuda"), torch.full((R, K), 7.0, dtype=bf, device="cuda")
    i8.expert_linear_fwd(X, *q, offsets, rows, out=gy)
    i8.expert_linear_bwd(dY, X, *q, offsets, rows, dX=gx, want_dw=False)
    for g, t in ((gy, Y), (gx, dX)):
        assert torch.equal(g[out], t[out]) and bool((g[:front] == 7).all()) and bool((g[front + used:] == 7).all())


def test_two_halves_of_the_experts_are_the_layer():
    """A layer whose experts are taken in two calls, each with its slice of the offsets: outputs and the tokens'
    gradients add up to the whole one's, whose parts the other call leaves at zero."""
    tokens, E, k, D, H = 200, 6, 2, 72, 136
    x, w = randn(1, tokens, D), randn(2, E, H, D, std=0.1)
    logits = torch.randn(tokens, E, generator=torch.Generator().manual_seed(4)).cuda()
    g = randn(5, tokens * k, H)
    r = i8.expert_route(logits, k)
    want = []
    for lo, hi in ((0, E), (0, 2), (2, E)):
        xs = x.clone().requires_grad_()
        leave_nan((tokens * k, H), (tokens * k, D))
        y = T.expert_linear(xs, w[lo:hi], r.offsets[lo:hi + 1], r.rows, r.places)
        leave_nan((tokens * k, H), (tokens * k, D))
        want.append((y.detach(), torch.autograd.grad(y, xs, g)[0]))
    (y, dx), (ya, dxa), (yb, dxb) = want
    cut = int(r.offsets[2])
    assert torch.equal(torch.cat((ya[:cut], yb[cut:])), y) and not bool(ya[cut:].any()) and not bool(yb[:cut].any())
    # each of a token's two rows in either half, so a sum of two halves has no third rounding beyond bf16's own
    err = (dxa.double() + dxb.double() - dx.double()).abs()
    assert bool((err <= 2.0**-8 * (dx.double().abs() + dxa.double().abs() + dxb.double().abs())).all())
