"""The combination's gradient where places were taken away after the routing, as a limit on an expert's rows does:
rows of Y that no place names have a gradient of zero, whatever the rows' tokens still say."""
import pytest
import torch

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from int8_mixed_precision_rowwise_amd import training  # noqa: E402

nan = float("nan")


@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (40, 6, 3), (130, 40, 32), (3000, 8, 2)])
@pytest.mark.parametrize("N", [24, 13, 520])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_places_taken_away(T, E, k, N, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, E, generator=g, device="cuda")
    x[T // 2] = -float("inf") if T > 1 else x[T // 2]
    r = i8.expert_route(x, k)
    places = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.4, -1, r.places)
    R = T * k
    Y, dout = (torch.randn(n, N, generator=g, device="cuda").to(dtype) for n in (R, T))
    want, dw = i8.expert_combine_bwd(dout, Y, places, r.weights)  # clears first
    kept = torch.zeros(R, dtype=torch.bool, device="cuda")
    kept[places[places >= 0].long()] = True
    assert not bool(want[~kept].any())
    for given in (True, False):
        blocks = [torch.full((R, N), nan, dtype=dtype, device="cuda") for _ in range(3)]
        out = blocks.pop() if given else None
        del blocks  # NaN for the allocator to give again
        dY, again = i8.expert_combine_bwd(dout, Y, places, r.weights, rows=r.rows, dY=out)
        assert torch.equal(dY, want) and torch.equal(again, dw)
    beyond = torch.where(kept, r.rows, T + 5)  # a token that there is not
    assert torch.equal(i8.expert_combine_bwd(dout, Y, places, r.weights, rows=beyond, dY=torch.full_like(Y, nan))[0], want)
    y = Y.clone().requires_grad_()
    out = training.expert_combine(y, places, r.weights, rows=r.rows)
    blocks = [torch.full((R, N), nan, dtype=dtype, device="cuda") for _ in range(3)]
    del blocks
    assert torch.equal(torch.autograd.grad(out, y, dout)[0], want)


def test_a_layer_whose_places_are_taken_away_in_place():
    """As expert by expert over the rows that are left; the experts' weights see nothing of the others."""
    tokens, E, k, D = 90, 5, 2, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(tokens, E, generator=g, device="cuda").requires_grad_()
    y_of = torch.randn(tokens * k, D, generator=g, device="cuda")
    dout = torch.randn(tokens, D, generator=g, device="cuda")
    drop = torch.rand(tokens, k, generator=g, device="cuda") < 0.3
    grads = []
    for in_place in (True, False):
        y = y_of.clone().requires_grad_()
        r = training.expert_route(logits, k)
        places = r.places.masked_fill_(drop, -1) if in_place else r.places.masked_fill(drop, -1)
        out = training.expert_combine(y, places, r.weights, rows=r.rows)
        grads.append(torch.autograd.grad(out, (logits, y), dout))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    assert bool(grads[0][0].any()) and not bool(grads[0][1][r.places[drop].long()].any())
