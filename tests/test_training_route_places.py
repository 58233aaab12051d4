"""Places taken away in place after the routing, on the host with stand-ins: the tensors of a route are one
allocation's parts, and a change of one of them is no change of the others."""
import pytest
import torch

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
from int8_mixed_precision_rowwise_amd import block_operators as B  # noqa: E402
from int8_mixed_precision_rowwise_amd import training as T  # noqa: E402

i32 = torch.int32


@pytest.fixture
def route(monkeypatch):
    """A route of 6 tokens to 2 of 4 experts; its gradient is 1 at what the experts say."""
    def forward(x, k, score, normalize):
        n = x.shape[0] * k
        ints = torch.arange(3 * n + x.shape[1] + 1, dtype=i32)
        experts, places, rows, offsets = ints.split_with_sizes((n, n, n, x.shape[1] + 1))
        return B.Route(torch.ones(x.shape[0], k), experts.view(-1, k), places.view(-1, k), rows, offsets)

    monkeypatch.setattr(B, "expert_route", forward)
    monkeypatch.setattr(B, "expert_route_bwd", lambda x, e, dw, *a: torch.ones_like(x))
    x = torch.randn(6, 4).requires_grad_()
    return x, T.expert_route(x, 2)


@pytest.mark.parametrize("name", ["places", "rows", "offsets"])
def test_a_change_of_one_is_none_of_the_experts(route, name):
    x, r = route
    others = [getattr(r, o).clone() for o in B.Route._fields if o != name]
    getattr(r, name).fill_(-1)
    assert all(torch.equal(getattr(r, o), was) for o, was in zip((o for o in B.Route._fields if o != name), others))
    r.weights.sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x))


def test_a_change_of_the_experts_is_seen(route):
    x, r = route
    r.experts.fill_(-1)
    with pytest.raises(RuntimeError, match="inplace"):
        r.weights.sum().backward()


def test_what_a_layer_saved_of_a_route_is_only_what_it_saved(route, monkeypatch):
    """Places changed between two layers' calls: the first one's gradient at the tokens would be another, and is refused;
    a layer without them is not concerned."""
    x, r = route
    monkeypatch.setattr(B, "expert_linear_fwd", lambda x, c, e, o, rows=None: torch.ones(12, c.shape[1]))
    monkeypatch.setattr(B, "expert_linear_bwd", lambda dy, x, c, e, o, rows=None, a=True, b=True: (torch.zeros(12, c.shape[2]), None))
    monkeypatch.setattr(B, "expert_combine", lambda y, p, *a: torch.zeros(p.shape[0], y.shape[1]))
    q = torch.zeros(4, 8, 16, dtype=torch.uint8), torch.zeros(4, 1, 1, dtype=torch.uint8)
    w = torch.zeros(4, 8, 16)
    tokens, rows = torch.zeros(6, 16).requires_grad_(), torch.zeros(12, 16).requires_grad_()
    y = T.expert_linear(tokens, w, r.offsets, r.rows, r.places, quantized=q)
    z = T.expert_linear(rows, w, r.offsets, quantized=q)
    r.places[2] = -1
    z.sum().backward()
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
