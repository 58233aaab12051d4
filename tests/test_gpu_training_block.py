"""Gradients through the autograd forms of the block-scaled linears, the experts' linears and
their routing."""
import numpy as np
import pytest
import torch

from . import block_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from int8_mixed_precision_rowwise_amd import training as T  # noqa: E402

bf = torch.bfloat16


def randn(seed, *shape, dtype=bf, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


@pytest.mark.parametrize("lead,N,K", [((5,), 40, 24), ((2, 70), 264, 136), ((3, 2, 50), 130, 100), ((), 24, 16), ((0,), 24, 16)])
def test_linear_block(lead, N, K):
    """Any leading dimensions, rows that do not start every 16 bytes, gradients that are expanded."""
    x, w = randn(1, *lead, K).requires_grad_(), randn(2, N, K, std=0.1).requires_grad_()
    y = T.linear_block(x, w)
    assert y.shape == (*lead, N)
    g = randn(3, *lead, N)
    dx, dw = torch.autograd.grad(y, (x, w), g, retain_graph=True)
    x64, w64, g64 = ref.to64(x).reshape(-1, K), ref.to64(w), ref.to64(g).reshape(-1, N)
    ref.close(y.reshape(-1, N), *ref.forward(x64, w64), "y")
    ref.close(dx.reshape(-1, K), *ref.grad_input(g64, w64), "dx")
    ref.close(dw, *ref.grad_weight(g64, x64), "dw")
    y.sum().backward()  # one number for all
    ref.close(w.grad, *ref.grad_weight(np.ones_like(g64), x64), "dw of a sum")
    assert x.grad.shape == x.shape
    q = i8.quantize_block_weight(w.detach()) if K % 8 == 0 else None
    if q:
        assert torch.equal(T.linear_block(x, w, quantized=q), y)


def test_a_layer_of_experts():
    """The gradients of a whole layer are those that its operators give one after the other."""
    N_TOK, E, k, D, H = 130, 5, 2, 136, 264
    x = randn(1, N_TOK, D).requires_grad_()
    w1, w2 = randn(2, E, H, D, std=0.1).requires_grad_(), randn(3, E, D, H, std=0.1).requires_grad_()
    logits = randn(4, N_TOK, E, dtype=torch.float32)
    logits[11] = -float("inf")
    logits.requires_grad_()
    g = randn(5, N_TOK, D)

    r = T.expert_route(logits, k, score="sigmoid")
    h = torch.nn.functional.silu(T.expert_linear(x, w1, r.offsets, r.rows, r.places))
    y = T.expert_linear(h, w2, r.offsets)
    out = T.expert_combine(y, r.places, r.weights, residual=x, rows=r.rows)
    grads = torch.autograd.grad(out, (x, w1, w2, logits), g)

    with torch.no_grad():
        q1, q2 = i8.quantize_block_weight(w1), i8.quantize_block_weight(w2)
        s = i8.expert_route(logits, k, score="sigmoid")
        assert all(torch.equal(a, b) for a, b in zip(r, s))
        z = i8.expert_linear_fwd(x, *q1, s.offsets, s.rows)
    z.requires_grad_()
    a = torch.nn.functional.silu(z)
    with torch.no_grad():
        y2 = i8.expert_linear_fwd(a, *q2, s.offsets)
        assert torch.equal(out, i8.expert_combine(y2, s.places, s.weights, x))
        dy, dwt = i8.expert_combine_bwd(g, y2, s.places, s.weights, rows=s.rows)
        da, dw2 = i8.expert_linear_bwd(dy, a, *q2, s.offsets)
    (dz,) = torch.autograd.grad(a, z, da)
    dxs, dw1 = i8.expert_linear_bwd(dz, x.detach(), *q1, s.offsets, s.rows)
    dx = i8.expert_combine(dxs, s.places) + g  # both bf16: autograd adds the residual's part
    want = dx, dw1, dw2, i8.expert_route_bwd(logits.detach(), s.experts, dwt, score="sigmoid")
    for name, got, w in zip(("x", "w1", "w2", "logits"), grads, want):
        assert torch.equal(got, w), name
    with torch.no_grad():  # without a backward: the same numbers
        assert torch.equal(T.expert_linear(x, w1, r.offsets, r.rows, r.places), z)


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_and_combination_against_differences(score, normalize):
    """Directional differences, in 64 bits, of sum(G * combine(Y, weights(logits))) for the choice made."""
    N_TOK, E, k, N = 40, 12, 3, 24
    logits, Y, G = (randn(i, *s, dtype=torch.float32).requires_grad_() for i, s in ((1, (N_TOK, E)), (2, (N_TOK * k, N)), (3, (N_TOK, N))))
    res = randn(4, N_TOK, N, dtype=torch.float32).requires_grad_()
    r = T.expert_route(logits, k, score=score, normalize=normalize)
    out = T.expert_combine(Y, r.places, r.weights, residual=res)
    dl, dY, dr = torch.autograd.grad((out * G).sum(), (logits, Y, res))
    e, p, g64 = r.experts.cpu().numpy(), r.places.cpu().numpy(), ref.to64(G)

    def f(x, y, z):
        at = np.take_along_axis(x, e, 1)
        s = 1 / (1 + np.exp(-at)) if score == "sigmoid" else np.exp(at)
        total = s.sum(1, keepdims=True) if normalize else 1.0 if score == "sigmoid" else np.exp(x).sum(1, keepdims=True)
        return (((s / total)[..., None] * y[p]).sum(1) * g64).sum() + (z * g64).sum()

    rng, h = np.random.default_rng(7), 1e-5
    a, b, c = ref.to64(logits), ref.to64(Y), ref.to64(res)
    va, vb, vc = (rng.standard_normal(t.shape) for t in (a, b, c))
    diff = (f(a + h * va, b + h * vb, c + h * vc) - f(a - h * va, b - h * vb, c - h * vc)) / (2 * h)
    got = (ref.to64(dl) * va).sum() + (ref.to64(dY) * vb).sum() + (ref.to64(dr) * vc).sum()
    # the difference's own error is of order h^2 and 2^-52 / h of the sums; the gradients' are fp32 steps of theirs
    size = sum(np.abs(ref.to64(d) * v).sum() for d, v in ((dl, va), (dY, vb), (dr, vc)))
    assert abs(diff - got) <= 1e-5 * size


def test_replayed_from_a_graph():
    """A step captured whole, forward and backward, replayed over other inputs."""
    M, N, K = 200, 264, 136
    x, w, g = randn(1, M, K).requires_grad_(), randn(2, N, K, std=0.1).requires_grad_(), randn(3, M, N)
    logits, w3 = randn(4, M, 6).requires_grad_(), randn(5, 6, N, K, std=0.1).requires_grad_()

    def step():
        r = T.expert_route(logits, 2)
        y = T.expert_combine(T.expert_linear(x, w3, r.offsets, r.rows, r.places), r.places, r.weights, rows=r.rows)
        y = y + T.linear_block(x, w)
        return (y.detach(), *torch.autograd.grad(y, (x, w, logits, w3), g))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(3):
        with torch.no_grad():
            for i, t in enumerate((x, g, logits)):
                t.copy_(randn(10 * rep + i, *t.shape))
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(mine, step()))


@pytest.mark.parametrize("tokens,padding", [(0, False), (20, True)])
def test_a_layer_without_rows(tokens, padding):
    """No tokens at all, and padding alone: what comes in goes out, and the weights' gradients are zeros."""
    E, k, D, H = 4, 2, 40, 24
    x = randn(1, tokens, D).requires_grad_()
    w1, w2 = randn(2, E, H, D).requires_grad_(), randn(3, E, D, H).requires_grad_()
    logits = torch.full((tokens, E), -float("inf"), device="cuda").requires_grad_()
    r = T.expert_route(logits, k)
    y = T.expert_linear(T.expert_linear(x, w1, r.offsets, r.rows, r.places), w2, r.offsets)
    out = T.expert_combine(y, r.places, r.weights, residual=x, rows=r.rows)
    assert torch.equal(out, x)
    g = randn(4, tokens, D)
    dx, dw1, dw2, dl = torch.autograd.grad(out, (x, w1, w2, logits), g)
    assert torch.equal(dx, g) and not dw1.any() and not dw2.any() and not dl.any()
    assert dw1.shape == w1.shape and dl.shape == logits.shape
