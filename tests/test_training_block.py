"""The autograd forms of the block-scaled linears, the experts' linears and their routing on
the host: shapes, what is refused, which gradients are asked for; the workspace that a call
takes outlives it."""
import weakref

import pytest
import torch

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
from int8_mixed_precision_rowwise_amd import block_operators as B  # noqa: E402
from int8_mixed_precision_rowwise_amd import training as T  # noqa: E402

bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


@pytest.fixture
def plain(monkeypatch):
    """Stand-ins in plain torch over unquantized weights; the list of what was called with which wants."""
    seen = []

    def quantize(W):
        seen.append("quantize")
        return W.detach().clone(), torch.zeros(1)

    def fwd(x, w, e, *a):
        return x @ w.transpose(-1, -2) if w.dim() == 2 else torch.cat([x @ w[0].t()] + [z(0, w.shape[1])])

    def bwd(dy, x, w, e, want_dx=True, want_dw=True):
        seen.append(("bwd", want_dx, want_dw))
        return dy @ w if want_dx else None, dy.t() @ x if want_dw else None

    def ebwd(dy, x, w, e, offsets, rows=None, want_dx=True, want_dw=True):
        seen.append(("ebwd", want_dx, want_dw))
        return dy @ w[0] if want_dx else None, torch.zeros_like(w) if want_dw else None

    def combine(y, places, weights=None, residual=None):
        s = y[places.long()] * (1 if weights is None else weights[..., None].to(y.dtype))
        return s.sum(1) + (0 if residual is None else residual)

    def combine_bwd(dout, y, places, weights=None, rows=None, want_dy=True, want_dweights=True):
        seen.append(("combine_bwd", want_dy, want_dweights))
        return torch.zeros_like(y) if want_dy else None, torch.zeros(places.shape) if want_dweights else None

    def route(x, k, score, normalize):
        w, e = x.softmax(1).topk(k)
        ints = torch.zeros(3 * e.numel() + x.shape[1] + 1, dtype=i32)
        n = e.numel()
        a, b, c, d = ints.split_with_sizes((n, n, n, x.shape[1] + 1))
        return B.Route(w, a.view(e.shape), b.view(e.shape), c, d)

    for name, f in dict(quantize_block_weight=quantize, linear_block_fwd=fwd, linear_block_bwd=bwd, expert_linear_fwd=fwd,
                        expert_linear_bwd=ebwd, expert_combine=combine, expert_combine_bwd=combine_bwd, expert_route=route,
                        expert_route_bwd=lambda x, e, dw, *a: torch.zeros_like(x)).items():
        monkeypatch.setattr(B, name, f)
    return seen


@pytest.mark.parametrize("lead,N,K", [((3,), 16, 8), ((2, 3), 24, 40), ((), 16, 8), ((0,), 16, 8), ((2, 0), 16, 8)])
def test_shapes(plain, lead, N, K):
    x, w = z(*lead, K).requires_grad_(), z(N, K).requires_grad_()
    y = T.linear_block(x, w)
    assert y.shape == (*lead, N)
    dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
    assert dx.shape == x.shape and dw.shape == w.shape and plain == ["quantize", ("bwd", True, True)]


def test_the_codes_given_are_the_ones_used(plain):
    x, w = torch.randn(4, 8).to(bf), torch.randn(16, 8).to(bf).requires_grad_()
    other = torch.randn(16, 8).to(bf)
    y = T.linear_block(x, w, quantized=(other, torch.zeros(1)))
    assert torch.equal(y, x @ other.t()) and plain == []
    y.sum().backward()
    assert plain == [("bwd", False, True)]
    with pytest.raises(ValueError, match="are not those of a weight"):
        T.linear_block(x, w, quantized=(other[:8], torch.zeros(1)))
    with pytest.raises(ValueError, match="are not those of a weight"):
        T.expert_linear(x, w.detach()[None], z(2, dtype=i32), quantized=(other, torch.zeros(1)))


def test_only_what_is_needed_is_asked_for(plain):
    x, w = torch.randn(4, 8).to(bf), torch.randn(16, 8).to(bf)
    T.linear_block(x.requires_grad_(), w).sum().backward()
    T.expert_linear(x, w[None], z(2, dtype=i32)).sum().backward()
    y, places, wt = torch.randn(8, 16).to(bf), torch.arange(8, dtype=i32).view(4, 2), torch.rand(4, 2)
    r = torch.randn(4, 16).to(bf).requires_grad_()
    plain.clear()
    out = T.expert_combine(y, places, wt, r)
    g = torch.randn(4, 16).to(bf)
    assert torch.equal(torch.autograd.grad(out, r, g)[0], g) and plain == []  # the output's own
    T.expert_combine(y.requires_grad_(), places, wt).sum().backward()
    T.expert_combine(y.detach(), places, wt.requires_grad_()).sum().backward()
    assert plain == [("combine_bwd", True, False), ("combine_bwd", False, True)]
    with torch.no_grad():
        assert not T.expert_combine(y, places, wt).requires_grad and not T.linear_block(x, w).requires_grad


def test_the_weights_alone_have_a_gradient(plain):
    logits = torch.randn(5, 6, requires_grad=True)
    r = T.expert_route(logits, 2)
    assert isinstance(r, B.Route) and r.weights.requires_grad and not any(t.requires_grad for t in r[1:])
    (d,) = torch.autograd.grad(r.weights.sum(), logits)
    assert d.shape == logits.shape


def test_refusals():
    w3, off = z(2, 16, 8), z(3, dtype=i32)
    for x, w in ((z(4, 9), z(16, 8)), (z(4, 8), w3), (torch.tensor(1.0), z(16, 8))):
        with pytest.raises(ValueError, match="do not match"):
            T.linear_block(x, w)
    for x, w in ((z(4, 9), w3), (z(2, 4, 8), w3), (z(4, 8), z(16, 8))):
        with pytest.raises(ValueError, match="do not match"):
            T.expert_linear(x, w, off)
    with pytest.raises(ValueError, match="together"):
        T.expert_linear(z(4, 8), w3, off, rows=z(8, dtype=i32))
    with pytest.raises(ValueError, match="each of 4 tokens"):
        T.expert_linear(z(4, 8), w3, off, rows=z(8, dtype=i32), places=z(3, 2, dtype=i32))
    with pytest.raises(ValueError, match="device tensors"):
        T.linear_block(z(4, 8), z(16, 8))


def test_second_derivatives_are_refused(plain):
    x, w = torch.randn(4, 8).to(bf).requires_grad_(), torch.randn(16, 8).to(bf).requires_grad_()
    w3 = w.detach()[None].clone().requires_grad_()
    y, wt = torch.randn(8, 16).to(bf).requires_grad_(), torch.rand(4, 2).requires_grad_()
    logits, places, off = torch.randn(5, 6, requires_grad=True), torch.arange(8, dtype=i32).view(4, 2), z(2, dtype=i32)
    for out, leaves in ((T.linear_block(x, w), (x, w)), (T.expert_linear(x, w3, off), (x, w3)),
                        (T.expert_combine(y, places, wt), (y, wt)), (T.expert_route(logits, 2).weights, (logits,))):
        for part in torch.autograd.grad(out.square().sum(), leaves, create_graph=True):
            with pytest.raises(RuntimeError, match="no second derivative"):
                (part.sum() + leaves[0].square().sum()).backward(retain_graph=True)


@pytest.mark.parametrize("which", ["fwd", "bwd", "experts fwd", "experts bwd", "route"])
def test_the_workspace_is_alive_in_the_call(monkeypatch, which):
    taken, seen, empty = [], [], torch.empty

    def recording_empty(*args, **kw):
        t = empty(*args, **kw)
        if t.dtype == u8:
            taken.append((weakref.ref(t), t.data_ptr(), t.numel()))
        return t

    def call(dev, name, *args):
        seen.append((name, len(taken), all(r() is not None for r, _, _ in taken), [(p, n) in zip(args, args[1:]) for _, p, n in taken]))

    monkeypatch.setattr(B, "_on_gpu", lambda *t: True)
    monkeypatch.setattr(i8, "_device", lambda *t: t[0].device)
    monkeypatch.setattr(torch, "empty", recording_empty)
    monkeypatch.setattr(B, "_call", call)
    X, codes, exps = z(300, 64), z(48, 64, dtype=u8), z(1, 1, dtype=u8)
    off = torch.tensor([0, 100, 300], dtype=i32)
    if which == "fwd":
        B.linear_block_fwd(X, codes, exps)
    elif which == "bwd":
        B.linear_block_bwd(z(300, 48), X, codes, exps)
    elif which == "experts fwd":
        B.expert_linear_fwd(X, codes.expand(2, 48, 64).contiguous(), z(2, 1, 1, dtype=u8), off)
    elif which == "experts bwd":
        B.expert_linear_bwd(z(300, 48), X, codes.expand(2, 48, 64).contiguous(), z(2, 1, 1, dtype=u8), off)
    else:
        B.expert_route(z(3000, 8), 2)
    ((_, n, alive, given),) = seen
    assert n == 1 and alive and all(given)
