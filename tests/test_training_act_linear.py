"""The linear module with an epilogue, and the autograd forms of the operators, on the host."""
import pytest
import torch

pytest.importorskip("int8_mixed_precision_rowwise_amd")
from int8_mixed_precision_rowwise_amd import training as T  # noqa: E402

bf = torch.bfloat16


@pytest.mark.parametrize("bias", [True, False])
def test_from_linear_keeps_the_parameters(bias):
    lin = torch.nn.Linear(24, 16, bias=bias, dtype=bf)
    cfg = T.Int8MixedPrecisionConfig(stochastic_rounding=True)
    m = T.Int8MixedPrecisionActLinear.from_linear(lin, cfg, 7, activation="silu")
    assert type(m) is T.Int8MixedPrecisionActLinear and m.weight is lin.weight and m.bias is lin.bias
    assert (m.in_features, m.out_features, m.config, m.seed, m.step, m.activation) == (24, 16, cfg, 7, 0, "silu")
    assert "activation=silu" in repr(m) and f"bias={bias}" in repr(m)
    assert T.Int8MixedPrecisionActLinear.from_linear(lin, cfg, 7).activation == "none"
    again = T.Int8MixedPrecisionActLinear(24, 16, bias=bias, activation="silu", config=cfg)
    again.load_state_dict(m.state_dict())
    assert again.seed == 7 and torch.equal(again.weight, lin.weight)
    # what the forward hands on is all there: the call is refused for its device only
    with pytest.raises(ValueError, match="device tensors"):
        m(torch.zeros(3, 24, dtype=bf))


def test_from_linear_refuses_what_the_constructor_refuses():
    lin = torch.nn.Linear(24, 16, dtype=bf)
    for bad in (dict(fp8=True), dict(output=False), dict(grad_input=False), dict(grad_weight=False)):
        with pytest.raises(ValueError, match="all three GEMMs in INT8"):
            T.Int8MixedPrecisionActLinear.from_linear(lin, T.Int8MixedPrecisionConfig(**bad), 0)
    with pytest.raises(ValueError, match="activation must be one of"):
        T.Int8MixedPrecisionActLinear.from_linear(lin, T.Int8MixedPrecisionConfig(), 0, activation="tanh")


@pytest.fixture
def forwards(monkeypatch):
    """Names of the forwards called, with stand-ins that compute nothing but the shapes."""
    seen = []

    def plain(x, w, bias, activation, residual, rounding, seed, offset):
        seen.append("plain")
        return torch.zeros(x.shape[0], w.shape[0], dtype=bf)

    def train(x, w, *rest):
        seen.append("train")
        y = torch.zeros(x.shape[0], w.shape[0], dtype=bf)
        return y, torch.zeros_like(y), torch.zeros(x.shape[1]), torch.zeros(x.shape[1])

    monkeypatch.setattr(T._ops, "linear_act_fwd", plain)
    monkeypatch.setattr(T._ops, "linear_act_fwd_train", train)
    return seen


def test_the_pre_activation_is_kept_for_a_backward_only(forwards):
    x, w, b, r = torch.zeros(2, 3, 8, dtype=bf), torch.zeros(16, 8, dtype=bf), torch.zeros(16, dtype=bf), torch.zeros(2, 3, 16, dtype=bf)
    assert T.linear_act(x, w, b, "silu", r).shape == (2, 3, 16) and forwards == ["plain"]
    m = T.Int8MixedPrecisionActLinear(8, 16, activation="silu")
    with torch.no_grad():
        assert m(x, r).shape == (2, 3, 16)
    with torch.inference_mode():
        m(x)
    assert forwards == ["plain"] * 3
    y = m(x)
    assert y.requires_grad and forwards[3:] == ["train"]
    for leaf in ("x", "w", "b"):
        a = dict(x=x, w=w, b=b)
        a[leaf] = a[leaf].clone().requires_grad_()
        T.linear_act(a["x"], a["w"], a["b"], "silu", r)
    assert forwards[4:] == ["train"] * 3
    res = r.clone().requires_grad_()  # the residual's gradient is the output's own
    out = T.linear_act(x, w, b, "silu", res)
    assert forwards[7:] == ["plain"]
    g = torch.ones(2, 3, 16, dtype=bf)
    assert torch.equal(torch.autograd.grad(out, res, g)[0], g)


def test_second_derivatives_are_right_or_refused(monkeypatch):
    """Rotary's is the rotation itself; the others have none and say so."""
    def turned(q, k, positions, freqs, pairs="half", inverse=False):  # a quarter turn of both halves, on the CPU
        a, b = q.chunk(2, -1)
        return (torch.cat((b, -a), -1) if inverse else torch.cat((-b, a), -1)), k

    monkeypatch.setattr(T._ops, "rotary", turned)
    q = torch.randn(1, 2, 3, 8, dtype=torch.float64, requires_grad=True)
    g = torch.randn(1, 2, 3, 8, dtype=torch.float64, requires_grad=True)
    out, _ = T.rotary(q, None, None, None)
    (dq,) = torch.autograd.grad(out, q, g, create_graph=True)
    v = torch.randn_like(q)
    (dg,) = torch.autograd.grad(dq, g, v)
    assert torch.equal(dq, turned(g, None, None, None, inverse=True)[0]) and torch.equal(dg, turned(v, None, None, None)[0])

    y = torch.zeros(4, 16)
    monkeypatch.setattr(T._ops, "distill_loss", lambda x, *a: (x.sum(1), torch.zeros(4, 8, dtype=torch.float64)))
    monkeypatch.setattr(T._ops, "distill_loss_bwd", lambda x, *a: x * 2)
    x = torch.randn(4, 16, requires_grad=True)
    (d,) = torch.autograd.grad(T.distill_loss(x, y, y).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        (d.sum() + x.square().sum()).backward()

    monkeypatch.setattr(T._ops, "linear_act_fwd_train", lambda x, w, *a: (x @ w.t(), x @ w.t(), x[0].float(), x[0].float()))
    monkeypatch.setattr(T._ops, "linear_act_bwd", lambda dy, z, x, w, *a, **k: (dy @ w, dy.t() @ x, None))
    x, w = torch.randn(4, 8, dtype=bf, requires_grad=True), torch.randn(16, 8, dtype=bf, requires_grad=True)
    d = torch.autograd.grad(T.linear_act(x, w).square().sum(), (x, w), create_graph=True)
    for part in d:
        with pytest.raises(RuntimeError, match="no second derivative"):
            (part.sum() + x.square().sum()).backward(retain_graph=True)
    T.linear_act(x, w).square().sum().backward()  # the first is as it was
    assert x.grad.grad_fn is None and torch.equal(w.grad, d[1].detach())


@pytest.mark.parametrize("lead,N,K", [((3,), 16, 0), ((2, 3), 0, 8), ((2, 0), 16, 8), ((0,), 0, 0), ((), 16, 8)])
def test_empty_dimensions(forwards, monkeypatch, lead, N, K):
    """No columns in, none out, no rows, and a single vector: shapes forward and backward."""
    def bwd(dy, z, x, w, *a, **k):
        return torch.zeros_like(x), torch.zeros_like(w), torch.zeros(w.shape[0])

    monkeypatch.setattr(T._ops, "linear_act_bwd", bwd)
    x, w = torch.zeros(*lead, K, dtype=bf, requires_grad=True), torch.zeros(N, K, dtype=bf, requires_grad=True)
    b, r = torch.zeros(N, dtype=bf, requires_grad=True), torch.zeros(*lead, N, dtype=bf, requires_grad=True)
    y = T.linear_act(x, w, b, "silu", r)
    assert y.shape == (*lead, N)
    grads = torch.autograd.grad(y, (x, w, b, r), torch.ones_like(y))
    assert [g.shape for g in grads] == [x.shape, w.shape, b.shape, r.shape]
    with torch.no_grad():
        assert T.linear_act(x, w, b, "silu", r).shape == (*lead, N)
