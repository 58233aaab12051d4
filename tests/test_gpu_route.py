"""Routing on the GPU: choices, places and offsets equal, weights and gradients against 64 bits."""
import numpy as np
import pytest
import torch

from . import block_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
inf, nan = float("inf"), float("nan")


def randn(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# exp and the reciprocal sigmoid are good to a few fp32 steps (expf to 1, the sum of up to 1024 terms to 10 in
# a tree of adds over lanes and 16 in a lane, the quotient to 1), and exp's argument x - m, rounded, to |x - m| < 10
# half steps: 40 half steps in all
REL = 40 * 2.0**-24


def check_route(x, k, score, normalize):
    r = i8.expert_route(x, k, score=score, normalize=normalize)
    w, experts, places, rows, offsets = ref.route(ref.to64(x), k, score, normalize)
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.places.cpu().numpy(), places)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    got = ref.to64(r.weights)
    assert np.array_equal(np.isnan(got), np.isnan(w))
    ok = ~np.isnan(w)
    assert (np.abs(got - w)[ok] <= REL * np.abs(w)[ok] + 2.0**-126).all()
    return r


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 3, 3), (7, 64, 6), (255, 8, 2), (256, 63, 4), (257, 65, 5), (300, 256, 8),
                                   (100, 257, 3), (50, 1024, 32), (1000, 16, 16), (3001, 40, 4)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_route(T, E, k, dtype):
    x = randn(T + E, T, E, dtype=dtype)
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            check_route(x, k, score, normalize)


@pytest.mark.parametrize("E", [68, 72, 128, 132, 208, 264, 512, 516, 528, 1000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_lanes_of_many_experts(E, dtype):
    """Each number of scores a lane, read whole and one by one, with ties; gradients against the formula."""
    T, k = 45, 6
    x = (4 * randn(E, T, E)).round().div(4).to(dtype)
    x[3], x[4, 5:] = -inf, -inf
    g = randn(E + 1, T, k)
    for score, normalize in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        r = check_route(x, k, score, normalize)
        d = i8.expert_route_bwd(x, r.experts, g, score=score, normalize=normalize)
        e, dw = r.experts.cpu().numpy(), ref.to64(g)
        want = ref.route_grad(ref.to64(x), e, dw, score, normalize)
        # as in test_route_gradient: differences of terms of size |g| w, then one rounding
        scale = np.abs(dw).sum(1, keepdims=True)
        p = np.abs(ref.route_grad(ref.to64(x), e, np.abs(dw), "sigmoid", False)) if score == "sigmoid" else 1.0
        err = np.abs(ref.to64(d) - want)
        assert (err <= half_step(dtype) * np.abs(want) + 4 * REL * scale * np.maximum(p, 1.0) + (2.0**-25 if dtype == torch.float16 else 0)).all()


def test_many_tokens():
    check_route(randn(1, 70001, 8), 2, "softmax", True)  # blocks of more than 256 tokens


def test_equal_scores_and_missing_experts():
    x = randn(1, 400, 24).round()  # many ties
    x[:, 5] = -inf
    x[10] = -inf
    x[11, 1:] = -inf
    x[12] = 0.0
    x[13] = 1e30
    x[14] = -1e30
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            r = check_route(x, 4, score, normalize)
            assert r.experts[10].tolist() == [-1] * 4 and r.weights[10].tolist() == [0.0] * 4
            assert r.experts[12].tolist() == [0, 1, 2, 3]
    check_route(torch.full((300, 4), -inf, device="cuda"), 2, "softmax", True)


def test_scores_that_are_not_finite():
    x = randn(1, 20, 24)
    x[3, 7], x[4, 8], x[5] = nan, inf, nan
    for score in ("softmax", "sigmoid"):
        check_route(x, 3, score, True)
    d = i8.expert_route_bwd(x, i8.expert_route(x, 3).experts, randn(2, 20, 3))
    bad = torch.zeros(20, dtype=torch.bool, device="cuda")
    bad[3:6] = True
    assert bool(d[bad].isnan().all()) and not bool(d[~bad].isnan().any())


def test_views_and_no_tokens():
    x = randn(1, 50, 40)
    a, b = i8.expert_route(x[:, 3:33], 3), i8.expert_route(x[:, 3:33].contiguous(), 3)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    r = i8.expert_route(torch.zeros(0, 5, device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 6 and r.rows.numel() == 0 and r.weights.shape == (0, 2)
    assert i8.expert_route_bwd(torch.zeros(0, 5, device="cuda"), r.experts, r.weights).shape == (0, 5)


@pytest.mark.parametrize("E,k", [(1, 1), (5, 5), (64, 6), (200, 8), (1000, 3)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient(E, k, dtype, score, normalize):
    T = 70
    x = randn(E, T, E, dtype=dtype)
    x[3] = -inf
    x[4, E // 2:] = -inf
    dw = randn(2, T, k)
    r = i8.expert_route(x, k, score=score, normalize=normalize)
    d = i8.expert_route_bwd(x, r.experts, dw, score=score, normalize=normalize)
    assert d.dtype == dtype
    x64, e, g = ref.to64(x), r.experts.cpu().numpy(), ref.to64(dw)
    want = ref.route_grad(x64, e, g, score, normalize)
    # terms of size |g| w: differences of them are good to REL of the largest, then one rounding
    scale = np.abs(g).sum(1, keepdims=True)
    p = np.abs(ref.route_grad(x64, e, np.abs(g), "sigmoid", False)) if score == "sigmoid" else 1.0
    err = np.abs(ref.to64(d) - want)
    assert (err <= half_step(dtype) * np.abs(want) + 4 * REL * scale * np.maximum(p, 1.0) + (2.0**-25 if dtype == torch.float16 else 0)).all()
    assert not d[3].any()
    if dtype == torch.float32:  # against differences of the weights in 64 bits
        rng = np.random.default_rng(1)
        v = np.where(np.isfinite(x64), rng.standard_normal(x64.shape), 0)
        h = 1e-5

        def f(z):
            w = np.zeros((T, k))
            for t in range(T):
                at = e[t][e[t] >= 0]
                if at.size == 0:
                    continue
                s = 1 / (1 + np.exp(-z[t, at])) if score == "sigmoid" else np.exp(z[t, at])
                total = s.sum() if normalize else 1.0 if score == "sigmoid" else np.exp(z[t]).sum()
                w[t, :at.size] = s / total
            return (w * g).sum()

        diff = (f(x64 + h * v) - f(x64 - h * v)) / (2 * h)
        assert abs(diff - (ref.to64(d) * v).sum()) <= 1e-6 * (1 + np.abs(g).sum())


# ------------------------------------------------------------------ combination


def combine_ref(Y, places, w, residual=None):
    y, p = ref.to64(Y), places.cpu().numpy()
    R = y.shape[0]
    ok = (p >= 0) & (p < R)
    z = np.where(ok[..., None], y[np.clip(p, 0, R - 1)], 0.0)
    weights = np.ones(p.shape) if w is None else ref.to64(w)
    terms = z * weights[..., None]
    r = 0.0 if residual is None else ref.to64(residual)
    return terms.sum(1) + r, np.abs(terms).sum(1) + np.abs(r), z


def random_places(T, k, R, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randperm(max(R, T * k), generator=g)[:T * k].view(T, k).to(torch.int32)
    p[torch.rand(T, k, generator=g) < 0.1] = -1
    return torch.where(p < R, p, -1).cuda()


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 2, 8), (5, 3, 13), (37, 4, 2040), (300, 2, 512), (64, 8, 520), (2, 32, 24)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_combine(T, k, N, dtype):
    R = T * k + 3
    Y, w, places, dout = randn(1, R, N, dtype=dtype), randn(2, T, k), random_places(T, k, R, T), randn(3, T, N, dtype=dtype)
    res = randn(4, T, N, dtype=dtype)
    eps, tiny = half_step(dtype), 2.0**-25 if dtype == torch.float16 else 0
    for weights, residual in ((w, None), (None, res), (w, res)):
        out = i8.expert_combine(Y, places, weights, residual)
        want, size, _ = combine_ref(Y, places, weights, residual)
        assert (np.abs(ref.to64(out) - want) <= eps * np.abs(want) + (k + 2) * 2.0**-24 * (1 + eps) * size + tiny).all()
    inplace = res.clone()
    assert i8.expert_combine(Y, places, w, inplace, out=inplace) is inplace and torch.equal(inplace, out)
    # gradients
    rows = torch.full((R,), -1, dtype=torch.int32)
    p = places.cpu()
    for t in range(T):
        for j in range(k):
            if p[t, j] >= 0:
                rows[p[t, j]] = t
    dY, dw = i8.expert_combine_bwd(dout, Y, places, w, rows=rows.cuda())
    plain, _ = i8.expert_combine_bwd(dout, Y, places, w)
    assert torch.equal(dY, plain)
    _, _, z = combine_ref(Y, places, w)
    d, ww = ref.to64(dout), ref.to64(w)
    wanted = np.zeros((R, N))
    for t in range(T):
        for j in range(k):
            if p[t, j] >= 0:
                wanted[p[t, j]] = ww[t, j] * d[t]
    assert (np.abs(ref.to64(dY) - wanted) <= (eps + 2.0**-24) * np.abs(wanted) * (1 + eps) + tiny).all()
    terms = z * d[:, None]
    assert (np.abs(ref.to64(dw) - terms.sum(2)) <= (N // 64 + 12) * 2.0**-24 * np.abs(terms).sum(2)).all()
    only, none = i8.expert_combine_bwd(dout, Y, places, None, rows=rows.cuda(), want_dweights=False)
    assert none is None
    wanted = np.where((rows >= 0).numpy()[:, None], d[rows.clamp_min(0).numpy()], 0)
    assert np.array_equal(ref.to64(only), wanted)
    none, again = i8.expert_combine_bwd(dout, Y, places, w, want_dy=False)
    assert none is None and torch.equal(again, dw)


def test_combine_of_views_and_given_outputs():
    Y, places, w = randn(1, 40, 64), random_places(10, 3, 40, 1), randn(2, 10, 3)
    store = randn(5, 40, 70)
    store[:, 3:67] = Y
    assert torch.equal(i8.expert_combine(store[:, 3:67], places, w), i8.expert_combine(Y, places, w))
    out = torch.full((10, 66), 7.0, device="cuda")
    i8.expert_combine(Y, places, w, out=out[:, 1:65])
    assert torch.equal(out[:, 1:65], i8.expert_combine(Y, places, w)) and bool((out[:, 0] == 7).all()) and bool((out[:, 65] == 7).all())
    # places outside the rows add nothing, and a given dY keeps the rows that none names
    p = torch.tensor([[0, 40], [-5, 2**31 - 1]], dtype=torch.int32, device="cuda")
    assert torch.equal(i8.expert_combine(Y, p), torch.stack((Y[0], torch.zeros_like(Y[0]))))
    dY = torch.full_like(Y, 7.0)
    dout = randn(3, 2, 64)
    i8.expert_combine_bwd(dout, Y, p, dY=dY)
    assert torch.equal(dY[0], dout[0]) and bool((dY[1:] == 7).all())


# ------------------------------------------------------------------ together


def test_a_layer_of_experts_and_its_replay():
    """Route, first products, second products and combination as a layer makes them, forward and backward,
    eagerly and from a graph, against the parts expert by expert."""
    T, E, k, D, H = 50, 6, 2, 136, 72
    bf = torch.bfloat16
    X, W1, W2 = randn(1, T, D, dtype=bf), 0.1 * randn(2, E, H, D, dtype=bf), 0.1 * randn(3, E, D, H, dtype=bf)
    logits, dout = randn(4, T, E), randn(5, T, D, dtype=bf)
    logits[7] = -inf  # padding
    q1, q2 = i8.quantize_block_weight(W1), i8.quantize_block_weight(W2)

    def layer():
        r = i8.expert_route(logits, k)
        h = i8.expert_linear_fwd(X, *q1, r.offsets, rows=r.rows)
        y = i8.expert_linear_fwd(h, *q2, r.offsets)
        out = i8.expert_combine(y, r.places, r.weights, residual=X)
        dy, dw = i8.expert_combine_bwd(dout, y, r.places, r.weights, rows=r.rows)
        dh, dw2 = i8.expert_linear_bwd(dy, h, *q2, r.offsets)
        dxs, dw1 = i8.expert_linear_bwd(dh, X, *q1, r.offsets, rows=r.rows)
        dx = i8.expert_combine(dxs, r.places, None, residual=dout)
        return [out, dx, dw1, dw2, i8.expert_route_bwd(logits, r.experts, dw), h, y, dy, dh, dxs, *r]

    out, dx, dw1, dw2, dl, h, y, dy, dh, dxs, weights, experts, places, rows, offsets = layer()
    off, x = offsets.tolist(), ref.to64(X)
    assert off[-1] == k * (T - 1) and torch.equal(out[7], X[7]) and torch.equal(dx[7], dout[7]) and not dl[7].any()
    tok = rows.cpu().numpy()
    for e in range(E):
        at = slice(off[e], off[e + 1])
        ref.close(h[at], *ref.forward(x[tok[at]], ref.to64(W1[e])), "h")
        ref.close(y[at], *ref.forward(ref.to64(h[at]), ref.to64(W2[e])), "y")
        ref.close(dh[at], *ref.grad_input(ref.to64(dy[at]), ref.to64(W2[e])), "dh")
        ref.close(dw2[e], *ref.grad_weight(ref.to64(dy[at]), ref.to64(h[at])), "dW2")
        ref.close(dxs[at], *ref.grad_input(ref.to64(dh[at]), ref.to64(W1[e])), "dX rows")
        ref.close(dw1[e], *ref.grad_weight(ref.to64(dh[at]), x[tok[at]]), "dW1")
    assert not bool(h[off[-1]:].any()) and not bool(dy[off[-1]:].any())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = layer()
    for rep in range(3):
        X.copy_(randn(10 + rep, T, D, dtype=bf))
        logits.copy_(randn(20 + rep, T, E))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, layer()))
