"""The routing's weights and gradients, element by element, where scores lie far from zero or from each other."""
import numpy as np
import pytest
import torch

from . import block_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

inf = float("inf")
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
FORMS = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]


def shares(x, experts, score, normalize):
    """(weights of the taken [T, k], complements 1 - sigmoid, shares of all [T, E]) in 64 bits, from the logarithms."""
    at = np.take_along_axis(x, np.maximum(experts, 0), 1)
    ok = experts >= 0
    log = np.where(ok, -np.logaddexp(0, -at) if score == "sigmoid" else at, -np.inf)
    over = x if score == "softmax" and not normalize else log
    top = over.max(1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    total = np.exp(over - top).sum(1, keepdims=True)
    total = np.where(total > 0, total, 1.0)
    if score == "sigmoid" and not normalize:
        top, total = 0.0, 1.0
    return np.exp(log - top) / total, np.exp(-np.logaddexp(0, at)), np.exp(x - top) / total


def gradient(x, experts, g, score, normalize):
    """(gradient, the size of the terms it is a sum of) in 64 bits."""
    w, c, all_w = shares(x, experts, score, normalize)
    ok = experts >= 0
    g = np.where(ok, g, 0.0)
    inner, inner_size = (g * w).sum(1, keepdims=True), (np.abs(g) * w).sum(1, keepdims=True)
    d, size = np.zeros_like(x), np.zeros_like(x)
    if score == "sigmoid":
        taken, taken_size = ((g - inner) * w * c, (np.abs(g) + inner_size) * w * c) if normalize else (g * w * c, np.abs(g) * w * c)
    else:
        taken, taken_size = w * (g - inner), w * (np.abs(g) + inner_size)
        if not normalize:
            d, size = -all_w * inner, all_w * inner_size
    for t, j in zip(*np.nonzero(ok)):
        d[t, experts[t, j]], size[t, experts[t, j]] = taken[t, j], taken_size[t, j]
    return d, size


# In half steps of fp32 (2^-24): exp to 2 and its argument, rounded, to |x - m| < 16 of them; a sum of up to 1024
# exponentials to 10 in a tree over lanes and 16 in a lane; a quotient, a complement's sum and each product to 1.  At most 50 for
# a weight, the same for <g, w>, and 4 for the difference and the products that follow.
REL = 110 * 2.0**-24


def check(x, experts, g, score, normalize):
    d = i8.expert_route_bwd(x, experts, g, score=score, normalize=normalize)
    want, size = gradient(ref.to64(x), experts.cpu().numpy(), ref.to64(g), score, normalize)
    err = np.abs(ref.to64(d) - want)
    half = torch.finfo(x.dtype).eps / 2
    # below a type's smallest normal number a rounding is off by half its smallest step (fp16 2^-25, the others about 2^-126 at most)
    bound = REL * size + half * (np.abs(want) + REL * size) + (2.0**-25 if x.dtype == torch.float16 else 2.0**-126)
    assert (err <= bound).all(), (score, normalize, int((err > bound).sum()), float((err / bound).max()))


def randn(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("E,k", [(24, 4), (100, 3), (300, 8)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sigmoid_of_confident_scores(E, k, dtype, normalize):
    """Scores from 10 to 40 in both directions: a gradient of 4e-8 is as good as one of 0.25."""
    T = 60
    x = 10 + 30 * torch.rand(T, E, generator=torch.Generator().manual_seed(E)).cuda()
    x[T // 3:] *= torch.where(torch.rand(T - T // 3, E, generator=torch.Generator().manual_seed(1)) < 0.95, -1.0, 1.0).cuda()
    x = x.to(dtype)
    check(x, i8.expert_route(x, k, score="sigmoid", normalize=normalize).experts, randn(2, T, k), "sigmoid", normalize)


@pytest.mark.parametrize("score,normalize", FORMS)
@pytest.mark.parametrize("E,k", [(1, 1), (5, 5), (64, 6), (100, 4), (200, 8), (528, 6), (1000, 3), (1000, 32)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_each_element(E, k, dtype, score, normalize):
    """Every expert's gradient to its own size, the untaken ones' of a softmax over all too."""
    T = 50
    x = (2 * randn(E, T, E)).clamp(-6, 6).to(dtype)
    x[3] = -inf
    x[4, E // 2:] = -inf
    check(x, i8.expert_route(x, k, score=score, normalize=normalize).experts, randn(2, T, k), score, normalize)
