"""Sigmoid weights over their sum where all of a token's scores lie far below zero: each sigmoid alone is below
fp32's numbers there, their shares are not."""
import numpy as np
import pytest
import torch

from . import block_ref as ref
from .test_gpu_route_gradient import REL, check, shares

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("low", [-15.0, -80.0, -100.0, -300.0, -690.0])
@pytest.mark.parametrize("E,k", [(8, 3), (100, 4), (300, 6)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_shares_of_small_sigmoids(low, E, k, dtype):
    """Weights and gradients; in a third of the tokens one score is near zero."""
    T = 45
    x = low + 5 * torch.rand(T, E, generator=torch.Generator().manual_seed(E)).cuda()
    x[::3, E // 2] = torch.linspace(-12, 12, 15).cuda()
    x = x.to(dtype)
    r = i8.expert_route(x, k, score="sigmoid", normalize=True)
    w, _, _ = shares(ref.to64(x), r.experts.cpu().numpy(), "sigmoid", True)
    assert (np.abs(ref.to64(r.weights) - w) <= REL * w + 2.0**-126).all()
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    check(x, r.experts, g, "sigmoid", True)
    check(x, r.experts, g, "sigmoid", False)


def test_no_share_of_nothing():
    """Below -700 a sigmoid counts as 0, and so do the weights over a sum of such."""
    x = torch.full((4, 6), -1e30, device="cuda")
    x[1], x[2], x[3, 1:] = -700.5, torch.linspace(-720, -701, 6).cuda(), -800.0
    x[3, 0] = -3.0
    r = i8.expert_route(x, 2, score="sigmoid", normalize=True)
    assert not r.weights[:3].any() and r.weights[3].tolist() == [1.0, 0.0]
    d = i8.expert_route_bwd(x, r.experts, torch.ones(4, 2, device="cuda"), score="sigmoid", normalize=True)
    assert not d.any()
