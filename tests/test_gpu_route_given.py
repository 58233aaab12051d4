"""The routing's gradient for a choice of experts that is not the largest scores', as another rule of choosing gives it."""
import pytest
import torch

from .test_gpu_route_gradient import FORMS, check, randn

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("score,normalize", FORMS)
@pytest.mark.parametrize("E", [24, 100, 300, 1000])
@pytest.mark.parametrize("above", [0.0, 30.0, 90.0, 300.0])
def test_experts_far_below_the_largest_score(E, above, score, normalize):
    """One expert's score is far above all, and nobody takes it: the weights are shares of the taken ones' sum."""
    T, k = 40, 4
    x = randn(E, T, E).clamp(-6, 6)
    x[:, 7] += above
    experts = torch.rand(T, E, generator=torch.Generator().manual_seed(1))
    experts[:, 7] = -1  # never among the largest
    experts = experts.topk(k, 1).indices.to(torch.int32).cuda()
    experts[5, 2:] = -1
    check(x, experts, randn(2, T, k), score, normalize)
