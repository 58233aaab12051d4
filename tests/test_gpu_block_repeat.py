"""The same call gives the same bits, in tiles of either size, with contractions in parts and over experts."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf = torch.bfloat16


def randn(seed, *shape, std=1.0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").mul_(std).to(bf)


def same_bits(call):
    """Four times, each into other memory, with other work between."""
    want = [t.clone() for t in call()]
    keep = []
    for rep in range(3):
        keep.append(torch.randn(1 << (18 + rep), device="cuda").sort())
        got = call()
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))
        keep.append(got)


@pytest.mark.parametrize("M,N,K", [(1, 14336, 4096), (33, 5632, 2048), (64, 4096, 14336), (1000, 1000, 1000), (8192, 5632, 2048), (8011, 2048, 5632)])
def test_linear(M, N, K):
    X, dY = randn(1, M, K), randn(3, M, N, std=1e-3)
    q = i8.quantize_block_weight(randn(2, N, K, std=0.02))
    same_bits(lambda: [i8.linear_block_fwd(X, *q), *i8.linear_block_bwd(dY, X, *q)])


@pytest.mark.parametrize("counts,N,K", [([2, 0, 1, 7], 1024, 2048), ([130, 0, 77, 50, 1], 1000, 712), ([1400, 0, 600, 3000, 0, 260], 2056, 2056)])
def test_experts(counts, N, K):
    R, tokens = sum(counts) + 9, 300
    X, dY = randn(1, tokens, K), randn(3, R, N, std=1e-3)
    q = i8.quantize_block_weight(randn(2, len(counts), N, K, std=0.02))
    offsets = torch.tensor(np.cumsum([0, *counts]), dtype=torch.int32, device="cuda")
    rows = ((torch.arange(R, dtype=torch.int32) * 7) % tokens).cuda()
    same_bits(lambda: [i8.expert_linear_fwd(X, *q, offsets, rows), *i8.expert_linear_bwd(dY, X, *q, offsets, rows)])
