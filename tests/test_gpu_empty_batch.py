"""The linear chains with an empty batch (or no outputs), INT8 and FP8: the column maxima
that the forward hands to the backward are written, and the gradients are 0, with the
allocator's blocks full of NaN."""
import pytest
import torch

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf = torch.bfloat16


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(bf)


def leave_nan_behind(*sizes):
    held = [torch.full((n,), float("nan"), device="cuda") for n in sizes for _ in range(4)]
    del held


@pytest.mark.parametrize("fmt", ["rne", "sr", "fp8"])
@pytest.mark.parametrize("M,N,K", [(0, 32, 64), (32, 0, 64), (0, 0, 16), (0, 16, 20000), (16, 0, 20000)])
def test_maxima_and_gradients_of_empty_operands(M, N, K, fmt):
    X, W, dY = randn(1, M, K), randn(2, N, K), randn(3, M, N)
    leave_nan_behind(K, K, 4096, 1 << 16)
    if fmt == "fp8":
        Y, cx, cw = i8.linear_fwd_fp8_colmax(X, W)
        dX, dW = i8.linear_bwd_fp8(dY, X, W, colmax_x=cx, colmax_w=cw)
    else:
        Y, cx, cw = i8.linear_fwd_colmax(X, W, fmt, 3, 4)
        dX, dW = i8.linear_bwd(dY, X, W, fmt, 3, 4, colmax_x=cx, colmax_w=cw)
    assert Y.shape == (M, N)
    assert torch.equal(cx, X.abs().amax(0).float() if M else torch.zeros(K, device="cuda"))
    assert torch.equal(cw, W.abs().amax(0).float() if N else torch.zeros(K, device="cuda"))
    assert torch.equal(dX, torch.zeros_like(X)) and torch.equal(dW, torch.zeros_like(W))


@pytest.mark.parametrize("fp8", [False, True])
def test_empty_batch_through_the_module(fp8):
    from int8_mixed_precision_rowwise_amd import training
    m = training.Int8MixedPrecisionLinear(64, 32, training.Int8MixedPrecisionConfig(fp8=fp8), device="cuda")
    leave_nan_behind(64, 4096, 1 << 16)
    m(torch.zeros(0, 64, dtype=bf, device="cuda", requires_grad=True)).sum().backward()
    assert torch.equal(m.weight.grad, torch.zeros_like(m.weight))
