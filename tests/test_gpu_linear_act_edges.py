"""Edges of the linears with an epilogue on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf = torch.bfloat16


def randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(bf)


def leave_nan_behind(*sizes):
    """Blocks full of NaN in the allocator's cache, for the calls' own tensors to be cut from."""
    held = [torch.full((n,), float("nan"), device="cuda") for n in sizes for _ in range(4)]
    del held


@pytest.mark.parametrize("K", [16, 264, 20000])
@pytest.mark.parametrize("M,N", [(0, 24), (24, 0), (0, 0)])
def test_empty_operands_have_column_maxima(M, N, K):
    X, W, bias = randn(1, M, K), randn(2, N, K), randn(3, N)
    for rounding in ("rne", "sr"):
        leave_nan_behind(K, K, 4096, 1 << 16)
        Y, Z, cx, cw = i8.linear_act_fwd_train(X, W, bias=bias, activation="gelu", rounding=rounding)
        assert torch.equal(cx, X.abs().amax(0).float() if M else torch.zeros(K, device="cuda"))
        assert torch.equal(cw, W.abs().amax(0).float() if N else torch.zeros(K, device="cuda"))
        dX, dW, db = i8.linear_act_bwd(Y, Z, X, W, "gelu", want_dbias=True, colmax_x=cx, colmax_w=cw, rounding=rounding)
        assert torch.equal(dX, torch.zeros_like(X)) and torch.equal(dW, torch.zeros_like(W)) and torch.equal(db, torch.zeros(N, device="cuda"))


def test_empty_batch_through_autograd():
    from int8_mixed_precision_rowwise_amd import training
    w, b = randn(2, 24, 40).requires_grad_(), randn(3, 24).requires_grad_()
    x = randn(1, 0, 40).requires_grad_()
    leave_nan_behind(40, 4096, 1 << 16)
    training.linear_act(x, w, b, "silu").sum().backward()
    assert torch.equal(w.grad, torch.zeros_like(w)) and torch.equal(b.grad, torch.zeros_like(b)) and x.grad.shape == (0, 40)


@pytest.mark.parametrize("M,N,K,pitch", [(16500, 260, 64, 1 << 24), (16500, 260, 64, 1 << 23), (100, 130, 40, (1 << 25) + 16), (200, 7, 520, 1 << 28)])
def test_weight_rows_far_apart(M, N, K, pitch):
    """Views whose rows lie further apart than a tile's 32-bit offsets reach: the bits of dense weights."""
    X, W, bias, R = randn(1, M, K), randn(2, N, K), randn(3, N), randn(4, M, (N + 7) // 8 * 8)[:, :N]
    Wq, ws = i8.quantize_rowwise(W)
    store = torch.empty(N * pitch, dtype=torch.int8, device="cuda")
    far = store.view(N, pitch)[:, :K]
    far.copy_(Wq)
    kw = dict(bias=bias, activation="silu", residual=R)
    want = i8.linear_wq_fwd(X, Wq, ws, **kw)
    out = torch.full((M, N + 1), 7.0, dtype=bf, device="cuda")
    got = i8.linear_wq_fwd(X, far, ws, out=out[:, :N], **kw)
    assert torch.equal(got, want) and bool((out[:, N] == 7).all())


@pytest.mark.parametrize("act", list(i8.ACTIVATIONS)[1:])
def test_derivatives_far_out(act):
    """Finite pre-activations up to the type's largest.  On the right the derivative is 1;
    on the left at most 64 exp(-64), below 2^-80 (and 0 from 10^4 on): the gradients and
    the activation itself are those of 1 and 0 within 16 such numbers."""
    far = torch.tensor([64.0, 1e4, 1.5e13, 1e14, 1e19, 2e19, 1e30, 3.3e38])
    z = torch.cat((far, -far)).to(bf).cuda()
    N = z.numel()
    Z = z.expand(8, N).contiguous()
    dY = torch.ones(8, N, dtype=bf, device="cuda")
    X, W = torch.ones(8, 16, dtype=bf, device="cuda"), torch.eye(N, dtype=bf, device="cuda")
    dX, dW, db = i8.linear_act_bwd(dY, Z, X, W, act, want_dbias=True)
    one = (z > 0).to(bf)
    Y = i8.linear_act_fwd(torch.zeros(8, 16, dtype=bf, device="cuda"), W[:, :16].contiguous(), bias=z, activation=act)
    for got, want in ((db, 8 * one), (dX, one.expand(8, N)), (dW, 8 * one[:, None].expand(N, 16)),
                      (Y, torch.where(z > 0, z, 0.0).expand(8, N))):
        assert bool(((got.double() - want.double()).abs() <= 2.0 ** -76).all())


@pytest.mark.parametrize("act,M,N,K", [("silu", 33, 4107, 2040), ("gelu", 48, 4100, 1001), ("gelu_tanh", 49, 5003, 520),
                                       ("relu", 64, 4099, 8200), ("none", 64, 4097, 24)])
def test_many_few_tokens_over_wide_outputs(act, M, N, K):
    """33 to 64 rows with two column tiles a workgroup: against 64 bits, with kept
    pre-activations, and the same bits over weights quantized once and where rows of the
    output start anywhere."""
    import oracle
    from tests.gpu_util import tensor_bits
    from tests.test_gpu_linear_act import check_forward, product, rows
    X, W = rows(randn(1, M, K)), rows(randn(2, N, K))
    bias, residual = randn(3, N), rows(randn(4, M, N))
    p = product(*oracle.quantize_rowwise(tensor_bits(X), oracle.RNE, 0, 0), *oracle.quantize_rowwise(tensor_bits(W), oracle.RNE, 0, 0))
    kw = dict(bias=bias, activation=act, residual=residual)
    Y, Z, cx, cw = i8.linear_act_fwd_train(X, W, **kw)
    check_forward(p, bias, act, residual, Y, Z)
    assert torch.equal(cx, X.abs().amax(0).float()) and torch.equal(cw, W.abs().amax(0).float())
    Wq, ws = i8.quantize_rowwise(W)
    store = torch.full((M, N + 3), 7.0, dtype=bf, device="cuda")
    got = i8.linear_wq_fwd(X, Wq, ws, out=store[:, :N], **kw)
    assert torch.equal(got, Y) and bool((store[:, N:] == 7).all())
