"""The operators past the sizes that one launch, or 32 bits, hold: against their own
results on parts of the same inputs, and against the definitions on sampled rows."""
import pytest
import torch

from tests import operators_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf = torch.bfloat16


def test_distillation_of_more_rows_than_a_launch_holds():
    """2^23 rows of a workgroup each are 2^32 work items."""
    T, V, k = (1 << 23) + 77, 5, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, V, generator=g, device="cuda").to(bf)
    t = torch.randn(T, k, generator=g, device="cuda").to(bf)
    idx = torch.randint(0, V - 1, (T, 1), generator=g, device="cuda", dtype=torch.int32) + torch.arange(k, device="cuda", dtype=torch.int32)
    lse = (torch.logsumexp(t.float(), 1) + 0.05)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    grad = torch.rand(T, generator=g, device="cuda")
    kw = dict(temperature=1.0, ce_weight=0.5)
    loss, stats = i8.distill_loss(x, t, idx, teacher_lse=lse, labels=labels, **kw)
    d = i8.distill_loss_bwd(x, t, idx, stats, grad, teacher_lse=lse, labels=labels, **kw)
    loss1, d1 = i8.distill_loss_and_grad(x, t, idx, grad, teacher_lse=lse, labels=labels, **kw)
    assert torch.equal(loss, loss1) and torch.equal(d, d1)
    for lo in range(0, T, 1 << 22):
        s = slice(lo, min(T, lo + (1 << 22)))
        part, dp = i8.distill_loss_and_grad(x[s], t[s], idx[s], grad[s], teacher_lse=lse[s], labels=labels[s], **kw)
        assert torch.equal(loss[s], part) and torch.equal(d[s], dp)


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
def test_rotary_of_more_tokens_than_a_launch_holds(pairs):
    """2^28 tokens, 16 a workgroup, are 2^32 work items: in place, against parts of the same call."""
    S = (1 << 28) + 1001
    q = torch.randn(1, S, 1, 2, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.float16)
    pos = torch.arange(S, dtype=torch.int32, device="cuda")
    freqs = i8.rotary_frequencies(2, device="cuda") * 1e-3
    out, _ = i8.rotary(q, None, pos, freqs, pairs=pairs)
    for lo in (0, (1 << 27) - 7, (1 << 28) - 50, (1 << 28) - 16, (1 << 28) + 1):
        part = slice(lo, min(S, lo + 3000))
        assert torch.equal(out[:, part], i8.rotary(q[:, part], None, pos[part], freqs, pairs=pairs)[0])
    want = ref.rotary(q[:, -2000:], pos[-2000:], freqs, pairs)
    tol = ref.rotary_scale(q[:, -2000:], freqs, pairs) * 2.0 ** -22
    tol = tol + ref.half_step(torch.float16) * (want.abs() + tol) + 2.0 ** -24
    assert bool(((out[:, -2000:].cpu().double() - want).abs() <= tol).all())


def test_rotary_in_place_on_heads_major_projections():
    B, HQ, HK, S, D = 3, 4, 2, 37, 64
    packed = torch.randn(B, HQ + 2 * HK, S, D, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(bf)
    q, k = packed[:, :HQ].transpose(1, 2), packed[:, HQ:HQ + HK].transpose(1, 2)
    v = packed[:, HQ + HK:].clone()
    pos, freqs = torch.arange(S, device="cuda") + 100, i8.rotary_frequencies(D, device="cuda")
    want = i8.rotary(q.contiguous(), k.contiguous(), pos, freqs)
    i8.rotary(q, k, pos, freqs, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(packed[:, HQ + HK:], v)


def rows_of(seed, M, N, scale=1.0):
    """bf16 [M, N], made a slab at a time."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(M, N, dtype=bf, device="cuda")
    for lo in range(0, M, 4096):
        out[lo:lo + 4096] = scale * torch.randn(min(4096, M - lo), N, generator=g, device="cuda")
    return out


@pytest.mark.parametrize("tau,ce", [(1.0, 0.0), (2.0, 0.5)])
def test_distillation_past_2_31_logits(tau, ce):
    from tests.test_gpu_distill import check
    T, V, k = 17001, 128256, 24
    assert T * V > 1 << 31
    x = rows_of(1, T, V, 2.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    idx = (torch.randint(0, V, (T, 1), generator=g, device="cuda") + 5003 * torch.arange(k, device="cuda")) % V
    t = (4 + 2 * torch.randn(T, k, generator=g, device="cuda")).to(bf)
    x.scatter_(1, idx, (t.float() + torch.randn(T, k, generator=g, device="cuda")).to(bf))
    lse = (torch.logsumexp(t.double() / tau, 1) + 0.05).float()
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    grad = torch.rand(T, generator=g, device="cuda")
    rows = torch.tensor([0, 1, (1 << 31) // V, (1 << 31) // V + 1, T - 2, T - 1])
    kw = dict(temperature=tau, teacher_lse=lse, labels=labels if ce else None, ce_weight=ce)
    loss, d = i8.distill_loss_and_grad(x, t, idx, grad, **kw)
    check(x, t, idx, tau, lse, labels if ce else None, ce, grad, loss, d, rows)
    loss, stats = i8.distill_loss(x, t, idx, **kw)
    d = i8.distill_loss_bwd(x, t, idx, stats, grad, out=d, **kw)
    check(x, t, idx, tau, lse, labels if ce else None, ce, grad, loss, d, rows)


def test_rotary_past_2_31_elements():
    S, HQ, HK, D = 530001, 28, 4, 128
    packed = rows_of(3, S, (HQ + HK) * D)
    assert packed.numel() > 1 << 31
    q, k = packed[:, :HQ * D].view(1, S, HQ, D), packed[:, HQ * D:].view(1, S, HK, D)
    pos, freqs = torch.arange(S, device="cuda"), i8.rotary_frequencies(D, 500000.0, device="cuda")
    at = torch.tensor([0, 1, (1 << 31) // ((HQ + HK) * D), S - 2, S - 1]).cuda()
    keep = [h[:, at].clone() for h in (q, k)]
    a, b = i8.rotary(q, k, pos, freqs)
    for x, y in zip(keep, (a, b)):
        want = ref.rotary(x, pos[at], freqs, "half")
        tol = ref.rotary_scale(x, freqs, "half") * 2.0 ** -22
        tol = tol + ref.half_step(bf) * (want.abs() + tol) + 2.0 ** -133
        assert bool(((y[:, at].cpu().double() - want).abs() <= tol).all())
    i8.rotary(q, k, pos, freqs, out_q=q, out_k=k)
    assert torch.equal(q, a) and torch.equal(k, b)


def test_linear_past_2_31_outputs():
    """Forward with the pre-activation kept, and the backward that reads it: sampled rows and
    columns.  ReLU and gradients of powers of two, so dZ is known exactly; a product's
    sum is exact, its conversion and two scales are three roundings to fp32 (2^-22) and one to bf16."""
    import oracle
    from tests.gpu_util import tensor_bits
    from tests.test_gpu_linear_act import check_forward, product
    M, N, K = 65601, 32776, 16
    assert M * N > 1 << 31
    X, W, bias = rows_of(4, M, K), rows_of(5, N, K), rows_of(6, 1, N)[0]
    R = rows_of(7, M, N)
    Y, Z, cx, cw = i8.linear_act_fwd_train(X, W, bias=bias, activation="relu", residual=R)
    at = torch.tensor([0, 1, (1 << 31) // N, (1 << 31) // N + 1, M - 2, M - 1])
    on = at.cuda()
    qw, sw = oracle.quantize_rowwise(tensor_bits(W), oracle.RNE, 0, 0)
    p = product(*oracle.quantize_rowwise(tensor_bits(X[on]), oracle.RNE, 0, 0), qw, sw)
    check_forward(p, bias, "relu", R[on], Y[on], Z[on])
    Wq, ws = i8.quantize_rowwise(W)
    assert torch.equal(i8.linear_wq_fwd(X, Wq, ws, bias=bias, activation="relu", residual=R, out=R.clone()), Y)
    del Y, R
    g = torch.Generator(device="cuda").manual_seed(8)
    dY = torch.empty(M, N, dtype=bf, device="cuda")
    for lo in range(0, M, 4096):
        n = min(4096, M - lo)
        dY[lo:lo + n] = torch.exp2(torch.randint(-8, 3, (n, N), generator=g, device="cuda").float())
    dX, dW, db = i8.linear_act_bwd(dY, Z, X, W, "relu", want_dbias=True, colmax_x=cx, colmax_w=cw)
    half = ref.half_step(bf)

    def near(got, want):
        tol = 2.0 ** -22 * want.abs()
        assert bool(((got.cpu().double() - want).abs() <= tol + half * (want.abs() + tol) + 2.0 ** -126).all())

    rowz = torch.where(Z[on] > 0, dY[on], 0)
    wt, xt = W.t().contiguous(), X.t().contiguous()
    near(dX[on], product(*oracle.quantize_rowwise(tensor_bits(rowz), oracle.RNE, 0, 0), *oracle.quantize_rowwise(tensor_bits(wt), oracle.RNE, 0, 0)))
    cols = torch.tensor([0, 1, 17, N // 2, N - 2, N - 1]).cuda()
    colz = torch.where(Z[:, cols] > 0, dY[:, cols], 0).t().contiguous()
    near(dW[cols], product(*oracle.quantize_rowwise(tensor_bits(colz), oracle.RNE, 0, 0), *oracle.quantize_rowwise(tensor_bits(xt), oracle.RNE, 0, 0)))
    want = colz.double().sum(1).cpu()  # some 2^16 additions in fp32, in 256 bands and 8 waves: below 2^9 a chain
    assert bool(((db[cols].cpu().double() - want).abs() <= 2.0 ** -15 * want).all())
