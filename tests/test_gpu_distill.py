"""Distillation loss on the GPU against the definition in 64 bits.

Tolerances.  An exponential 2^a relative to the row's maximum is off by the
rounding of its argument (|a| 2^-24 ln 2, with the rounding of 1 / temperature
|a| 2^-24 more, and |a| below 100 wherever 2^a matters), by the instruction
(2^-23) and, in a sum, by a few dozen fp32 additions (64 x 2^-24): together under
2^-17 of the value.  A loss's logarithms carry that once per class of mass 1;
each term of a gradient carries it, before the terms cancel; then one rounding
to the output's type."""
import pytest
import torch

from tests import operators_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf, fp, f32 = torch.bfloat16, torch.float16, torch.float32
REL = 2.0 ** -17
TINY = {bf: 2.0 ** -120, fp: 2.0 ** -24, f32: 2.0 ** -120}


def inputs(T, V, k, dtype, seed, tau=1.0, rest=False, idx_dtype=torch.int32, t_dtype=bf):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = 2.0 * r(T, V)
    order = torch.argsort(torch.rand(T, V, generator=g, device="cuda"), 1)[:, :k] if V * T < 1 << 22 else \
        (torch.randint(0, V, (T, 1), generator=g, device="cuda") + torch.arange(k, device="cuda") * max(1, V // max(k, 1) - 1)) % V
    t = 12.0 - 2.0 * torch.log1p(torch.arange(k, device="cuda").float()) + 0.7 * r(T, k)
    x.scatter_(1, order, t + 1.5 * r(T, k))
    t = t.to(t_dtype)
    lse = (torch.logsumexp(t.double() / tau, 1) + 0.05).float() if rest and k else None
    idx = order.to(idx_dtype)
    if T > 2 and k > 1:
        idx[1, k // 2:] = -1  # fewer entries than there is room for
        idx[2] = -1  # none
    if T > 4 and k > 2:
        idx[4, 1] = V  # no such class
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    if T > 3:
        labels[3] = -100
    if T > 5 and k:
        labels[5] = idx[5, 0].long()  # the label among the kept
    grad = (0.5 + torch.rand(T, generator=g, device="cuda")) / T * (4096 if dtype == fp else 1)
    return x.to(dtype), t, idx, lse, labels, grad


def check(x, t, idx, tau, lse, labels, ce, grad, loss, d=None, rows=None):
    T = x.shape[0]
    rows = torch.arange(T) if rows is None else rows
    pick = lambda v: None if v is None else v[rows.to(v.device)]  # noqa: E731
    want, dw, scale = ref.distill(pick(x), pick(t), pick(idx), tau, pick(lse), pick(labels), ce, -100, pick(grad))
    got = pick(loss).cpu().double()
    tol = (tau * tau + abs(ce)) * 2 * REL + 2.0 ** -24 * want.abs()
    assert bool(((got == want) | ((got - want).abs() <= tol)).all()), (got, want)  # equal: infinities
    if d is not None:
        gd = pick(d).cpu().double()
        tol = scale * REL
        tol = tol + ref.half_step(x.dtype) * (dw.abs() + tol) + TINY[x.dtype]
        assert d.shape == x.shape and d.dtype == x.dtype
        assert bool(((gd - dw).abs() <= tol).all()), float(((gd - dw).abs() / tol).max())


# T, V, k: one class; rows shorter than a chunk; each of the kernels that hold a row (odd
# lengths, so rows start anywhere in a chunk); segments: few long rows, rows too long to hold
SHAPES = [(1, 1, 1), (3, 5, 3), (9, 500, 20), (7, 4001, 64), (130, 8003, 33), (6, 2000, 600), (130, 32003, 100),
          (129, 64001, 64), (128, 128256, 1024), (2, 128256, 32), (1, 300001, 50), (6, 32000, 0)]
MODES = [(1.0, False, 0.0), (2.0, False, 0.5), (1.5, True, 0.25), (1.0, True, 1.0), (4.0, True, 0.0)]


@pytest.mark.parametrize("tau,rest,ce", MODES)
@pytest.mark.parametrize("dtype", [bf, fp, f32])
@pytest.mark.parametrize("T,V,k", SHAPES)
def test_loss_and_gradient(T, V, k, dtype, tau, rest, ce):
    x, t, idx, lse, labels, grad = inputs(T, V, k, dtype, T + V, tau, rest)
    labels = labels if ce else None
    rows = None if T * V < 1 << 21 else torch.tensor([0, 1, 2, 3, 4, 5, T // 2, T - 1])
    kw = dict(temperature=tau, teacher_lse=lse, labels=labels, ce_weight=ce)
    loss, d = i8.distill_loss_and_grad(x, t, idx, grad, **kw)
    check(x, t, idx, tau, lse, labels, ce, grad, loss, d, rows)
    loss, stats = i8.distill_loss(x, t, idx, **kw)
    d = i8.distill_loss_bwd(x, t, idx, stats, grad, **kw)
    check(x, t, idx, tau, lse, labels, ce, grad, loss, d, rows)


@pytest.mark.parametrize("V,T", [(1003, 6), (40007, 3), (40007, 140)])
@pytest.mark.parametrize("dtype", [bf, f32])
def test_strides_types_and_outputs(dtype, V, T):
    x, t, idx, lse, labels, grad = inputs(T, V, 40, dtype, 3, 1.5, True, torch.int64, f32)
    store = torch.zeros(T * (V + 13) + 3, dtype=dtype, device="cuda")
    view = store[3:].view(T, V + 13)[:, :V]
    view.copy_(x)
    wide_t, wide_i = torch.zeros(T, 50, device="cuda"), torch.zeros(T, 50, dtype=torch.int64, device="cuda")
    wide_t[:, 5:45], wide_i[:, 5:45] = t, idx
    t, idx, lab32 = wide_t[:, 5:45], wide_i[:, 5:45], labels.int()
    out = torch.full((T * (V + 8) + 1,), 7.0, dtype=dtype, device="cuda")
    o = out[1:].view(T, V + 8)[:, :V]
    rows = torch.tensor([0, 1, 2, T - 1])
    kw = dict(temperature=1.5, teacher_lse=lse, labels=lab32, ce_weight=0.5)
    loss, d = i8.distill_loss_and_grad(view, t, idx, grad, out=o, **kw)
    assert d is o
    check(x, t, idx, 1.5, lse, labels, 0.5, grad, loss, d, rows)
    assert bool((out[1:].view(T, V + 8)[:, V:] == 7).all()) and float(out[0]) == 7
    one = torch.tensor(0.25, device="cuda").expand(T)  # a broadcast gradient
    loss, stats = i8.distill_loss(view, t, idx, **kw)
    d = i8.distill_loss_bwd(view, t, idx, stats, one, **kw)
    assert d.stride(0) == view.stride(0)
    check(x, t, idx, 1.5, lse, labels, 0.5, one, loss, d, rows)


@pytest.mark.parametrize("T,V", [(6, 700), (130, 33000), (4, 33000)])
@pytest.mark.parametrize("dtype", [bf, f32])
def test_masked_classes_and_rows_that_are_not_finite(dtype, T, V):
    x, t, idx, lse, labels, grad = inputs(T, V, 16, dtype, 5, 2.0, True)
    keep = torch.rand(T, V, generator=torch.Generator().manual_seed(1)).cuda() < 0.3
    keep.scatter_(1, idx.clamp(0, V - 1).long(), True)
    keep.scatter_(1, labels.clamp_min(0)[:, None], True)
    x = x.masked_fill(~keep, -float("inf"))
    kw = dict(temperature=2.0, teacher_lse=lse, labels=labels, ce_weight=0.5)
    loss, d = i8.distill_loss_and_grad(x, t, idx, grad, **kw)
    rows = torch.tensor([0, 1, 2, T - 1])
    check(x, t, idx, 2.0, lse, labels, 0.5, grad, loss, d, rows)
    assert bool((d[~keep] == 0).all())
    low = x.masked_fill(~keep, torch.finfo(dtype).min / 4)  # masks of the type's lowest values
    loss2, d2 = i8.distill_loss_and_grad(low, t, idx, grad, **kw)
    assert torch.equal(loss, loss2) and torch.equal(d, d2)
    bad = x.clone()
    bad[0, V // 2], bad[1, V - 1] = float("nan"), float("inf")
    loss3, d3 = i8.distill_loss_and_grad(bad, t, idx, grad, **kw)
    assert bool(loss3[:2].isnan().all()) and bool(d3[:2].isnan().all())
    assert torch.equal(loss3[2:], loss[2:]) and torch.equal(d3[2:], d[2:])


def test_nothing_to_do_and_same_bits():
    x, t, idx, lse, labels, grad = inputs(200, 5000, 30, bf, 9)
    empty = i8.distill_loss_and_grad(x[:0], t[:0], idx[:0], grad[:0])
    assert empty[0].shape == (0,) and empty[1].shape == (0, 5000)
    a = i8.distill_loss_and_grad(x, t, idx, grad, labels=labels, ce_weight=1.0)
    b = i8.distill_loss_and_grad(x, t, idx, grad, labels=labels, ce_weight=1.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("tau,rest,ce", MODES)
def test_gradient_against_differences(tau, rest, ce):
    """Along a direction v the fp32 losses' difference quotient is off by h^2 / 6 of
    the third derivative (below 4 |v|^3 / tau + 4 |v|^3 for softmax sums with |v| <= 1)
    and by two losses' tolerance over 2 h."""
    from int8_mixed_precision_rowwise_amd import training
    x, t, idx, lse, labels, _ = inputs(8, 300, 12, f32, 11, tau, rest)
    labels = labels if ce else None
    g = torch.Generator(device="cuda").manual_seed(2)
    v = torch.rand(x.shape, generator=g, device="cuda") * 2 - 1
    leaf = x.clone().requires_grad_()
    loss = training.distill_loss(leaf, t, idx, tau, lse, labels, ce)
    loss.sum().backward()
    along = (leaf.grad.double() * v.double()).sum(1)
    h = 2.0 ** -5
    kw = dict(temperature=tau, teacher_lse=lse, labels=labels, ce_weight=ce)
    up, down = (i8.distill_loss(x + s * h * v, t, idx, **kw)[0].double() for s in (1, -1))
    tol = h * h / 6 * 8 * max(1.0, tau * tau) + (tau * tau + ce) * 4 * REL / (2 * h) + 2.0 ** -24 * up.abs() / h
    assert bool((((up - down) / (2 * h) - along).abs() <= tol).all())


@pytest.mark.parametrize("T,V", [(140, 9001), (3, 70000)])
def test_captured_and_on_another_stream(T, V):
    from int8_mixed_precision_rowwise_amd import training
    x, t, idx, lse, labels, grad = inputs(T, V, 24, bf, 13)
    kw = dict(temperature=2.0, labels=labels, ce_weight=0.5)
    need = max(1, i8.lib.i8mp_distill_workspace_bytes(T, V, 24, 0))
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty_like(x)
    want = i8.distill_loss_and_grad(x, t, idx, grad, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = i8.distill_loss_and_grad(x, t, idx, grad, **kw)
    s.synchronize()
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    graph = torch.cuda.CUDAGraph()
    leaf = x.clone().requires_grad_()
    with torch.cuda.graph(graph):
        loss, d = i8.distill_loss_and_grad(x, t, idx, grad, out=out, workspace=ws, **kw)
        (leaf_grad,) = torch.autograd.grad(training.distill_loss(leaf, t, idx, 2.0, None, labels, 0.5), leaf, grad)
    for seed in range(3):
        x2 = inputs(T, V, 24, bf, 20 + seed)[0]
        x.copy_(x2)
        with torch.no_grad():
            leaf.copy_(x2)
        graph.replay()
        torch.cuda.synchronize()
        want = i8.distill_loss_and_grad(x2, t, idx, grad, **kw)
        l2, stats = i8.distill_loss(x2, t, idx, **kw)
        d2 = i8.distill_loss_bwd(x2, t, idx, stats, grad, **kw)
        assert torch.equal(loss, want[0]) and torch.equal(d, want[1]) and torch.equal(leaf_grad, d2)


# each size of row that a workgroup holds, full to the last chunks
@pytest.mark.parametrize("dtype", [bf, fp, f32])
@pytest.mark.parametrize("T,V,k", [(5, 1003, 20), (5, 2033, 40), (5, 4079, 128), (5, 8171, 300), (5, 16360, 64),
                                   (129, 32747, 9), (129, 49131, 64), (129, 65521, 640), (129, 98281, 64), (129, 131049, 64)])
def test_every_size_of_row(T, V, k, dtype):
    rows = torch.tensor([0, 1, 2, 3, 4, T - 1])
    for tau, ce in ((1.0, 0.0), (2.0, 0.5), (1.5, 0.25)):
        x, t, idx, lse, labels, grad = inputs(T, V, k, dtype, V, tau, True)
        labels = labels if ce else None
        kw = dict(temperature=tau, teacher_lse=lse, labels=labels, ce_weight=ce)
        loss, d = i8.distill_loss_and_grad(x, t, idx, grad, **kw)
        check(x, t, idx, tau, lse, labels, ce, grad, loss, d, rows)


@pytest.mark.parametrize("tau,ce", [(1.0, 0.0), (2.0, 0.5), (1.5, 0.25)])
@pytest.mark.parametrize("T,V", [(9, 700), (130, 33001), (9, 40001)])
@pytest.mark.parametrize("dtype", [bf, f32])
def test_logits_far_from_zero(dtype, T, V, tau, ce):
    """Rows that lie at 2^20 ... 2^60 and at the type's lowest value: nearly every
    exponential is 0 or that of the maximum.  log2(e) / temperature is rounded once
    (2^-24 of a loss) and the loss once; the rest as above."""
    x, t, idx, lse, labels, grad = inputs(T, V, 16, dtype, 8, tau)
    labels = labels if ce else None
    g = torch.Generator(device="cuda").manual_seed(1)
    for r, at in enumerate((2.0 ** 20, -2.0 ** 20, 2.0 ** 22, -2.0 ** 23, 2.0 ** 25, -2.0 ** 60, 2.0 ** 60)):
        x[r] = (at * (1 + torch.randint(0, 3, (V,), generator=g, device="cuda") / 64)).to(dtype)
    x[7] = torch.finfo(dtype).min
    x[8, 5:] = torch.finfo(dtype).min
    rows = torch.arange(9)
    pick = lambda v: None if v is None else v[:9]  # noqa: E731
    want, dw, scale = ref.distill(pick(x), pick(t), pick(idx), tau, None, pick(labels), ce, -100, pick(grad))
    kw = dict(temperature=tau, labels=labels, ce_weight=ce)
    loss, d = i8.distill_loss_and_grad(x, t, idx, grad, **kw)
    loss2, stats = i8.distill_loss(x, t, idx, **kw)
    d2 = i8.distill_loss_bwd(x, t, idx, stats, grad, **kw)
    for lo, gd in ((loss, d), (loss2, d2)):
        tol = (tau * tau + ce) * 2 * REL + 2.0 ** -23 * want.abs()
        got = lo[rows].cpu()
        assert bool(((got == want.float()) | ((got.double() - want).abs() <= tol)).all())  # equal: beyond fp32's range
        tol = scale * REL
        tol = tol + ref.half_step(dtype) * (dw.abs() + tol) + TINY[dtype]
        assert bool(((gd[rows].cpu().double() - dw).abs() <= tol).all())
