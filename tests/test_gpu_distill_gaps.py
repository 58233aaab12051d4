"""Kept logits that stand far above (or below) all others, with the teacher's remaining
mass as a class of its own: the rest's share of the student is then below what fp32
holds relative to the row's maximum, and the loss and the gradient hang on it.

Tolerances as for the ordinary rows: 2^-17 of each exponential and of each term of a
gradient before they cancel, then one rounding.  Two things more at these sizes: a
loss is large itself (rounded once to fp32, 2^-24 of it), and log2(e) / temperature
is rounded to fp32 for logits of 16 bits (2^-24), which moves a distance of G
temperatures, and the logarithms of the exponentials, by 2^-24 G (at temperature 1,
for the labels' part, by 2^-24 G temperature)."""
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
GAPS = (60.0, 86.0, 90.0, 100.0, 150.0, 500.0, -60.0, -150.0)


def inputs(V, dtype, tau, seed, T=len(GAPS) + 2):
    """Row r: its kept logits GAPS[r] temperatures above the rest; then rows with nothing beside the kept."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = 12
    x = torch.randn(T, V, generator=g, device="cuda")
    idx = torch.argsort(torch.rand(T, V, generator=g, device="cuda"), 1)[:, :k] if V < 100000 else \
        (torch.randint(0, V, (T, 1), generator=g, device="cuda") + 3001 * torch.arange(k, device="cuda")) % V
    kept = torch.randn(T, k, generator=g, device="cuda")
    for r, gap in enumerate(GAPS):
        kept[r] = kept[r] + gap * tau
    x.scatter_(1, idx, kept)
    alone = torch.full_like(x, -float("inf"))
    alone.scatter_(1, idx, kept)
    x[len(GAPS):] = alone[len(GAPS):]
    t = (2.0 * torch.randn(T, k, generator=g, device="cuda")).to(bf)
    lse = (torch.logsumexp(t.double() / tau, 1) + 0.05).float()
    lse[len(GAPS) + 1] = torch.logsumexp(t[len(GAPS) + 1].double() / tau, 0).float() - 0.01  # no mass left
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    labels[1], labels[4] = idx[1, 0], idx[4, 3]
    grad = (0.5 + torch.rand(T, generator=g, device="cuda")) * (256 if dtype == fp else 1)
    return x.to(dtype), t, idx.to(torch.int32), lse, labels, grad


def check(args, tau, ce, loss, d):
    x, t, idx, lse, labels, grad = args
    n = len(GAPS)
    part = [v[:n] for v in (x, t, idx)]
    want, dw, scale = ref.distill(*part, tau, lse[:n], labels[:n] if ce else None, ce, -100, grad[:n])
    far = torch.tensor([abs(v) for v in GAPS], dtype=torch.float64)
    moved = 2.0 ** -24 * (far + 20) * max(1.0, tau) if x.dtype != f32 else torch.zeros_like(far)
    got = loss[:n].cpu().double()
    tol = (tau * tau + abs(ce)) * (2 * REL + moved) + 2.0 ** -23 * want.abs()
    assert bool(((got - want).abs() <= tol).all()), (got, want)
    gd = d[:n].cpu().double()
    tol = scale * (REL + 2 * moved[:, None])
    tol = tol + ref.half_step(x.dtype) * (dw.abs() + tol) + TINY[x.dtype]
    assert bool(((gd - dw).abs() <= tol).all()), float(((gd - dw).abs() / tol).max())
    # nothing beside the kept: a loss without bound where mass is left for it, and gradients finite all the same
    assert float(loss[n]) == float("inf")
    assert ce or bool(loss[n + 1].isfinite())
    inf = torch.isinf(x[n:])
    assert bool(d[n:].isfinite().all())
    lab = torch.zeros_like(inf)
    if ce:
        lab.scatter_(1, labels[n:, None], True)
    assert bool((d[n:][inf & ~lab] == 0).all())


@pytest.mark.parametrize("tau,ce", [(1.0, 0.0), (2.0, 0.5), (1.5, 0.25), (0.5, 0.0)])
@pytest.mark.parametrize("dtype", [bf, fp, f32])
@pytest.mark.parametrize("V", [2000, 33001, 40007, 300007])
def test_kept_logits_far_from_the_rest(V, dtype, tau, ce):
    for T in (len(GAPS) + 2, 30):  # few rows of more than 32768 bf16 classes go in segments
        args = inputs(V, dtype, tau, V + T, T)
        x, t, idx, lse, labels, grad = args
        kw = dict(temperature=tau, teacher_lse=lse, labels=labels if ce else None, ce_weight=ce)
        loss, d = i8.distill_loss_and_grad(x, t, idx, grad, **kw)
        check(args, tau, ce, loss, d)
        loss, stats = i8.distill_loss(x, t, idx, **kw)
        check(args, tau, ce, loss, i8.distill_loss_bwd(x, t, idx, stats, grad, **kw))


@pytest.mark.parametrize("V", [2000, 300007])
@pytest.mark.parametrize("dtype", [bf, f32])
def test_a_rest_masked_with_the_lowest_value(dtype, V):
    """All but the kept classes at the type's lowest value, no mass left for them: the
    loss is that over the kept classes alone, and the gradient elsewhere is 0."""
    x, t, idx, _, _, grad = inputs(V, dtype, 1.0, 5)
    low = torch.full_like(x, torch.finfo(dtype).min)
    low.scatter_(1, idx.long(), x.gather(1, idx.long()))
    lse = torch.logsumexp(t.double(), 1).float() - 2.0 ** -10
    loss, d = i8.distill_loss_and_grad(low, t, idx, grad, teacher_lse=lse)
    want, dw, scale = ref.distill(low, t, idx, 1.0, lse, grad=grad)
    assert bool(((loss.cpu().double() - want).abs() <= 2 * REL + 2.0 ** -23 * want.abs()).all())
    tol = scale * REL
    tol = tol + ref.half_step(dtype) * (dw.abs() + tol) + TINY[dtype]
    assert bool(((d.cpu().double() - dw).abs() <= tol).all())
