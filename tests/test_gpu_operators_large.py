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
