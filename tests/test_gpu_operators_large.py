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
