"""Rotary positions on the GPU against the definition in 64 bits.

Tolerance of an element of the pair (a, b): the fp32 sine and cosine are off by
at most 2^-23 (a remainder rounded once and a polynomial of a few roundings on
values up to 1), the two products and their sum by two more half steps of
2^-24 of (|a| + |b|): together (|a| + |b|) 2^-22; then one rounding to the
output's type.  Copied elements are equal."""
import pytest
import torch

from tests import operators_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def check(got, x, positions, freqs, pairs, inverse=False):
    want = ref.rotary(x, positions, freqs, pairs, inverse)
    tol = ref.rotary_scale(x, freqs, pairs) * 2.0 ** -22
    tol = tol + ref.half_step(x.dtype) * (want.abs() + tol) + TINY[x.dtype]
    r = 2 * freqs.numel()
    tol[..., r:] = 0
    err = (got.cpu().to(torch.float64) - want).abs()
    assert got.shape == x.shape and bool((err <= tol).all()), float((err - tol).max())


def heads(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


# B, S, HQ, HK, D, rot, first position: one token; odd numbers of everything;
# halves that no 16-byte access divides (rot / 2 = 10, 3, 1); many tokens (several a
# workgroup); more items a head than threads
SHAPES = [(1, 1, 1, 1, 64, 64, 0), (3, 7, 5, 3, 128, 128, 120000), (2, 33, 4, 1, 40, 20, 900000), (1, 5, 3, 2, 48, 6, 17),
          (2, 3, 2, 1, 6, 2, 5), (2, 1500, 9, 2, 64, 32, 4000), (1, 4099, 4, 4, 96, 48, 1 << 20), (1, 3, 2, 1, 4096, 4096, 77),
          (64, 1, 32, 8, 128, 128, 3)]


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_rotary_against_the_definition(shape, dtype, pairs):
    B, S, HQ, HK, D, rot, first = shape
    packed = heads((B, S, (HQ + 2 * HK) * D), dtype, 1)
    q = packed[..., : HQ * D].view(B, S, HQ, D)
    k = packed[..., HQ * D: (HQ + HK) * D].view(B, S, HK, D)
    pos = (first + 3 * torch.arange(B)[:, None] + torch.arange(S)).cuda()
    freqs = i8.rotary_frequencies(rot, 500000.0, device="cuda")
    for inverse in (False, True):
        a, b = i8.rotary(q, k, pos, freqs, pairs=pairs, inverse=inverse)
        check(a, q, pos, freqs, pairs, inverse)
        check(b, k, pos, freqs, pairs, inverse)


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
def test_layouts_positions_and_outputs(pairs):
    B, S, H, D = 3, 10, 4, 32
    freqs = i8.rotary_frequencies(24, device="cuda")
    pos32 = torch.randint(-50, 1 << 24, (B, S), dtype=torch.int32, device="cuda")
    # heads before positions, positions 32 bits wide and strided
    q = heads((B, H, S, D), torch.bfloat16, 2).transpose(1, 2)
    a, none = i8.rotary(q, None, pos32, freqs, pairs=pairs)
    assert none is None
    check(a, q, pos32, freqs, pairs)
    pos = torch.arange(4 * S, device="cuda")[::4]  # one row of positions for every sequence
    check(i8.rotary(q, None, pos, freqs, pairs=pairs)[0], q, pos, freqs, pairs)
    # an odd address and odd strides: elements one by one
    store = heads((B * S * H * (D + 1) + 1,), torch.bfloat16, 3)
    odd = store[1:].view(B, S, H, D + 1)[..., :D]
    check(i8.rotary(odd, None, pos, freqs, pairs=pairs)[0], odd, pos, freqs, pairs)
    # into the caller's own tensors, here both parts of one packed row, the rest untouched
    packed = torch.full((B, S, 3 * H * D), 7.0, dtype=torch.bfloat16, device="cuda")
    oq, ok = packed[..., : H * D].view(B, S, H, D), packed[..., H * D: 2 * H * D].view(B, S, H, D)
    k = heads((B, S, H, D), torch.bfloat16, 4)
    i8.rotary(q, k, pos32, freqs, pairs=pairs, out_q=oq, out_k=ok)
    check(oq, q, pos32, freqs, pairs)
    check(ok, k, pos32, freqs, pairs)
    assert bool((packed[..., 2 * H * D:] == 7).all())
    # in place
    both = packed.clone()
    bq, bk = both[..., : H * D].view(B, S, H, D), both[..., H * D: 2 * H * D].view(B, S, H, D)
    i8.rotary(bq, bk, pos32, freqs, pairs=pairs, out_q=bq, out_k=bk)
    check(bq, oq, pos32, freqs, pairs)
    check(bk, ok, pos32, freqs, pairs)
    assert bool((both[..., 2 * H * D:] == 7).all())
    # nothing to do
    e = torch.empty((0, S, H, D), dtype=torch.bfloat16, device="cuda")
    assert i8.rotary(e, e, torch.empty((0, S), dtype=torch.int64, device="cuda"), freqs)[0].shape == e.shape


def test_infinities_and_nan_stay_in_their_pair():
    freqs = i8.rotary_frequencies(16, device="cuda")
    pos = torch.arange(1, 6, device="cuda")
    for pairs in ("half", "interleaved"):
        x = heads((1, 5, 2, 24), torch.float32, 5)
        x[0, 2, 1, 3], x[0, 2, 1, 20], x[0, 3, 0, 16] = float("inf"), float("nan"), float("-inf")
        y = i8.rotary(x, None, pos, freqs, pairs=pairs)[0].cpu()
        hit = (3, 11) if pairs == "half" else (2, 3)
        bad = torch.zeros(y.shape, dtype=torch.bool)
        bad[0, 2, 1, list(hit)] = bad[0, 2, 1, 20] = bad[0, 3, 0, 16] = True
        assert bool(torch.isfinite(y[~bad]).all()) and not bool(torch.isfinite(y[bad]).any())


def test_backward_is_the_inverse():
    """The gradient of sum(G * rotary(x)) against the formula's, and against
    differences of the 64-bit definition."""
    from int8_mixed_precision_rowwise_amd import training as T

    B, S, H, D = 2, 5, 3, 16
    freqs = i8.rotary_frequencies(12, device="cuda")
    pos = torch.arange(S, device="cuda") + 1000
    for pairs in ("half", "interleaved"):
        q = heads((B, S, H, D), torch.float32, 6).requires_grad_()
        k = heads((B, S, 1, D), torch.float32, 7).requires_grad_()
        G = heads((B, S, H, D), torch.float32, 8)
        a, b = T.rotary(q, k, pos, freqs, pairs)
        (a * G).sum().backward()
        check(q.grad, G, pos, freqs, pairs, inverse=True)
        assert k.grad is None or not bool(k.grad.any())  # only q' was used
        i = (1, 3, 2, 5)
        step = torch.zeros((B, S, H, D), dtype=torch.float64)
        step[i] = 1e-3
        x = q.detach().cpu().double()
        f = lambda v: (ref.rotary(v, pos, freqs, pairs) * G.cpu().double()).sum()  # noqa: E731
        slope = float((f(x + step) - f(x - step)) / 2e-3)
        assert abs(slope - float(q.grad[i])) <= 2.0 ** -20 * float(G.abs().max()) * 2


def test_other_stream_and_graph():
    B, S, H, D = 4, 65, 6, 64
    freqs = i8.rotary_frequencies(D, device="cuda")
    pos = torch.arange(S, device="cuda")
    q = heads((B, S, H, D), torch.bfloat16, 9)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        i8.rotary(q, None, pos, freqs, out_q=out)
    torch.cuda.current_stream().wait_stream(side)
    check(out, q, pos, freqs, "half")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        i8.rotary(q, None, pos, freqs, out_q=out)
    for rep in range(3):
        q.copy_(heads((B, S, H, D), torch.bfloat16, 20 + rep))
        pos.add_(1000)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, i8.rotary(q, None, pos, freqs)[0])
        check(out, q, pos, freqs, "half")


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,step", [(torch.bfloat16, 40), (torch.float16, 36), (torch.float32, 40)])
def test_large_calls_give_what_their_parts_give(dtype, step, pairs):
    S, D = 8200, 128 if dtype != torch.float32 else 64
    store = torch.randn(2, S, step, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    q, k = store[:, :, :32], store[:, :, 32:36]
    pos = torch.arange(S, device="cuda").expand(2, S)
    freqs = i8.rotary_frequencies(D // 2).cuda()  # the other half is copied
    a, b = i8.rotary(q, k, pos, freqs, pairs=pairs)
    for at in range(0, S, 2050):
        p, r = i8.rotary(q[:, at:at + 2050], k[:, at:at + 2050], pos[:, at:at + 2050], freqs, pairs=pairs)
        assert torch.equal(a[:, at:at + 2050], p) and torch.equal(b[:, at:at + 2050], r)
    i8.rotary(q, k, pos, freqs, pairs=pairs, out_q=q, out_k=k)  # in place
    assert torch.equal(a, q) and torch.equal(b, k)
