"""The block-scaled linears at the ends of what they accept."""
import numpy as np
import pytest
import torch

from . import block_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf, u8 = torch.bfloat16, torch.uint8


def test_the_longest_contractions():
    """2^23 - 8 of the contraction, whose codes lie 2^23 apart, in as many tiles as fill the GPU: zeros but for its last
    120, which a tile's last row and column must not lose.  The forward, and the gradient at the input."""
    M, L, N = 1792, (1 << 23) - 8, 4864  # 7 x 19 tiles of 256 x 256
    part = 120                           # of the last block of 128
    g = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn(M, part, generator=g, device="cuda").to(bf)
    w = torch.randn(N, part, generator=g, device="cuda").clamp(-3, 3).to(torch.float8_e4m3fn)
    X = torch.zeros(M, L, dtype=bf, device="cuda")
    X[:, -part:] = tail
    store = torch.zeros(N * (L + 8), dtype=u8, device="cuda")
    codes = store.view(N, L + 8)
    codes[:, L - part:L] = w.view(u8)
    exps = torch.full((N // 128, (L + 127) // 128), 127, dtype=u8, device="cuda")  # scales of 1
    want = ref.product(ref.quantize_rows(ref.to64(tail))[0], ref.to64(w.float()))
    ref.close(i8.linear_block_fwd(X, codes, exps), *want, "Y")
    # dX of dY [M, L] and weights [L, N]: the same product
    codes[:, L - part:L] = 0
    codes = store[:L * N].view(L, N)
    codes[L - part:] = w.view(u8).t()
    none = torch.zeros(M, N, dtype=bf, device="cuda")
    dX, _ = i8.linear_block_bwd(X, none, codes, exps.t().contiguous(), want_dw=False)
    ref.close(dX, *want, "dX")
    del X, store, codes
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N", [16, 12])
def test_falling_offsets_of_many_experts_touch_nothing_outside(N):
    """Every second expert has all rows, which by the sum of their tiles is more than 32 bits hold; N: big and small tiles."""
    E, R, K = 65535, 7 << 22, 16
    X = torch.zeros(R, K, dtype=bf, device="cuda")
    codes, exps = torch.zeros(E, N, K, dtype=u8, device="cuda"), torch.full((E, 1, 1), 127, dtype=u8, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = R

    def framed(*shape):
        n = int(np.prod(shape))
        store = torch.full((n + (1 << 20),), 7.0, dtype=bf, device="cuda")
        return store, store[1 << 19:(1 << 19) + n].view(shape)

    (sy, y), (sx, dx) = framed(R, N), framed(R, K)
    dY = torch.zeros(R, 16, dtype=bf, device="cuda")[:, :N]
    i8.expert_linear_fwd(X, codes, exps, offsets, out=y)
    i8.expert_linear_bwd(dY, X, codes, exps, offsets, dX=dx, want_dw=False)
    torch.cuda.synchronize()
    for s in (sy, sx):
        assert bool((s[:1 << 19] == 7).all()) and bool((s[-(1 << 19):] == 7).all())
    # the same experts with offsets that rise: what the rows are is right
    offsets = torch.linspace(0, R, E + 1, dtype=torch.float64, device="cuda").long()
    offsets[1:400] = 0  # empty ones first
    X.copy_(torch.randn(R, K, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"))
    w = torch.randn(E, N, K, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").clamp(-3, 3).to(torch.float8_e4m3fn)
    Y = i8.expert_linear_fwd(X, w.view(u8), exps, offsets)
    off = offsets.tolist()
    for e in (0, 398, 399, 400, 30000, E - 1):
        at = slice(off[e], off[e + 1])
        ref.close(Y[at], *ref.product(ref.quantize_rows(ref.to64(X[at]))[0], ref.to64(w[e].float())), f"Y of expert {e}")
