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
