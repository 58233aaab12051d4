"""Which views of one tensor rotary takes for its outputs, on the host: fake
addresses that nothing dereferences (a call with nothing wrong is refused for want of
a device)."""
import random

import pytest
import torch

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
EINVAL, EDEVICE = 1, 3

if torch.cuda.is_available():
    pytest.skip("addresses are made up: for hosts without a device", allow_module_level=True)

BASE = 1 << 24


def call(q, k, B, S, D):
    """In place on two views (heads, offset, strides of batch, token and head) of bf16 at one base."""
    h = [i8._Heads(BASE + 2 * off, BASE + 2 * off, H, b, s, hs, b, s, hs) for H, off, b, s, hs in (q, k)]
    st = i8.lib.i8mp_rotary(h[0], h[1], B, S, D, D, 0, 0, 0, 1 << 40, 64, 0, 1, 1 << 41, None)
    assert st in (EINVAL, EDEVICE)
    return st == EDEVICE


def places(v, B, S, D):
    H, off, b, s, hs = v
    return {off + i * b + j * s + h * hs + e for i in range(B) for j in range(S) for h in range(H) for e in range(D)}


@pytest.mark.parametrize("B,S", [(1, 1), (1, 5), (3, 1), (3, 5)])
def test_packed_projections_in_place(B, S):
    HQ, HK, D = 4, 2, 8
    n = HQ + 2 * HK
    # tokens before heads [B, S, n, D], and heads before tokens [B, n, S, D]: q, k and v heads in any order
    for b, s, hs in ((S * n * D, n * D, D), (n * S * D, D, S * D), (D, B * n * D, B * D)):
        for q0, k0 in ((0, HQ), (2 * HK, 0), (HK, 0), (0, HQ + HK)):
            assert call((HQ, q0 * hs, b, s, hs), (HK, k0 * hs, b, s, hs), B, S, D), (b, s, hs, q0, k0)
        assert not call((HQ, 0, b, s, hs), (HK, (HQ - 1) * hs, b, s, hs), B, S, D)  # one head of both
    # one key head, whose own stride says nothing
    assert call((HQ, 0, n * S * D, D, S * D), (1, HQ * S * D, n * S * D, D, 0), B, S, D)
    assert call((1, HQ * S * D, n * S * D, D, 7), (HQ, 0, n * S * D, D, S * D), B, S, D)


def test_views_that_share_an_element_are_refused():
    rng = random.Random(1)
    taken = 0
    for _ in range(20000):
        B, S, D = rng.randint(1, 3), rng.randint(1, 3), 2
        b, s = rng.choice((2, 4, 6, 8, 12, 16, 24, 36)), rng.choice((2, 4, 6, 8, 12, 16, 24))
        q = (rng.randint(1, 3), 0, b, s, rng.choice((2, 4, 8, 12)))
        k = (rng.randint(1, 3), rng.randint(0, 40), b, s, rng.choice((q[4], 2, 6)))
        if rng.random() < 0.5:
            q, k = k, q
        if call(q, k, B, S, D):
            taken += 1
            a, c = places(q, B, S, D), places(k, B, S, D)
            assert not a & c and len(a) == q[0] * B * S * D and len(c) == k[0] * B * S * D, (q, k, B, S)
    assert taken > 500
