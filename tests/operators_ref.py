"""Plain 64-bit implementations of the operators around the linears, on the
CPU, written from their definitions (no code of the package)."""
import math

import torch

F64 = torch.float64


def half_step(dtype) -> float:
    """Largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def rotary(x, positions, freqs, pairs, inverse=False):
    """x [B, S, H, D] in 64 bits; positions [B, S] or [S]."""
    x = x.detach().to("cpu", F64)
    angle = positions.cpu().to(F64)[..., None] * freqs.cpu()
    angle = -angle if inverse else angle
    c, s = angle.cos(), angle.sin()
    if positions.dim() == 1:
        c, s = c[None], s[None]
    c, s = c[:, :, None], s[:, :, None]
    r = 2 * freqs.numel()
    out = x.clone()
    first, second = (slice(0, r // 2), slice(r // 2, r)) if pairs == "half" else (slice(0, r, 2), slice(1, r, 2))
    a, b = x[..., first], x[..., second]
    out[..., first] = a * c - b * s
    out[..., second] = a * s + b * c
    return out


def rotary_scale(x, freqs, pairs):
    """|a| + |b| of the pair that each element belongs to (0 for copied ones)."""
    x = x.detach().to("cpu", F64).abs()
    r = 2 * freqs.numel()
    out = torch.zeros_like(x)
    first, second = (slice(0, r // 2), slice(r // 2, r)) if pairs == "half" else (slice(0, r, 2), slice(1, r, 2))
    out[..., first] = out[..., second] = x[..., first] + x[..., second]
    return out
