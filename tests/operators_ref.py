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


def distill(logits, teacher, idx, temperature, lse=None, labels=None, ce=0.0, ignore=-100, grad=None):
    """(loss, gradient or None, scale) in 64 bits; scale: what the gradient's
    terms add up to before they cancel."""
    x, t = logits.detach().to("cpu", F64), teacher.detach().to("cpu", F64) / temperature
    idx = idx.cpu().long()
    T, V = x.shape
    loss, d, scale = torch.zeros(T, dtype=F64), torch.zeros(T, V, dtype=F64), torch.zeros(T, V, dtype=F64)
    for r in range(T):
        ok = (idx[r] >= 0) & (idx[r] < V)
        at = idx[r][ok]
        logq = torch.log_softmax(x[r] / temperature, 0)
        if at.numel():
            p = torch.exp(t[r][ok] - float(lse[r])) if lse is not None else torch.softmax(t[r][ok], 0)
            target = torch.zeros(V, dtype=F64)
            target[at] = p
            kl = torch.special.xlogy(p, p).sum() - torch.where(p > 0, p * logq[at], 0.0).sum()
            factor = torch.full((V,), float(p.sum()), dtype=F64)
            if lse is not None:
                left = max(0.0, 1.0 - float(p.sum()))
                away = torch.ones(V, dtype=torch.bool)
                away[at] = False
                factor += left
                if left > 0:
                    log_left = torch.logsumexp(logq[away], 0)
                    kl = kl + left * (math.log(left) - log_left)
                    factor[away] -= left / torch.exp(log_left)
            else:
                factor[:] = 1.0
            loss[r] = temperature ** 2 * kl
            q = logq.exp()
            d[r] = temperature * (factor * q - target)
            scale[r] = temperature * (factor.abs() * q + target)
            if lse is not None and left > 0:
                scale[r][away] = temperature * (1.0 + left / torch.exp(log_left)) * q[away]
        lab = int(labels[r]) if labels is not None else ignore
        if ce and lab != ignore and 0 <= lab < V:
            logp = torch.log_softmax(x[r], 0)
            loss[r] -= ce * logp[lab]
            hot = torch.zeros(V, dtype=F64)
            hot[lab] = 1.0
            d[r] += ce * (logp.exp() - hot)
            scale[r] += abs(ce) * (logp.exp() + hot)
    if grad is None:
        return loss, None, None
    g = grad.detach().to("cpu", F64)[:, None]
    return loss, d * g, scale * g.abs()


def activation(z, act):
    """act(z) in 64 bits, from the definitions."""
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def activation_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        b = math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-2 * b * (z + 0.044715 * z ** 3)))
        return s + z * s * (1 - s) * 2 * b * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    return torch.ones_like(z)
