"""Block-scaled E4M3 quantization, products, routing and combination in 64 bits on the
CPU, written from their definitions (no code of the package)."""
import numpy as np
import torch

BLOCK = 128


def to64(t) -> np.ndarray:
    return t.detach().to("cpu", torch.float64).numpy()


def pad16(n):
    return (n + 15) // 16 * 16


def exponent(a: np.ndarray) -> np.ndarray:
    """The least e >= -126 with a <= 448 * 2^e."""
    _, x = np.frexp(np.where(np.isfinite(a), a, 1.0))
    e = x - 9  # 448 * 2^(x - 9) = 0.875 * 2^x, and a < 2^x
    e = np.where(a > np.ldexp(448.0, e), e + 1, e)
    return np.maximum(np.where(a > 0, e, -126), -126)


def e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest E4M3 values (ties to even) of |v| <= 448."""
    _, x = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(x, -5) - 4)
    return np.rint(v / step) * step  # numpy rounds half to even


def code_bytes(v: np.ndarray) -> np.ndarray:
    """Bytes of E4M3 values."""
    a = np.abs(v)
    _, x = np.frexp(a)
    normal = a >= 2.0**-6
    high = np.where(normal, x + 6, 0)
    low = np.where(normal, np.ldexp(a, 4 - x) - 8, a * 512)
    return (np.signbit(v) * 128 + high * 8 + low).astype(np.uint8)


def quantize_rows(x: np.ndarray):
    """(values under the scales times the scales, exponents) with a block for each row and 128 columns."""
    M, K = x.shape
    nb = -(-K // BLOCK)
    out, es = np.zeros_like(x), np.zeros((M, nb), dtype=np.int64)
    for b in range(nb):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        es[:, b] = exponent(np.abs(part).max(1, initial=0.0))
        s = np.ldexp(1.0, es[:, b])[:, None]
        out[:, b * BLOCK:(b + 1) * BLOCK] = e4m3(part / s) * s
    return out, es


def quantize_weight(w: np.ndarray):
    """(codes' values, exponents) with a block for each 128 x 128."""
    N, K = w.shape
    out, es = np.zeros_like(w), np.zeros((-(-N // BLOCK), -(-K // BLOCK)), dtype=np.int64)
    for i in range(es.shape[0]):
        for j in range(es.shape[1]):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            es[i, j] = exponent(np.abs(w[at]).max())
            out[at] = e4m3(w[at] / np.ldexp(1.0, es[i, j]))
    return out, es


def weight_values(w: np.ndarray) -> np.ndarray:
    v, es = quantize_weight(w)
    return v * np.ldexp(1.0, np.repeat(np.repeat(es, BLOCK, 0), BLOCK, 1)[:w.shape[0], :w.shape[1]])


def product(a: np.ndarray, b: np.ndarray):
    """(a @ b.T, a bound on what the matrix core's sums may lack).

    The matrix core takes the products of 8 contraction indices at a time and cuts each
    off at 2^-13 of the largest's power of two, so a group may lack 7 * 2^-13 of its largest
    product; adding the groups and the instructions' sums in fp32 costs at most 2^-21 of the sum
    of magnitudes for each 64 of the contraction, and 2^-24 of it for each join of two sums."""
    K = a.shape[1]
    y = a @ b.T
    if K == 0:
        return y, np.zeros_like(y)
    pad = -K % 8
    ga = np.abs(np.pad(a, ((0, 0), (0, pad)))).reshape(a.shape[0], (K + pad) // 8, 8).max(2)
    gb = np.abs(np.pad(b, ((0, 0), (0, pad)))).reshape(b.shape[0], (K + pad) // 8, 8).max(2)
    return y, 7 * 2.0**-13 * (ga @ gb.T) + (-(-K // 64) * 2.0**-21 + 64 * 2.0**-24) * (np.abs(a) @ np.abs(b).T)


def close(got, want, slack, what):
    """bf16 outputs within half a step of bf16 (2^-8) and the sums' bound; the same places NaN."""
    g = to64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{what}: NaN elsewhere"
    ok = ~np.isnan(want)
    err = np.abs(g - want)[ok]
    bound = (slack + 2.0**-8 * (np.abs(want) + slack) + 2.0**-134)[ok]
    assert (err <= bound).all(), f"{what}: {int((err > bound).sum())} of {err.size} outside, worst {float((err / bound).max())}"


def forward(x, w):
    """Y of [M, K] and [N, K] 64-bit matrices, and its slack."""
    return product(quantize_rows(x)[0], weight_values(w))


def grad_input(dy, w):
    return product(quantize_rows(dy)[0], weight_values(w).T)


def grad_weight(dy, x):
    return product(quantize_rows(dy.T.copy())[0], quantize_rows(x.T.copy())[0])


# ------------------------------------------------------------------ routing


def route(x: np.ndarray, k: int, score: str, normalize: bool):
    """(weights, experts, places, rows, offsets) token by token."""
    T, E = x.shape
    weights, experts = np.zeros((T, k)), np.full((T, k), -1)
    for t in range(T):
        usable = [e for e in range(E) if x[t, e] > -np.inf]  # NaN is not
        taken = sorted(usable, key=lambda e: (-x[t, e], e))[:k]
        experts[t, :len(taken)] = taken
        if not np.all(x[t] < np.inf):  # NaN or +inf
            weights[t] = np.nan
            continue
        if not taken:
            continue
        top = x[t, taken]
        if score == "sigmoid":
            s = 1 / (1 + np.exp(np.minimum(-top, 700.0)))
            s = np.where(top < -700, 0.0, s)
            weights[t, :len(taken)] = s / (s.sum() or 1.0) if normalize else s
        else:
            s = np.exp(top - top[0])
            weights[t, :len(taken)] = s / (s.sum() if normalize else np.exp(x[t] - top[0]).sum())
    places, rows, offsets = np.full((T, k), -1), np.full(T * k, -1), np.zeros(E + 1, dtype=np.int64)
    n = 0
    order = np.argsort(np.where(experts.ravel() < 0, E, experts.ravel()), kind="stable")
    for i in order:
        e = experts.ravel()[i]
        if e < 0:
            break
        places.ravel()[i], rows[n] = n, i // k
        offsets[e + 1] += 1
        n += 1
    return weights, experts, places, rows, np.cumsum(offsets)


def route_grad(x: np.ndarray, experts: np.ndarray, dw: np.ndarray, score: str, normalize: bool):
    """Gradient of sum(dw * weights) at x by the derivative of each weight at each score."""
    T, E = x.shape
    d = np.zeros_like(x)
    for t in range(T):
        j = experts[t] >= 0
        at, g = experts[t][j], dw[t][j]
        if at.size == 0:
            continue
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-x[t, at]))
            slope = s * (1 - s)
            if normalize:
                S = s.sum()
                jac = np.diag(slope) / S - np.outer(s, slope) / S**2  # d w_i / d x_j
                d[t, at] = g @ jac
            else:
                d[t, at] = g * slope
        else:
            use = at if normalize else np.flatnonzero(x[t] > -np.inf)
            p = np.exp(x[t, use] - x[t, use].max())
            p /= p.sum()
            full = np.zeros(use.size)
            full[[int(np.flatnonzero(use == a)[0]) for a in at]] = g
            d[t, use] = p * (full - full @ p)
    return d
