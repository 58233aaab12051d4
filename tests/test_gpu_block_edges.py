"""The block-scaled linears, the experts' linears and the routing at their borders: between two kernels, past
32 bits, from two threads."""
import threading

import numpy as np
import pytest
import torch

from . import block_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8


def randn(seed, *shape, std=1.0, dtype=bf):
    """Made on the GPU: some of these are large."""
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=dtype) * std


def far(t, ld):
    store = torch.zeros((t.shape[0], ld), dtype=t.dtype, device="cuda")
    store[:, :t.shape[1]] = t
    return store[:, :t.shape[1]]


# ------------------------------------------------------------------ between two kernels


@pytest.mark.parametrize("M", [16, 17, 32, 33])
@pytest.mark.parametrize("N", [4096, 4097])
@pytest.mark.parametrize("K", [128, 2048, 2056])
def test_few_rows(M, N, K):
    X, W = randn(M, M, K), randn(N, N, K, std=0.02)
    codes, exps = i8.quantize_block_weight(W)
    ref.close(i8.linear_block_fwd(X, codes, exps), *ref.forward(ref.to64(X), ref.to64(W)), "Y")


@pytest.mark.parametrize("counts", [[100, 0, 0, 28], [33, 0, 0, 0, 0, 0, 0, 0], [17, 16, 15, 0, 1], [64, 64], [0, 128, 0, 0], [100, 1, 0, 28],
                                    [2] * 64, [2] * 65])
def test_few_rows_of_experts(counts):
    """All of them few, one expert's not, on either side of 128 rows."""
    E, N, K = len(counts), 136, 264
    R = sum(counts)
    X, W = randn(1, R, K), randn(2, E, N, K, std=0.02)
    offsets = torch.tensor([0, *np.cumsum(counts)], dtype=i32, device="cuda")
    Y = i8.expert_linear_fwd(X, *i8.quantize_block_weight(W), offsets)
    x, w, a = ref.to64(X), ref.to64(W), 0
    for e, n in enumerate(counts):
        ref.close(Y[a:a + n], *ref.forward(x[a:a + n], w[e]), f"Y of expert {e}")
        a += n


@pytest.mark.parametrize("M,N,K", [(128, 200, 4096), (100, 136, 1544), (70, 1000, 12296)])
def test_split_contractions(M, N, K):
    """Few tiles over a long contraction: its parts are summed apart and joined; forward and both gradients."""
    X, W, dY = randn(1, M, K), randn(2, N, K, std=0.02), randn(3, M, N)
    codes, exps = i8.quantize_block_weight(W)
    x, w, dy = ref.to64(X), ref.to64(W), ref.to64(dY)
    ref.close(i8.linear_block_fwd(X, codes, exps), *ref.forward(x, w), "Y")
    dX, dW = i8.linear_block_bwd(dY, X, codes, exps)
    ref.close(dX, *ref.grad_input(dy, w), "dX")
    ref.close(dW, *ref.grad_weight(dy, x), "dW")
    # the same product the other way round: a long contraction over N and over the rows
    X, dY = randn(4, K, M // 8 * 8), randn(5, K, N)
    W = randn(6, N, M // 8 * 8, std=0.02)
    dX, dW = i8.linear_block_bwd(dY, X, *i8.quantize_block_weight(W))
    ref.close(dX, *ref.grad_input(ref.to64(dY), ref.to64(W)), "dX of many rows")
    ref.close(dW, *ref.grad_weight(ref.to64(dY), ref.to64(X)), "dW of many rows")


@pytest.mark.parametrize("counts", [[3, 1], [40, 70, 0, 100], [700, 0, 300, 1500, 0, 130]])
def test_one_token_in_every_row(counts):
    """An index that names few tokens again and again, the first and the last among them."""
    R, E, N, K, tokens = sum(counts), len(counts), 264, 520, 3
    X, W = randn(1, tokens, K), randn(2, E, N, K, std=0.02)
    offsets = torch.tensor([0, *np.cumsum(counts)], dtype=i32, device="cuda")
    rows = (torch.arange(R, dtype=i32, device="cuda") * 7) % tokens
    codes, exps = i8.quantize_block_weight(W)
    dY = randn(3, R, N)
    assert torch.equal(i8.expert_linear_fwd(X, codes, exps, offsets, rows), i8.expert_linear_fwd(X[rows.long()], codes, exps, offsets))
    a, b = i8.expert_linear_bwd(dY, X, codes, exps, offsets, rows), i8.expert_linear_bwd(dY, X[rows.long()], codes, exps, offsets)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("counts", [[3, 0, 9, 2], [130, 0, 77, 50], [1400, 0, 600, 3000, 0, 260]])
def test_what_no_expert_has_reaches_nothing(counts):
    """Rows behind the last expert's, and tokens that no row names, hold NaN."""
    used, E, N, K, tokens = sum(counts), len(counts), 264, 520, 60
    R = used + 70
    W, X, Xt, dY = randn(2, E, N, K, std=0.02), randn(1, R, K), randn(4, tokens, K), randn(3, R, N)
    rows = (torch.arange(R, dtype=i32, device="cuda") * 7) % (tokens - 11)
    rows[used:] = -1
    offsets = torch.tensor([0, *np.cumsum(counts)], dtype=i32, device="cuda")
    q = i8.quantize_block_weight(W)

    def run():
        return [*(i8.expert_linear_fwd(x, *q, offsets, r) for x, r in ((X, None), (Xt, rows))),
                *(t for x, r in ((X, None), (Xt, rows)) for t in i8.expert_linear_bwd(dY, x, *q, offsets, r))]

    want = run()
    nan = float("nan")
    X[used:], Xt[tokens - 11:], dY[used:] = nan, nan, nan
    got = run()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not any(bool(t.isnan().any()) for t in got)


@pytest.mark.parametrize("T", [128, 129, 255, 256, 257, 32768, 32769])
@pytest.mark.parametrize("E", [40, 65])
def test_blocks_of_tokens(T, E):
    x = torch.rand(T, E, device="cuda").argsort(1).float()  # no two scores of a token are equal
    r = i8.expert_route(x, 3)
    assert torch.equal(r.experts.long(), x.topk(3, 1).indices)
    order = torch.sort(r.experts.flatten(), stable=True).indices
    assert torch.equal(r.rows.long(), order // 3)
    assert torch.equal(r.places.flatten()[order].long(), torch.arange(3 * T, device="cuda"))
    assert torch.equal(r.offsets[1:].long(), torch.bincount(r.experts.flatten(), minlength=E).cumsum(0))


# ------------------------------------------------------------------ past 32 bits


@pytest.mark.parametrize("M,ld", [(30, (1 << 27) + 8), (40000, 65544)])
def test_rows_far_apart(M, ld):
    N, K = 264, 136
    X, W, dY = randn(1, M, K), randn(2, N, K, std=0.02), randn(3, M, N)
    codes, exps = i8.quantize_block_weight(W)
    Y = i8.linear_block_fwd(X, codes, exps)
    dX, dW = i8.linear_block_bwd(dY, X, codes, exps)
    xf = far(X, ld)
    assert torch.equal(i8.linear_block_fwd(xf, codes, exps), Y)
    off, rows = torch.tensor([0, M], device="cuda"), torch.arange(M, dtype=i32, device="cuda").flip(0)
    assert torch.equal(i8.expert_linear_fwd(xf, codes[None], exps[None], off, rows),
                       i8.expert_linear_fwd(X, codes[None], exps[None], off, rows))
    df = far(dY, ld)
    a, b = i8.linear_block_bwd(df, xf, codes, exps)
    assert torch.equal(a, dX) and torch.equal(b, dW)
    xf.fill_(7), df.fill_(7)
    i8.linear_block_fwd(X, codes, exps, out=df)
    i8.linear_block_bwd(dY, X, codes, exps, dX=xf, want_dw=False)
    assert torch.equal(df, Y) and torch.equal(xf, dX)


@pytest.mark.parametrize("M", [1, 30, 200])
def test_more_weights_than_31_bits(M):
    """2.4e9 codes: the last columns and the first against the reference, their codes against the same rows alone."""
    N, K = 300000, 8072
    W = torch.empty(N, K, dtype=bf, device="cuda")
    for lo in range(0, N, 30000):
        W[lo:lo + 30000] = randn(lo, 30000, K, std=0.02)
    codes, exps = i8.quantize_block_weight(W)
    X = randn(1, M, K)
    Y = i8.linear_block_fwd(X, codes, exps)
    for lo, hi in ((0, 128), (N // 128 * 128 - 128, N)):  # whole blocks
        c, e = i8.quantize_block_weight(W[lo:hi])
        assert torch.equal(c, codes[lo:hi]) and torch.equal(e, exps[lo // 128:(hi + 127) // 128])
        ref.close(Y[:, lo:hi], *ref.forward(ref.to64(X), ref.to64(W[lo:hi])), f"Y from {lo}")
    dY = torch.zeros(M, N, dtype=bf, device="cuda")
    dY[:, -100:] = randn(2, M, 100)
    dX, dW = i8.linear_block_bwd(dY, X, codes, exps)
    at = N // 128 * 128 - 128
    ref.close(dX, *ref.grad_input(ref.to64(dY[:, at:]), ref.to64(W[at:])), "dX")
    ref.close(dW[at:], *ref.grad_weight(ref.to64(dY[:, at:]), ref.to64(X)), "dW")
    assert not bool(dW[:at - 128].any())


def test_many_rows():
    """4.3e9 elements of X: the last rows against the reference, a corner of the weight's gradient."""
    M, N, K = (1 << 21) + 77, 136, 2048
    X = torch.empty(M, K, dtype=bf, device="cuda")
    for lo in range(0, M, 1 << 18):
        X[lo:lo + (1 << 18)] = randn(lo, min(1 << 18, M - lo), K)
    W, dY = randn(1, N, K, std=0.02), randn(2, M, N)
    codes, exps = i8.quantize_block_weight(W)
    Y = i8.linear_block_fwd(X, codes, exps)
    dX, dW = i8.linear_block_bwd(dY, X, codes, exps)
    for s in (slice(0, 200), slice((1 << 20) - 100, (1 << 20) + 100), slice(M - 200, M)):
        ref.close(Y[s], *ref.forward(ref.to64(X[s]), ref.to64(W)), "Y")
        ref.close(dX[s], *ref.grad_input(ref.to64(dY[s]), ref.to64(W)), "dX")
    for n, k in ((slice(0, 4), slice(0, 4)), (slice(N - 4, N), slice(K - 4, K))):
        ref.close(dW[n, k], *ref.grad_weight(ref.to64(dY[:, n]), ref.to64(X[:, k])), "dW")


def test_many_experts_weights():
    """4.3e9 codes of 64 experts: the last expert's rows and gradient, and the first's."""
    E, N, K, R = 64, 8200, 8192, 640
    codes = torch.empty(E, N, K, dtype=u8, device="cuda")
    exps = torch.empty(E, 65, 64, dtype=u8, device="cuda")
    W = [randn(10 + e, N, K, std=0.02) for e in (0, E - 1)]
    other = randn(9, N, K, std=0.02)
    for e in range(E):
        i8.quantize_block_weight(W[0] if e == 0 else W[1] if e == E - 1 else other, codes[e], exps[e])
    X, dY = randn(1, R, K), randn(2, R, N)
    for counts in ([10] * E, [R // 2] + [0] * (E - 2) + [R // 2], [100] + [1] * 62 + [478]):
        offsets = torch.tensor([0, *np.cumsum(counts)], dtype=i32, device="cuda")
        Y = i8.expert_linear_fwd(X, codes, exps, offsets)
        dX, dW = i8.expert_linear_bwd(dY, X, codes, exps, offsets)
        for e, w in ((0, W[0]), (E - 1, W[1])):
            at = slice(0, counts[0]) if e == 0 else slice(R - counts[-1], R)
            part = slice(N - 136, N)  # N is 64 blocks and 8 more: the last two blocks' columns
            assert (N - 136) % 128 == 0
            ref.close(Y[at, part], *ref.forward(ref.to64(X[at]), ref.to64(w[part])), f"Y of expert {e}")
            ref.close(dW[e, part], *ref.grad_weight(ref.to64(dY[at, part]), ref.to64(X[at])), f"dW of expert {e}")
            c = slice(K - 128, K)
            ref.close(dX[at, c], *ref.grad_input(ref.to64(dY[at]), ref.to64(w[:, c])), f"dX of expert {e}")


def test_routing_of_more_tokens_than_a_launch_holds():
    """2^28 tokens of 16 lanes each are 2^32 work items."""
    T = (1 << 28) + 77
    x = randn(1, T, 2)
    r = i8.expert_route(x, 1, score="sigmoid", normalize=False)
    want = (x[:, 1] > x[:, 0]).to(i32)
    assert torch.equal(r.experts[:, 0], want)
    ones = want.sum()
    assert r.offsets.tolist() == [0, T - int(ones), T]
    place = torch.where(want == 1, want.cumsum(0, dtype=torch.int64) - 1 + T - ones, (1 - want).cumsum(0, dtype=torch.int64) - 1)
    assert torch.equal(r.places[:, 0].long(), place)
    assert torch.equal(r.rows[r.places[:, 0].long()], torch.arange(T, dtype=i32, device="cuda"))
    del place
    dw = randn(2, T, 1, dtype=torch.float32)
    d = i8.expert_route_bwd(x, r.experts, dw, score="sigmoid", normalize=False)
    for s in (slice(0, 5000), slice((1 << 27) - 2500, (1 << 27) + 2500), slice(T - 5000, T)):
        assert torch.equal(d[s], i8.expert_route_bwd(x[s], r.experts[s], dw[s], score="sigmoid", normalize=False))
    assert bool((d.gather(1, 1 - r.experts.long()) == 0).all())


@pytest.mark.parametrize("N", [2056, 2051])
def test_combination_past_32_bits(N):
    T, k = (1 << 19) + 3, 4
    R = T * k
    Y = torch.empty(R, N, dtype=bf, device="cuda")
    for lo in range(0, R, 1 << 18):
        Y[lo:lo + (1 << 18)] = randn(lo, min(1 << 18, R - lo), N)
    places = torch.randperm(R, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").view(T, k).to(i32)
    weights, dout = torch.rand(T, k, device="cuda"), randn(2, T, N)
    out = i8.expert_combine(Y, places, weights)
    dY, dw = i8.expert_combine_bwd(dout, Y, places, weights)
    for s in (slice(0, 50), slice(T - 50, T)):
        p = places[s].long()
        y, w, d = ref.to64(Y[p]), ref.to64(weights[s]), ref.to64(dout[s])
        terms = y * w[..., None]
        size = np.abs(terms).sum(1)
        assert (np.abs(ref.to64(out[s]) - terms.sum(1)) <= 2.0**-8 * np.abs(terms.sum(1)) + 6 * 2.0**-24 * (1 + 2.0**-8) * size).all()
        want = w[..., None] * d[:, None]
        assert (np.abs(ref.to64(dY[p]) - want) <= (2.0**-8 + 2.0**-24) * (1 + 2.0**-8) * np.abs(want)).all()
        prods = y * d[:, None]
        assert (np.abs(ref.to64(dw[s]) - prods.sum(2)) <= (N // 64 + 12) * 2.0**-24 * np.abs(prods).sum(2)).all()


# ------------------------------------------------------------------ two threads


def test_two_threads_share_a_stream():
    M, N, K, E = 300, 264, 520, 4
    X, W, dY = randn(1, M, K), randn(2, E, N, K, std=0.02), randn(3, M, N)
    codes, exps = i8.quantize_block_weight(W)
    offsets = torch.tensor([0, 100, 100, 250, 300], dtype=i32, device="cuda")
    x, w = randn(4, 3000, 24, dtype=torch.float32), randn(5, 520, 264)
    jobs = [lambda: (i8.expert_linear_fwd(X, codes, exps, offsets), *i8.expert_linear_bwd(dY, X, codes, exps, offsets)),
            lambda: (*i8.expert_route(x, 4), i8.linear_block_fwd(X, codes[1], exps[1]),
                     *i8.linear_block_bwd(dY, X, codes[2], exps[2]), *i8.quantize_block_weight(w))]
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    wrong, errors = [0, 0], []

    def run(i):
        try:
            bad = torch.zeros((), dtype=torch.int64, device="cuda")
            for _ in range(100):
                for got, t in zip(jobs[i](), want[i]):
                    bad += (got != t).any()
            wrong[i] = int(bad)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors and wrong == [0, 0]


# ------------------------------------------------------------------ big tiles


@pytest.mark.parametrize("M,N,K", [(4100, 4104, 1000), (4100, 4104, 1160), (8195, 2568, 840)])
def test_big_tiles(M, N, K):
    """More tiles than CUs, of which the last are cut; the same rows in views."""
    X, W = randn(M, M, K), randn(N, N, K, std=0.02)
    codes, exps = i8.quantize_block_weight(W)
    want, slack = ref.forward(ref.to64(X), ref.to64(W))
    ref.close(i8.linear_block_fwd(X, codes, exps), want, slack, "Y")
    store = torch.full((M + 1, N + 24), 7.0, dtype=bf, device="cuda")
    i8.linear_block_fwd(far(X, K + 24), codes, exps, out=store[:M, 8:N + 8])
    ref.close(store[:M, 8:N + 8], want, slack, "Y in a view")
    assert bool((store[:, :8] == 7).all()) and bool((store[:, N + 8:] == 7).all()) and bool((store[M] == 7).all())


@pytest.mark.parametrize("K", [8, 72, 128, 136, 264])
def test_big_tiles_of_short_contractions(K):
    """Contractions of one block, of two and a part: some rows of many."""
    M, N = 8200, 8200
    X, W, dY = randn(1, M, K), randn(2, N, K, std=0.02), randn(3, M, K)
    codes, exps = i8.quantize_block_weight(W)
    Y = i8.linear_block_fwd(X, codes, exps)
    # the same sizes as gradients: dX over K columns of dY, dW over K rows
    Wt = randn(4, K, N, std=0.02)
    dX, none = i8.linear_block_bwd(dY, torch.zeros(M, N, dtype=bf, device="cuda"), *i8.quantize_block_weight(Wt), want_dw=False)
    dYt, Xt = randn(5, K, M), randn(6, K, N)
    none, dW = i8.linear_block_bwd(dYt, Xt, torch.zeros(M, (N + 15) // 16 * 16, dtype=u8, device="cuda"),
                                   torch.zeros((M + 127) // 128, (N + 127) // 128, dtype=u8, device="cuda"), want_dx=False)
    for s in (slice(0, 60), slice(4090, 4110), slice(M - 60, M)):
        ref.close(Y[s], *ref.forward(ref.to64(X[s]), ref.to64(W)), "Y")
        ref.close(dX[s], *ref.grad_input(ref.to64(dY[s]), ref.to64(Wt)), "dX")
        ref.close(dW[s], *ref.grad_weight(ref.to64(dYt[:, s]), ref.to64(Xt)), "dW")


@pytest.mark.parametrize("M,N,K", [(4100, 1000, 4104), (1000, 4104, 4104), (2100, 2056, 2056)])
def test_big_tiles_backward(M, N, K):
    X, W, dY = randn(M, M, K), randn(N, N, K, std=0.02), randn(K, M, N, std=1e-3)
    codes, exps = i8.quantize_block_weight(W)
    dX, dW = i8.linear_block_bwd(dY, X, codes, exps)
    dy = ref.to64(dY)
    ref.close(dX, *ref.grad_input(dy, ref.to64(W)), "dX")
    ref.close(dW, *ref.grad_weight(dy, ref.to64(X)), "dW")
    only_x, _ = i8.linear_block_bwd(dY, X, codes, exps, want_dw=False)
    _, only_w = i8.linear_block_bwd(dY, X, codes, exps, want_dx=False)
    assert torch.equal(only_x, dX) and torch.equal(only_w, dW)


@pytest.mark.parametrize("counts,N,K", [([1400, 0, 600, 3000, 0, 260], 2056, 2056), ([70, 0, 1, 200, 129, 64, 0, 130] * 8, 1032, 1032)])
@pytest.mark.parametrize("gather", [False, True])
def test_big_tiles_of_experts(counts, N, K, gather):
    used, E = sum(counts), len(counts)
    R, tokens = used + 5, 777
    W, dY = randn(2, E, N, K, std=0.02), randn(3, R, N, std=1e-3)
    X = randn(1, tokens if gather else R, K)
    rows = torch.randint(-1, tokens + 1, (R,), generator=torch.Generator().manual_seed(1)).to(i32).cuda() if gather else None
    x = ref.to64(X)
    if gather:
        r = rows.cpu().numpy()
        x = np.where(((r >= 0) & (r < tokens))[:, None], x[np.clip(r, 0, tokens - 1)], 0)
    codes, exps = i8.quantize_block_weight(W)
    offsets = torch.tensor([0, *np.cumsum(counts)], dtype=i32, device="cuda")
    Y = i8.expert_linear_fwd(X, codes, exps, offsets, rows)
    dX, dW = i8.expert_linear_bwd(dY, X, codes, exps, offsets, rows)
    w, dy, a = ref.to64(W), ref.to64(dY), 0
    for e, n in enumerate(counts):
        at, a = slice(a, a + n), a + n
        if E > 8 and e % 7:
            continue  # some of many
        ref.close(Y[at], *ref.forward(x[at], w[e]), f"Y of expert {e}")
        ref.close(dX[at], *ref.grad_input(dy[at], w[e]), f"dX of expert {e}")
        ref.close(dW[e], *ref.grad_weight(dy[at], x[at]), f"dW of expert {e}")
    assert not bool(Y[used:].any()) and not bool(dX[used:].any())
