"""Block-scaled FP8 linears on the GPU: codes bit for bit, products within the matrix core's
derived bound of 64-bit sums, and exactly where every partial sum is representable."""
import numpy as np
import pytest
import torch

from . import block_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf = torch.bfloat16
nan = float("nan")


def randn(seed, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(bf).cuda()


def padded(t, ld):
    """The same matrix with rows `ld` apart, NaN between them."""
    store = torch.full((t.shape[0], ld), nan, dtype=t.dtype, device=t.device)
    store[:, :t.shape[1]] = t
    return store[:, :t.shape[1]]


def rows_of(t):
    """A matrix whose rows start every 16 bytes."""
    return t if t.shape[1] % 8 == 0 else padded(t, (t.shape[1] + 7) // 8 * 8)


# ------------------------------------------------------------------ codes


def check_codes(W):
    codes, exps = i8.quantize_block_weight(W)
    torch.cuda.synchronize()
    w = ref.to64(W).reshape(-1, *W.shape[-2:])
    N, K = W.shape[-2:]
    for e in range(w.shape[0]):
        v, es = ref.quantize_weight(w[e])
        c, b = codes.view(-1, *codes.shape[-2:])[e].cpu().numpy(), exps.view(-1, *exps.shape[-2:])[e].cpu().numpy()
        assert np.array_equal(b, es + 127)
        assert np.array_equal(c[:, :K], ref.code_bytes(np.where(v == 0, np.copysign(v, w[e]), v)))
        assert not c[:, K:].any()


@pytest.mark.parametrize("shape", [(1, 8), (1, 1), (128, 128), (129, 136), (7, 1000), (300, 520), (3, 130, 264), (2, 1, 16)])
def test_weight_codes(shape):
    check_codes(rows_of(randn(1, *shape)) if len(shape) == 2 else randn(1, *shape))


def test_weight_codes_of_every_magnitude():
    """Blocks whose largest value is each bf16 from the smallest up, around the border at 1.75 of a
    power of two, beside the smallest and the ties below it."""
    top = torch.arange(1, 0x7F80, 31, dtype=torch.int32)[:1024].to(torch.int16).view(bf).float()
    w = torch.zeros(1024, 128)
    w[:, 0] = top
    w[:, 1:64] = top[:, None] * torch.linspace(-1, 1, 63)
    w[:, 64:] = top[:, None] * torch.exp2(-torch.arange(64, dtype=torch.float32))
    # one row of each block of 128 rows holds the values, the others are zeros
    tall = torch.zeros(128 * 128, 8 * 128, dtype=bf)
    tall[::128] = w.to(bf).view(128, 8 * 128)
    check_codes(tall.cuda())


def test_weight_codes_of_views_and_given_outputs():
    store = randn(2, 3, 2, 40, 64)
    check_codes(store[:, 1, :, :24])
    W = randn(3, 40, 64)
    codes, exps = torch.empty(40, 64, dtype=torch.uint8, device="cuda"), torch.empty(1, 1, dtype=torch.uint8, device="cuda")
    c, e = i8.quantize_block_weight(W, codes, exps)
    assert c is codes and e is exps
    assert torch.equal(c, i8.quantize_block_weight(W)[0])


# ------------------------------------------------------------------ products

SIZES = [(1, 1, 8), (1, 16, 16), (1, 300, 2040), (5, 40, 24), (16, 130, 136), (17, 64, 128), (33, 129, 520), (64, 257, 264),
         (65, 129, 264), (129, 136, 72), (200, 300, 1000), (300, 70, 128), (257, 520, 2040), (700, 520, 200),
         (4100, 2056, 264), (4100, 2051, 72)]  # enough tiles for the big ones; columns that they do not take


@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(M, N, K):
    X, W = randn(M, M, K), randn(N, N, K, std=0.02)
    X[:, K // 2] *= 20
    codes, exps = i8.quantize_block_weight(W)
    want, slack = ref.forward(ref.to64(X), ref.to64(W))
    ref.close(i8.linear_block_fwd(X, codes, exps), want, slack, "Y")
    # rows further apart, and outputs that start anywhere
    store = torch.full((M, N + 3), 7.0, dtype=bf, device="cuda")
    i8.linear_block_fwd(padded(X, K + 16), codes, exps, out=store[:, 1:N + 1])
    ref.close(store[:, 1:N + 1], want, slack, "Y in a view")
    assert bool((store[:, 0] == 7).all()) and bool((store[:, N + 1:] == 7).all())


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (5, 40, 24), (130, 136, 72), (65, 264, 136), (200, 304, 1000), (257, 520, 2040), (1000, 136, 128),
                                   (300, 4104, 2056), (4100, 264, 2056), (60, 4104, 2056)])
def test_backward(M, N, K):
    X, W, dY = randn(M, M, K), randn(N, N, K, std=0.02), randn(K, M, N, std=1e-3)
    codes, exps = i8.quantize_block_weight(W)
    dX, dW = i8.linear_block_bwd(dY, X, codes, exps)
    dy = ref.to64(dY)
    ref.close(dX, *ref.grad_input(dy, ref.to64(W)), "dX")
    ref.close(dW, *ref.grad_weight(dy, ref.to64(X)), "dW")
    only_x, none = i8.linear_block_bwd(dY, X, codes, exps, want_dw=False)
    assert none is None and torch.equal(only_x, dX)
    none, only_w = i8.linear_block_bwd(dY, X, codes, exps, want_dx=False)
    assert none is None and torch.equal(only_w, dW)


def test_products_of_representable_sums_are_exact():
    """Small whole numbers times a power of two for each block: every sum is exact, so the scales of
    rows, columns and blocks are checked to the bit."""
    g = torch.Generator().manual_seed(5)
    for M, N, K in ((3, 200, 640), (40, 200, 640), (300, 264, 1160)):
        nb = -(-K // 128)

        def whole(rows, cols, by_row, by_col):
            v = torch.randint(-2, 3, (rows, cols), generator=g).double()
            v[::, ::128] = 4  # the largest of each block of a row
            v[::128] = torch.where(v[::128] == 0, 1.0, v[::128])
            e = torch.randint(-1, 2, (-(-rows // by_row), -(-cols // by_col)), generator=g)
            return v * torch.exp2(e.double()).repeat_interleave(by_row, 0)[:rows].repeat_interleave(by_col, 1)[:, :cols]

        x, w, dy = whole(M, K, 1, 128), whole(N, K, 128, 128), whole(M, N, 1, 128)
        X, W, dY = (t.to(bf).cuda() for t in (x, w, dy))
        assert torch.equal(X.cpu().double(), x) and nb > 1
        codes, exps = i8.quantize_block_weight(W)
        assert torch.equal(i8.linear_block_fwd(X, codes, exps).cpu(), (x @ w.t()).to(bf))
        dX, dW = i8.linear_block_bwd(dY, X, codes, exps)
        assert torch.equal(dX.cpu(), (dy @ w).to(bf))
        # down the rows: powers of two of a column within a block of rows differ by at most 2^4, all kept by E4M3
        assert torch.equal(dW.cpu(), (dy.t() @ x).to(bf))


@pytest.mark.parametrize("M", [3, 40, 200])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), nan])
def test_a_value_that_is_not_finite_makes_what_it_meets_nan(M, value):
    N, K = 264, 392
    X, W, dY = randn(1, M, K), randn(2, N, K, std=0.02), randn(3, M, N)
    codes, exps = i8.quantize_block_weight(W)
    clean, (cx, cw) = i8.linear_block_fwd(X, codes, exps), i8.linear_block_bwd(dY, X, codes, exps)
    bad = X.clone()
    bad[1, 200] = value
    y = i8.linear_block_fwd(bad, codes, exps)
    assert bool(y[1].isnan().all())
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(y[keep], clean[keep])
    _, dw = i8.linear_block_bwd(dY, bad, codes, exps)
    cols = torch.arange(K, device="cuda") != 200
    assert bool(dw[:, 200].isnan().all()) and torch.equal(dw[:, cols], cw[:, cols])
    bad = dY.clone()
    bad[M - 1, 5] = value
    dx, dw = i8.linear_block_bwd(bad, X, codes, exps)
    assert bool(dx[M - 1].isnan().all()) and torch.equal(dx[:M - 1], cx[:M - 1])
    rows = torch.arange(N, device="cuda") != 5
    assert bool(dw[5].isnan().all()) and torch.equal(dw[rows], cw[rows])
    bad = W.clone()
    bad[130, 7] = value
    codes, exps = i8.quantize_block_weight(bad)
    assert int(exps[1, 0]) == 255
    y = i8.linear_block_fwd(X, codes, exps)
    part = (torch.arange(N, device="cuda") // 128) == 1
    assert bool(y[:, part].isnan().all()) and torch.equal(y[:, ~part], clean[:, ~part])


def test_zeros_and_the_smallest_values():
    M, N, K = 5, 40, 256
    X, W = torch.zeros(M, K, dtype=bf, device="cuda"), randn(2, N, K)
    codes, exps = i8.quantize_block_weight(W)
    assert not bool(i8.linear_block_fwd(X, codes, exps).any())
    X[2] = torch.finfo(bf).smallest_normal / 64  # a subnormal
    want, slack = ref.forward(ref.to64(X), ref.to64(W))
    ref.close(i8.linear_block_fwd(X, codes, exps), want, slack, "Y")
    X[3] = 3.0e38
    W2 = W * 2.0**-30
    codes, exps = i8.quantize_block_weight(W2)
    want, slack = ref.forward(ref.to64(X), ref.to64(W2))
    ref.close(i8.linear_block_fwd(X, codes, exps), want, slack, "Y of large values")


def test_empty_sizes():
    codes, exps = i8.quantize_block_weight(randn(1, 40, 64))
    X, dY = torch.zeros(0, 64, dtype=bf, device="cuda"), torch.zeros(0, 40, dtype=bf, device="cuda")
    assert i8.linear_block_fwd(X, codes, exps).shape == (0, 40)
    junk = torch.full((40, 64), nan, dtype=bf, device="cuda")
    dX, dW = i8.linear_block_bwd(dY, X, codes, exps, dW=junk)
    assert dX.shape == (0, 64) and dW is junk and not bool(dW.any())
    codes, exps = i8.quantize_block_weight(torch.zeros(40, 0, dtype=bf, device="cuda"))
    y = i8.linear_block_fwd(torch.zeros(3, 0, dtype=bf, device="cuda"), codes, exps,
                            out=torch.full((3, 40), nan, dtype=bf, device="cuda"))
    assert not bool(y.any())


def test_the_same_call_gives_the_same_bits_on_any_stream():
    M, N, K = 300, 264, 1000
    X, W, dY = randn(1, M, K), randn(2, N, K), randn(3, M, N)
    codes, exps = i8.quantize_block_weight(W)
    want = (i8.linear_block_fwd(X, codes, exps), *i8.linear_block_bwd(dY, X, codes, exps))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((i8.linear_block_fwd(X, codes, exps), *i8.linear_block_bwd(dY, X, codes, exps)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


def test_replayed_from_a_graph():
    M, N, K = 200, 264, 520
    X, W, dY, few = randn(1, M, K), randn(2, N, K), randn(3, M, N), randn(4, 3, K)

    def step():
        codes, exps = i8.quantize_block_weight(W)
        return (codes, exps, i8.linear_block_fwd(X, codes, exps), i8.linear_block_fwd(few, codes, exps),
                *i8.linear_block_bwd(dY, X, codes, exps))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for rep in range(3):
        for i, t in enumerate((X, W, dY, few)):
            t.copy_(randn(10 * rep + i, *t.shape))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_a_long_contraction_of_rows():
    """dW over 200000 rows: sums of many blocks, each with scales of its own."""
    M, N, K = 200001, 16, 24
    X, dY = randn(1, M, K), randn(2, M, N)
    X[::128] *= 50
    codes, exps = i8.quantize_block_weight(randn(3, N, K))
    _, dW = i8.linear_block_bwd(dY, X, codes, exps, want_dx=False)
    ref.close(dW, *ref.grad_weight(ref.to64(dY), ref.to64(X)), "dW")
