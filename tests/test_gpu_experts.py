"""The experts' linears on the GPU against the block reference, expert by expert."""
import numpy as np
import pytest
import torch

from . import block_ref as ref

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64


def randn(seed, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(bf).cuda()


# rows of each expert; N; K
CASES = [([0, 1, 0], 16, 16), ([3, 0, 0, 5, 1], 40, 24), ([0] * 70 + [2, 0, 1], 24, 40), ([17, 130, 0, 64], 136, 264),
         ([1] * 40, 264, 136), ([300, 0, 20, 129], 264, 136), ([128, 256, 127], 300, 200), ([600, 700], 264, 520),
         ([2000], 40, 72), ([0, 0], 40, 72), ([700, 0, 300, 1500, 0, 130], 2056, 2056)]  # the last in big tiles


def setup(counts, N, K, behind, dtype=i32, gather=False):
    E, used = len(counts), sum(counts)
    R = used + behind
    offsets = torch.tensor([0, *np.cumsum(counts)], dtype=dtype, device="cuda")
    tokens = max(1, used // 3)
    g = torch.Generator().manual_seed(used)
    if gather:
        X = randn(1, tokens, K)
        rows = torch.randint(0, tokens, (R,), generator=g).to(i32)
        rows[used:] = -1
        if used > 4:
            rows[used // 2], rows[used // 3] = -7, tokens  # no row of X: zeros
        inside = (rows >= 0) & (rows < tokens)
        x = np.where(inside.numpy()[:, None], ref.to64(X)[rows.clamp(0, tokens - 1).numpy()], 0)
        rows = rows.cuda()
    else:
        X, rows = randn(1, R, K), None
        x = ref.to64(X)
    W, dY = randn(2, E, N, K, std=0.02), randn(3, R, (N + 7) // 8 * 8, std=1e-3)[:, :N]  # rows start every 16 bytes
    return R, used, offsets, X, rows, x, W, dY


def parts(counts):
    a = 0
    for e, n in enumerate(counts):
        yield e, slice(a, a + n)
        a += n


@pytest.mark.parametrize("counts,N,K", CASES)
@pytest.mark.parametrize("gather,behind,dtype", [(False, 0, i32), (True, 5, i64)])
def test_forward_and_backward(counts, N, K, gather, behind, dtype):
    R, used, offsets, X, rows, x, W, dY = setup(counts, N, K, behind, dtype, gather)
    codes, exps = i8.quantize_block_weight(W)
    Y = i8.expert_linear_fwd(X, codes, exps, offsets, rows)
    dX, dW = i8.expert_linear_bwd(dY, X, codes, exps, offsets, rows)
    assert Y.shape == (R, N) and dX.shape == (R, K) and dW.shape == W.shape
    w, dy = ref.to64(W), ref.to64(dY)
    for e, at in parts(counts):
        ref.close(Y[at], *ref.forward(x[at], w[e]), f"Y of expert {e}")
        ref.close(dX[at], *ref.grad_input(dy[at], w[e]), f"dX of expert {e}")
        ref.close(dW[e], *ref.grad_weight(dy[at], x[at]), f"dW of expert {e}")
    assert not bool(Y[used:].any()) and not bool(dX[used:].any())
    # given outputs keep the rows behind the last expert's
    out, dx = torch.full((R, N), 7.0, dtype=bf, device="cuda"), torch.full((R, K), 7.0, dtype=bf, device="cuda")
    i8.expert_linear_fwd(X, codes, exps, offsets, rows, out=out)
    i8.expert_linear_bwd(dY, X, codes, exps, offsets, rows, dX=dx, want_dw=False)
    assert torch.equal(out[:used], Y[:used]) and bool((out[used:] == 7).all())
    assert torch.equal(dx[:used], dX[:used]) and bool((dx[used:] == 7).all())


def test_one_expert_with_all_rows_is_the_linear():
    for M in (3, 50, 300):
        X, W, dY = randn(1, M, 264), randn(2, 136, 264), randn(3, M, 136)
        offsets = torch.tensor([0, M], device="cuda")
        codes, exps = i8.quantize_block_weight(W)
        assert torch.equal(i8.expert_linear_fwd(X, codes[None], exps[None], offsets), i8.linear_block_fwd(X, codes, exps))
        a, b = i8.expert_linear_bwd(dY, X, codes[None], exps[None], offsets), i8.linear_block_bwd(dY, X, codes, exps)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1][0], b[1])


@pytest.mark.parametrize("offsets", [[0, 5, 3, 40], [-9, 4, 10, 20], [0, 10, 20, 10**6], [7, 7, 7, 7], [30, 20, 10, 0]])
@pytest.mark.parametrize("R", [40, 400])
def test_offsets_that_make_no_sense_touch_nothing_outside(offsets, R):
    """What lies around the outputs stays as it was, whatever the offsets hold."""
    N, K, E = 40, 72, 3
    X, dY, W = randn(1, R, K), randn(2, R, N), randn(3, E, N, K)
    codes, exps = i8.quantize_block_weight(W)
    off = torch.tensor(offsets, dtype=i64, device="cuda")

    def framed(*shape):
        n = int(np.prod(shape))
        store = torch.full((n + 2048,), 7.0, dtype=bf, device="cuda")
        return store, store[1024:1024 + n].view(shape)

    (sy, y), (sx, dx), (sw, dw) = framed(R, N), framed(R, K), framed(E, N, K)
    i8.expert_linear_fwd(X, codes, exps, off, out=y)
    i8.expert_linear_bwd(dY, X, codes, exps, off, dX=dx, dW=dw)
    torch.cuda.synchronize()
    for s in (sy, sx, sw):
        assert bool((s[:1024] == 7).all()) and bool((s[-1024:] == 7).all())


def test_replayed_from_a_graph_with_other_offsets():
    """The offsets are read on the GPU: a captured call follows them."""
    R, N, K, E = 300, 136, 264, 5
    X, dY, W = randn(1, R, K), randn(2, R, N), randn(3, E, N, K)
    codes, exps = i8.quantize_block_weight(W)
    offsets = torch.tensor([0, 60, 120, 180, 240, 300], dtype=i32, device="cuda")

    def step():
        return (i8.expert_linear_fwd(X, codes, exps, offsets), *i8.expert_linear_bwd(dY, X, codes, exps, offsets))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for off in ([0, 60, 120, 180, 240, 300], [0, 0, 300, 300, 300, 300], [0, 1, 2, 3, 4, 5], [0] * 6, [0, 128, 129, 257, 260, 290]):
        offsets.copy_(torch.tensor(off, dtype=i32))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
