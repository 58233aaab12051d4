"""Two Python threads on one stream: a library call lets the other thread run, and
neither may be given memory that the other's kernels still use."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

bf = torch.bfloat16


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(bf)


def test_two_threads_share_a_stream():
    M, N, K, T, V = 300, 264, 520, 3, 200000
    X, W, dY, Z = randn(1, M, K), randn(2, N, K), randn(3, M, N), randn(4, M, N)
    Wq, ws = i8.quantize_rowwise(W)
    logits, t = randn(5, T, V), randn(6, T, 8)
    idx = torch.arange(8, device="cuda", dtype=torch.int32).expand(T, 8).contiguous()
    grad = torch.ones(T, device="cuda")
    jobs = [lambda: (i8.linear_act_fwd(X, W, activation="silu"), i8.linear_wq_fwd(X, Wq, ws, activation="gelu"),
                     *i8.linear_act_bwd(dY, Z, X, W, "gelu", want_dbias=True)),
            lambda: i8.distill_loss_and_grad(logits, t, idx, grad)]
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    wrong, errors = [0, 0], []

    def run(i):
        try:
            bad = torch.zeros((), dtype=torch.int64, device="cuda")
            for _ in range(100):
                for got, w in zip(jobs[i](), want[i]):
                    bad += (got != w).any()
            wrong[i] = int(bad)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors and wrong == [0, 0]
