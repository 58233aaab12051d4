"""The workspace that an operator takes for itself lives until the library call
has returned: the call lets other threads run before it launches, and on a shared
stream they would be given a block that had gone back.  On the CPU, with the
launching call replaced by one that looks at what is still alive."""
import weakref

import pytest
import torch

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
from int8_mixed_precision_rowwise_amd import operators as ops  # noqa: E402

bf = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """[(name, whether every workspace taken so far is alive, its address and size as passed)]."""
    taken, seen, empty = [], [], torch.empty

    def recording_empty(*args, **kw):
        t = empty(*args, **kw)
        if t.dtype == torch.uint8:
            taken.append((weakref.ref(t), t.data_ptr(), t.numel()))
        return t

    def call(dev, name, *args):
        alive = [r() is not None for r, _, _ in taken]
        given = [(p, n) in zip(args, args[1:]) for _, p, n in taken]
        seen.append((name, len(taken), all(alive), all(given)))

    monkeypatch.setattr(ops, "_on_gpu", lambda *t: True)
    monkeypatch.setattr(i8, "_device", lambda *t: t[0].device)
    monkeypatch.setattr(torch, "empty", recording_empty)
    monkeypatch.setattr(ops, "_call", call)
    return seen


@pytest.mark.parametrize("which", ["fwd", "train", "wq", "bwd", "distill", "step"])
def test_the_workspace_is_alive_in_the_call(calls, which):
    X, W, Z = torch.zeros(32, 64, dtype=bf), torch.zeros(48, 64, dtype=bf), torch.zeros(32, 48, dtype=bf)
    logits, t, idx = torch.zeros(2, 200000, dtype=bf), torch.zeros(2, 4), torch.zeros(2, 4, dtype=torch.int32)  # rows in segments
    if which == "fwd":
        i8.linear_act_fwd(X, W)
    elif which == "train":
        i8.linear_act_fwd_train(X, W)
    elif which == "wq":
        i8.linear_wq_fwd(X, torch.zeros(48, 64, dtype=torch.int8), torch.ones(48))
    elif which == "bwd":
        i8.linear_act_bwd(Z, Z, X, W, "silu")
    elif which == "distill":
        i8.distill_loss(logits, t, idx)
    else:
        i8.distill_loss_and_grad(logits, t, idx, torch.ones(2))
    ((_, taken, alive, given),) = calls
    assert taken == 1 and given and alive


def test_a_given_workspace_is_the_one_passed(calls):
    logits, t, idx = torch.zeros(2, 200000, dtype=bf), torch.zeros(2, 4), torch.zeros(2, 4, dtype=torch.int32)
    need = i8.lib.i8mp_distill_workspace_bytes(2, 200000, 4, 0)
    i8.distill_loss(logits, t, idx, workspace=torch.empty(need, dtype=torch.uint8))
    i8.distill_loss(logits[:, :1000], t, idx)  # rows that need none
    assert [(c[1], c[2], c[3]) for c in calls][0] == (1, True, True)
    assert calls[1][1] == 1
