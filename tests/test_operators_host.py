"""The operators around the linears on the host: what the binding refuses
before any library call (the library is replaced by a recorder), what the C
ABI refuses before any HIP call (fake addresses that nothing dereferences),
and the host-side helpers."""
import ctypes
import math

import pytest
import torch

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
L = i8.lib
EINVAL, ERANGE, EDEVICE, EWORKSPACE = 1, 2, 3, 5


def accepted(call):
    """A call with nothing wrong but its made-up addresses: refused for want of
    a device.  Where there is one it is not made."""
    return torch.cuda.is_available() or call() == EDEVICE


bf, f32, f64, i64, i32, u8, s8 = (torch.bfloat16, torch.float32, torch.float64, torch.int64, torch.int32, torch.uint8,
                                  torch.int8)


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def f(*args):
            self.calls.append(name)
            return 0
        return f


@pytest.fixture
def lib(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(i8, "lib", rec)
    yield rec
    assert all(c.endswith("_workspace_bytes") for c in rec.calls), rec.calls


def t(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


# ------------------------------------------------------------------ rotary


def test_rotary_binding_checks(lib):
    q, k, pos, fr = t(2, 3, 4, 8), t(2, 3, 1, 8), t(2, 3, dtype=i64), t(4, dtype=f64)
    with pytest.raises(ValueError, match="device tensors"):
        i8.rotary(q, k, pos, fr)  # right but for the device
    with pytest.raises(TypeError, match="q"):
        i8.rotary(q.double(), k, pos, fr)
    with pytest.raises(TypeError, match="k: torch.bfloat16"):
        i8.rotary(q, k.float(), pos, fr)
    with pytest.raises(ValueError, match="4-D"):
        i8.rotary(q[0], None, pos, fr)
    with pytest.raises(ValueError, match="k: shape"):
        i8.rotary(q, t(2, 3, 1, 6), pos, fr)
    with pytest.raises(ValueError, match="adjacent"):
        i8.rotary(t(2, 3, 8, 4).transpose(2, 3), None, pos, t(2, dtype=f64))
    with pytest.raises(ValueError, match="pairs"):
        i8.rotary(q, k, pos, fr, pairs="both")
    with pytest.raises(TypeError, match="freqs"):
        i8.rotary(q, k, pos, fr.float())
    with pytest.raises(ValueError, match="frequencies"):
        i8.rotary(q, k, pos, t(5, dtype=f64))
    with pytest.raises(ValueError, match="frequencies"):
        i8.rotary(q, k, pos, t(0, dtype=f64))
    with pytest.raises(ValueError, match="head size"):
        i8.rotary(t(2, 3, 4, 7), None, pos, t(2, dtype=f64))
    with pytest.raises(TypeError, match="positions"):
        i8.rotary(q, k, pos.float(), fr)
    with pytest.raises(ValueError, match="positions"):
        i8.rotary(q, k, t(3, 2, dtype=i64), fr)
    with pytest.raises(ValueError, match="out_q"):
        i8.rotary(q, k, pos, fr, out_q=t(2, 3, 5, 8))
    with pytest.raises(ValueError, match="out_k"):
        i8.rotary(q, None, pos, fr, out_k=t(2, 3, 1, 8))


def _rot(q=None, k=None, B=2, S=3, D=8, rot=8, dtype=0, pairs=0, pos=1 << 30, bits=64, pb=3, ps=1, freqs=1 << 29):
    H = i8._Heads
    q = q or H(1 << 20, 1 << 24, 4, 96, 32, 8, 96, 32, 8)
    return L.i8mp_rotary(q, k, B, S, D, rot, dtype, pairs, 0, pos, bits, pb, ps, freqs, None)


def test_rotary_abi_validation():
    H = i8._Heads
    assert accepted(lambda: _rot())
    assert L.i8mp_rotary(None, None, 1, 1, 8, 8, 0, 0, 0, 1 << 30, 64, 0, 0, 1 << 29, None) == EINVAL
    for bad in (dict(dtype=3), dict(pairs=2), dict(B=-1), dict(B=1 << 20, S=1 << 20), dict(D=7), dict(D=4098), dict(rot=10),
                dict(rot=0), dict(rot=3), dict(bits=16), dict(pos=None), dict(pos=4), dict(freqs=None), dict(freqs=4),
                dict(pb=-1)):
        assert _rot(**bad) == EINVAL, bad
    x, y = 1 << 20, 1 << 24
    assert _rot(H(None, y, 4, 96, 32, 8, 96, 32, 8)) == EINVAL
    assert _rot(H(x + 1, y, 4, 96, 32, 8, 96, 32, 8)) == EINVAL  # half an element
    assert _rot(H(x, y, -1, 96, 32, 8, 96, 32, 8)) == EINVAL
    assert _rot(H(x, y, 4, -96, 32, 8, 96, 32, 8)) == EINVAL
    assert _rot(H(x, y, 4, 1 << 50, 32, 8, 96, 32, 8)) == EINVAL
    assert _rot(H(x, y, 4, 96, 32, 8, 96, 32, 4)) == EINVAL  # the output's heads overlap
    assert _rot(H(x, y, 4, 96, 32, 8, 64, 32, 8)) == EINVAL  # its sequences do
    assert _rot(H(x, x + 16, 4, 96, 32, 8, 96, 32, 8)) == EINVAL  # shifted into its own input
    assert accepted(lambda: _rot(H(x, x, 4, 96, 32, 8, 96, 32, 8)))  # in place
    assert _rot(H(x, x, 4, 0, 32, 8, 96, 32, 8)) == EINVAL  # not in place: other strides
    assert accepted(lambda: _rot(H(x, y, 4, 0, 0, 0, 96, 32, 8)))  # a broadcast input
    assert _rot(H(x, 1 << 30, 4, 96, 32, 8, 96, 32, 8)) == EINVAL  # onto the positions
    # both outputs in one packed row: apart, and overlapping by one head
    q, k = H(x, y, 4, 96, 32, 8, 144, 48, 8), H(1 << 22, y + 2 * 32, 2, 48, 16, 8, 144, 48, 8)
    assert accepted(lambda: _rot(q, k))
    k.y = y + 2 * 24
    assert _rot(q, k) == EINVAL
    k.y = y + 2 * 33  # past the end of the packed row
    assert _rot(q, k) == EINVAL
    # nothing to do: accepted without a device
    assert _rot(B=0) == 0 and _rot(H(None, None, 0, 0, 0, 0, 0, 0, 0)) == 0


def test_rotary_frequencies():
    f = i8.rotary_frequencies(8, 10000.0)
    assert f.dtype == f64 and torch.allclose(f, torch.tensor([1, 0.1, 0.01, 0.001], dtype=f64), rtol=1e-15, atol=0)
    assert torch.equal(i8.rotary_frequencies(8, 10000.0, factor=4.0), f / 4)
    # 100 positions hold 15.9, 1.59, 0.159 and 0.0159 turns
    g = i8.rotary_frequencies(8, 10000.0, factor=4.0, original_length=100)
    keep = (100 * 0.1 / (2 * math.pi) - 1) / 3
    want = torch.tensor([1, 0.1 * (keep + (1 - keep) / 4), 0.0025, 0.00025], dtype=f64)
    assert torch.allclose(g, want, rtol=1e-14, atol=0)
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, theta=0.0), dict(rot=8, factor=0.0),
                dict(rot=8, original_length=10, low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            i8.rotary_frequencies(**bad)


# ------------------------------------------------------------------ distillation loss


def test_distill_binding_checks(lib):
    x, te, ix, g, st = t(4, 30), t(4, 5), t(4, 5, dtype=i32), t(4, dtype=f32), t(4, 8, dtype=f64)
    with pytest.raises(ValueError, match="device tensors"):
        i8.distill_loss_and_grad(x, te, ix, g)  # right but for the device
    with pytest.raises(TypeError, match="logits"):
        i8.distill_loss(x.double(), te, ix)
    with pytest.raises(ValueError, match="logits: 2-D"):
        i8.distill_loss(x[0], te, ix)
    with pytest.raises(ValueError, match="logits: columns"):
        i8.distill_loss(t(30, 4).t(), te, ix)
    with pytest.raises(ValueError, match="classes"):
        i8.distill_loss(t(4, 0), te, ix)
    with pytest.raises(ValueError, match="teacher: 4 rows"):
        i8.distill_loss(x, t(3, 5), ix)
    with pytest.raises(TypeError, match="idx"):
        i8.distill_loss(x, te, ix.float())
    with pytest.raises(ValueError, match="idx: shape"):
        i8.distill_loss(x, te, t(4, 6, dtype=i32))
    with pytest.raises(ValueError, match="1024"):
        i8.distill_loss(x, t(4, 1025), t(4, 1025, dtype=i32))
    for tau in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(ValueError, match="temperature"):
            i8.distill_loss(x, te, ix, temperature=tau)
    with pytest.raises(ValueError, match="ce_weight"):
        i8.distill_loss(x, te, ix, ce_weight=math.nan)
    with pytest.raises(ValueError, match="without labels"):
        i8.distill_loss(x, te, ix, ce_weight=0.5)
    with pytest.raises(TypeError, match="labels"):
        i8.distill_loss(x, te, ix, labels=g, ce_weight=0.5)
    with pytest.raises(ValueError, match="labels"):
        i8.distill_loss(x, te, ix, labels=t(3, dtype=i64), ce_weight=0.5)
    with pytest.raises(TypeError, match="teacher_lse"):
        i8.distill_loss(x, te, ix, teacher_lse=g.double())
    with pytest.raises(TypeError, match="grad"):
        i8.distill_loss_and_grad(x, te, ix, g.double())
    with pytest.raises(TypeError, match="grad"):
        i8.distill_loss_and_grad(x, te, ix, None)
    with pytest.raises(ValueError, match="grad"):
        i8.distill_loss_bwd(x, te, ix, st, t(5, dtype=f32))
    with pytest.raises(ValueError, match="stats"):
        i8.distill_loss_bwd(x, te, ix, t(4, 7, dtype=f64), g)
    with pytest.raises(TypeError, match="stats"):
        i8.distill_loss_bwd(x, te, ix, None, g)
    with pytest.raises(ValueError, match="out"):
        i8.distill_loss_bwd(x, te, ix, st, g, out=t(4, 31))
    with pytest.raises(TypeError, match="workspace"):
        i8.distill_loss(x, te, ix, workspace=g)


def _dist(call="step", grad=1 << 33, grad_s=1, loss=1 << 34, d=1 << 35, d_ld=130, stats=1 << 36, ws=1 << 37, n=1 << 20, **over):
    a = dict(logits=1 << 20, T=300, V=130, ld=130, dtype=0, teacher=1 << 30, teacher_ld=5, teacher_dtype=0, idx=1 << 31,
             idx_ld=5, idx_bits=32, kept=5, temperature=1.0, lse=None, labels=None, label_bits=0, ignore_index=-100, ce_weight=0.0)
    p = i8._Distill(**{**a, **over})
    if call == "step":
        return L.i8mp_distill_step(p, grad, grad_s, loss, d, d_ld, ws, n, None)
    if call == "fwd":
        return L.i8mp_distill_fwd(p, loss, stats, ws, n, None)
    return L.i8mp_distill_bwd(p, stats, grad, grad_s, d, d_ld, None)


def test_distill_abi_validation():
    for call in ("step", "fwd", "bwd"):
        assert accepted(lambda: _dist(call))
        assert accepted(lambda: _dist(call, logits=(1 << 20) + 2, ld=133, d_ld=137))  # any alignment of elements
        for bad in (dict(dtype=3), dict(teacher_dtype=-1), dict(T=-1), dict(T=1 << 31), dict(V=0), dict(V=(1 << 30) + 1, ld=1 << 31),
                    dict(ld=129), dict(logits=None), dict(logits=(1 << 20) + 1), dict(kept=-1), dict(kept=1025), dict(teacher=None),
                    dict(teacher_ld=4), dict(idx=None), dict(idx_ld=4), dict(idx_bits=16), dict(idx=(1 << 31) + 2),
                    dict(temperature=0.0), dict(temperature=math.nan), dict(ce_weight=math.inf), dict(lse=3),
                    dict(labels=1 << 32, ce_weight=1.0, label_bits=8), dict(labels=(1 << 32) + 4, ce_weight=1.0, label_bits=64)):
            assert _dist(call, **bad) == EINVAL, (call, bad)
        assert _dist(call, T=0, logits=None, teacher=None, idx=None) == 0  # nothing to do
        assert accepted(lambda: _dist(call, kept=0, teacher=None, idx=None))
    for call in ("step", "bwd"):
        for bad in (dict(d=None), dict(d=1 << 20), dict(d=(1 << 20) + 260), dict(d=(1 << 35) + 1), dict(d_ld=129), dict(grad=None),
                    dict(grad=(1 << 33) + 2), dict(grad_s=-1), dict(grad=1 << 35), dict(d=1 << 30), dict(d=1 << 31)):
            assert _dist(call, **bad) == EINVAL, (call, bad)
        assert accepted(lambda: _dist(call, grad_s=0))
    for bad in (dict(loss=None), dict(loss=1 << 35), dict(loss=1 << 20)):
        assert _dist("step", **bad) == EINVAL, bad
    for bad in (dict(stats=4), dict(stats=1 << 34)):
        assert _dist("fwd", **bad) == EINVAL, bad
    assert accepted(lambda: _dist("fwd", stats=None))
    assert _dist("bwd", stats=None) == EINVAL and _dist("bwd", stats=1 << 35) == EINVAL
    # a few long rows are split: they need a workspace
    long = dict(T=2, V=40000, ld=40000, d_ld=40000)
    need = L.i8mp_distill_workspace_bytes(2, 40000, 5, 0)
    assert need > 0 and need % 256 == 0
    for call in ("step", "fwd"):
        assert _dist(call, ws=None, **long) == EWORKSPACE
        assert _dist(call, ws=(1 << 37) + 8, **long) == EWORKSPACE
        assert _dist(call, n=need - 1, **long) == EWORKSPACE
        assert accepted(lambda: _dist(call, n=need, **long))
        assert _dist(call, ws=1 << 34, **long) == EINVAL
    assert L.i8mp_distill_workspace_bytes(-1, 5, 5, 0) == 0 and L.i8mp_distill_workspace_bytes(5, 5, 5, 9) == 0


def test_distill_reference_gradient_is_the_derivative():
    from tests import operators_ref as ref
    g = torch.Generator().manual_seed(0)
    x = torch.randn(6, 40, generator=g, dtype=f64)
    te = torch.randn(6, 7, generator=g, dtype=f64)
    ix = torch.stack([torch.randperm(40, generator=g)[:7] for _ in range(6)])
    ix[1, 3:] = -1
    ix[2] = -1
    lab = torch.tensor([0, 5, -100, 7, int(ix[4, 2]), 39])
    for tau, rest, ce in ((1.0, False, 0.0), (2.0, True, 0.5), (1.5, False, 1.0)):
        lse = torch.logsumexp(te / tau, 1) + 0.1 if rest else None
        _, d, _ = ref.distill(x, te, ix, tau, lse, lab, ce, grad=torch.ones(6))
        v = torch.randn(6, 40, generator=g, dtype=f64)
        h = 1e-5
        up, down = (ref.distill(x + s * h * v, te, ix, tau, lse, lab, ce)[0] for s in (1, -1))
        assert torch.allclose((up - down) / (2 * h), (d * v).sum(1), rtol=1e-7, atol=1e-8)


# ------------------------------------------------------------------ linears with an epilogue


def test_linear_act_binding_checks(lib):
    lib.i8mp_linear_act_workspace_bytes = lib.i8mp_linear_wq_workspace_bytes = lambda *a: 0
    X, W, b, r, q, s = t(4, 16), t(8, 16), t(8), t(4, 8), t(8, 16, dtype=s8), t(8, dtype=f32)
    for call in (lambda **k: i8.linear_act_fwd(X, W, **k), lambda **k: i8.linear_act_fwd_train(X, W, **k),
                 lambda **k: i8.linear_wq_fwd(X, q, s, **k)):
        with pytest.raises(ValueError, match="device tensors"):
            call(bias=b, residual=r, activation="gelu")  # right but for the device
        with pytest.raises(ValueError, match="activation"):
            call(activation="tanh")
        with pytest.raises(TypeError, match="bias"):
            call(bias=b.float())
        with pytest.raises(ValueError, match="bias"):
            call(bias=t(9))
        with pytest.raises(ValueError, match="residual"):
            call(residual=t(4, 9))
        with pytest.raises(TypeError, match="residual"):
            call(residual=r.float())
        with pytest.raises(ValueError, match="out"):
            call(out=t(5, 8))
        with pytest.raises(TypeError, match="workspace"):
            call(workspace=s)
    with pytest.raises(TypeError, match="X"):
        i8.linear_act_fwd(X.float(), W)
    with pytest.raises(ValueError, match="W: 16 columns"):
        i8.linear_act_fwd(X, t(8, 24))
    with pytest.raises(TypeError, match="Wq"):
        i8.linear_wq_fwd(X, W, s)
    with pytest.raises(TypeError, match="w_scale"):
        i8.linear_wq_fwd(X, q, None)
    with pytest.raises(ValueError, match="w_scale"):
        i8.linear_wq_fwd(X, q, t(9, dtype=f32))
    dY, Z = t(4, 8), t(4, 8)
    with pytest.raises(ValueError, match="device tensors"):
        i8.linear_act_bwd(dY, Z, X, W, "silu")
    with pytest.raises(TypeError, match="Z"):
        i8.linear_act_bwd(dY, None, X, W, "silu")
    with pytest.raises(ValueError, match="Z"):
        i8.linear_act_bwd(dY, t(4, 9), X, W, "silu")
    with pytest.raises(ValueError, match="W: 8 rows"):
        i8.linear_act_bwd(dY, Z, X, t(9, 16), "silu")
    with pytest.raises(ValueError, match="X: shape"):
        i8.linear_act_bwd(dY, Z, t(5, 16), W, "silu")
    with pytest.raises(ValueError, match="dX"):
        i8.linear_act_bwd(dY, Z, X, W, "silu", dX=t(4, 15))
    with pytest.raises(TypeError, match="dbias"):
        i8.linear_act_bwd(dY, Z, X, W, "silu", want_dbias=True, dbias=t(8))
    with pytest.raises(ValueError, match="colmax_x"):
        i8.linear_act_bwd(dY, Z, X, W, "silu", colmax_x=t(15, dtype=f32))


G = 1 << 30


def _lact(call="fwd", opts=(0, 0, 0), cx=None, cw=None, ws=40 * G, n=1 << 30, q=41 * G, ldq=64, sc=42 * G, **over):
    a = dict(M=100, N=48, K=64, X=1 * G, ldx=64, W=2 * G, ldw=64, activation=2, bias=3 * G, residual=4 * G, ld_residual=48,
             Y=5 * G, ldy=48, Z=6 * G, ldz=48)
    p = i8._LinearAct(**{**a, **over})
    o = None if opts is None else i8._Opts(*opts)
    if call == "fwd":
        return L.i8mp_linear_act_fwd(p, o, cx, cw, ws, n, None)
    return L.i8mp_linear_wq_fwd(p, q, ldq, sc, ws, n, None)


def test_linear_act_abi_validation():
    for call in ("fwd", "wq"):
        assert accepted(lambda: _lact(call))
        assert accepted(lambda: _lact(call, bias=None, residual=None, Z=None, Y=5 * G + 2, ldy=51))
        for bad in (dict(M=-1), dict(N=1 << 40), dict(activation=5), dict(activation=-1), dict(X=None), dict(X=G + 8), dict(ldx=60),
                    dict(ldx=68), dict(Y=None), dict(Y=5 * G + 1), dict(ldy=47), dict(bias=3 * G + 1), dict(residual=4 * G + 8),
                    dict(ld_residual=47), dict(ld_residual=52), dict(Z=6 * G + 1), dict(ldz=40), dict(Y=1 * G), dict(Y=4 * G),
                    dict(Z=5 * G), dict(Z=1 * G + 64), dict(Y=3 * G), dict(M=1 << 30, N=1 << 30)):
            assert _lact(call, **bad) == EINVAL, (call, bad)
        assert _lact(call, K=133145, ldx=133152, ldw=133152, ldq=133152) == ERANGE
        assert _lact(call, ws=None) == EWORKSPACE and _lact(call, ws=40 * G + 16) == EWORKSPACE and _lact(call, n=100) == EWORKSPACE
        assert _lact(call, ws=5 * G) == EINVAL and _lact(call, ws=1 * G) == EINVAL
        assert _lact(call, M=0, X=None, Y=None, Z=None, residual=None) == 0
    assert _lact(opts=None) == EINVAL and _lact(opts=(2, 0, 0)) == EINVAL
    assert _lact(W=None) == EINVAL and _lact(W=2 * G + 2) == EINVAL and _lact(ldw=60) == EINVAL and _lact(Y=2 * G) == EINVAL
    assert accepted(lambda: _lact(cx=50 * G, cw=51 * G))
    assert _lact(cx=50 * G, cw=50 * G) == EINVAL and _lact(cx=5 * G) == EINVAL and _lact(cx=50 * G + 2) == EINVAL
    assert _lact("wq", q=None) == EINVAL and _lact("wq", q=41 * G + 4) == EINVAL and _lact("wq", ldq=60) == EINVAL
    assert _lact("wq", sc=None) == EINVAL and _lact("wq", Y=41 * G) == EINVAL and _lact("wq", Y=42 * G) == EINVAL
    need = L.i8mp_linear_act_workspace_bytes(100, 48, 64, 0)
    assert accepted(lambda: _lact(n=need)) and _lact(n=need - 1) == EWORKSPACE
    assert L.i8mp_linear_act_workspace_bytes(-1, 1, 1, 0) == 0 and L.i8mp_linear_wq_workspace_bytes(1, 1, 1 << 41) == 0


def _lbwd(opts=(0, 0, 0), cx=None, cw=None, ws=40 * G, n=1 << 30, **over):
    a = dict(M=100, N=48, K=64, dY=1 * G, lddy=48, Z=2 * G, ldz=48, X=3 * G, ldx=64, W=4 * G, ldw=64, activation=4, dX=5 * G,
             lddx=64, dW=6 * G, lddw=64, dbias=7 * G)
    return L.i8mp_linear_act_bwd(i8._LinearActGrad(**{**a, **over}), None if opts is None else i8._Opts(*opts), cx, cw, ws, n, None)


def test_linear_act_bwd_abi_validation():
    assert accepted(lambda: _lbwd()) and accepted(lambda: _lbwd(activation=0, Z=None))
    assert accepted(lambda: _lbwd(dX=None, W=None)) and accepted(lambda: _lbwd(dW=None, X=None))
    for bad in (dict(opts=None), dict(opts=(3, 0, 0)), dict(activation=9), dict(M=-1), dict(dY=None), dict(dY=G + 8), dict(lddy=44),
                dict(Z=None), dict(ldz=44), dict(Z=2 * G + 2), dict(X=None), dict(W=None), dict(ldx=60), dict(ldw=68), dict(lddx=63),
                dict(lddw=63), dict(dX=5 * G + 1), dict(dbias=7 * G + 2), dict(dX=6 * G), dict(dX=1 * G), dict(dW=3 * G),
                dict(dbias=2 * G), dict(dbias=5 * G), dict(cx=8 * G + 2), dict(cw=5 * G), dict(ws=1 * G), dict(ws=7 * G)):
        assert _lbwd(**bad) == EINVAL, bad
    assert _lbwd(M=133145) == ERANGE and _lbwd(N=133152, lddy=133152, ldz=133152) == ERANGE
    assert accepted(lambda: _lbwd(M=133145, dW=None))
    need = L.i8mp_linear_act_workspace_bytes(100, 48, 64, 1)
    assert accepted(lambda: _lbwd(n=need)) and _lbwd(n=need - 1) == EWORKSPACE and _lbwd(ws=None) == EWORKSPACE
    assert _lbwd(dX=None, dW=None, dbias=None) == 0 and _lbwd(M=0, N=0, dY=None, Z=None) == 0


def test_activation_derivatives_are_the_derivatives():
    from tests import operators_ref as ref
    z = torch.linspace(-8, 8, 999, dtype=f64) + 1e-3
    for act in i8.ACTIVATIONS:
        slope = (ref.activation(z + 1e-5, act) - ref.activation(z - 1e-5, act)) / 2e-5
        assert torch.allclose(slope, ref.activation_grad(z, act), atol=1e-8)
