"""The block-scaled linears, the experts' linears and the routing on the host: what the
binding refuses before any library call, and the C ABI before any HIP call (fake
addresses that nothing dereferences)."""
import ctypes

import pytest
import torch

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
L = i8.lib
EINVAL, EDEVICE, EWORKSPACE = 1, 3, 5
bf, f32, f64, i64, i32, u8, s8 = (torch.bfloat16, torch.float32, torch.float64, torch.int64, torch.int32, torch.uint8,
                                  torch.int8)


def accepted(call):
    """A call with nothing wrong but its made-up addresses: refused for want of a device.
    Where there is one it is not made."""
    return torch.cuda.is_available() or call() == EDEVICE


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


# ------------------------------------------------------------------ the binding


def test_quantize_block_weight_checks(lib):
    with pytest.raises(ValueError, match="device tensors"):
        i8.quantize_block_weight(t(40, 64))  # right but for the device
    with pytest.raises(TypeError, match="W: torch.bfloat16"):
        i8.quantize_block_weight(t(40, 64, dtype=f32))
    with pytest.raises(TypeError, match="W: torch.Tensor"):
        i8.quantize_block_weight(None)
    for w in (t(64), t(1, 2, 3, 8)):
        with pytest.raises(ValueError, match=r"\[E, N, K\]"):
            i8.quantize_block_weight(w)
    with pytest.raises(ValueError, match="at least one expert"):
        i8.quantize_block_weight(t(0, 8, 8))
    with pytest.raises(ValueError, match="adjacent"):
        i8.quantize_block_weight(t(64, 40).t())
    with pytest.raises(ValueError, match="adjacent"):
        i8.quantize_block_weight(t(8).expand(40, 8))
    with pytest.raises(ValueError, match=r"codes: shape \(40, 80\)"):
        i8.quantize_block_weight(t(40, 72), codes=t(40, 72, dtype=u8))
    with pytest.raises(TypeError, match="exponents: torch.uint8"):
        i8.quantize_block_weight(t(40, 72), exponents=t(1, 1, dtype=s8))
    with pytest.raises(ValueError, match="codes: contiguous"):
        i8.quantize_block_weight(t(40, 64), codes=t(64, 40, dtype=u8).t())


def test_linear_block_checks(lib):
    X, dY, c, e = t(5, 72), t(5, 40), t(40, 80, dtype=u8), t(1, 1, dtype=u8)
    with pytest.raises(ValueError, match="device tensors"):
        i8.linear_block_fwd(X, c, e)
    with pytest.raises(ValueError, match="device tensors"):
        i8.linear_block_bwd(dY, X, c, e)
    with pytest.raises(TypeError, match="X: torch.bfloat16"):
        i8.linear_block_fwd(X.float(), c, e)
    with pytest.raises(TypeError, match="X: torch.Tensor"):
        i8.linear_block_fwd(None, c, e)
    with pytest.raises(ValueError, match="X: 2-D"):
        i8.linear_block_fwd(X[0], c, e)
    with pytest.raises(TypeError, match="codes: torch.uint8"):
        i8.linear_block_fwd(X, c.to(s8), e)
    with pytest.raises(ValueError, match=r"codes: shape \(40, 96\)"):
        i8.linear_block_fwd(t(5, 88), c, e)
    with pytest.raises(ValueError, match=r"codes: \[N, K\]"):
        i8.linear_block_fwd(X, c[None], e)
    with pytest.raises(ValueError, match=r"exponents: shape \(1, 1\)"):
        i8.linear_block_fwd(X, c, t(2, 1, dtype=u8))
    with pytest.raises(ValueError, match=r"out: shape \(5, 40\)"):
        i8.linear_block_fwd(X, c, e, out=t(5, 41))
    with pytest.raises(ValueError, match="stride 1"):
        i8.linear_block_fwd(t(72, 5).t(), c, e)
    with pytest.raises(TypeError, match="workspace"):
        i8.linear_block_fwd(X, c, e, workspace=t(4, dtype=f32))
    with pytest.raises(ValueError, match=r"dY: shape \(5, 40\)"):
        i8.linear_block_bwd(t(5, 39), X, c, e)
    with pytest.raises(TypeError, match="dY: torch.Tensor"):
        i8.linear_block_bwd(None, X, c, e)
    with pytest.raises(ValueError, match="X: 6 rows"):
        i8.linear_block_bwd(t(6, 40), X, c, e)
    with pytest.raises(ValueError, match="dW: shape"):
        i8.linear_block_bwd(dY, X, c, e, dW=t(40, 80))
    with pytest.raises(ValueError, match="dX: shape"):
        i8.linear_block_bwd(dY, X, c, e, dX=t(5, 80))


def test_expert_linear_checks(lib):
    X, dY, c, e, off = t(5, 72), t(5, 40), t(3, 40, 80, dtype=u8), t(3, 1, 1, dtype=u8), t(4, dtype=i32)
    rows = t(9, dtype=i32)
    with pytest.raises(ValueError, match="device tensors"):
        i8.expert_linear_fwd(X, c, e, off)
    with pytest.raises(ValueError, match="device tensors"):
        i8.expert_linear_bwd(t(9, 40), X, c, e, off.long(), rows)
    for f, a in ((i8.expert_linear_fwd, ()), (i8.expert_linear_bwd, (dY,))):
        with pytest.raises(TypeError, match="offsets"):
            f(*a, X, c, e, None)
        with pytest.raises(TypeError, match="offsets: torch.int32 or"):
            f(*a, X, c, e, off.float())
        with pytest.raises(ValueError, match="offsets: 1-D tensor of 4"):
            f(*a, X, c, e, t(3, dtype=i32))
        with pytest.raises(ValueError, match=r"codes: \[E, N, K\]"):
            f(*a, X, c[0], e[0], off)
        with pytest.raises(ValueError, match="at least one expert"):
            f(*a, X, c[:0], e[:0], t(1, dtype=i32))
    with pytest.raises(ValueError, match="at least one row"):
        i8.expert_linear_fwd(X[:0], c, e, off, rows)
    with pytest.raises(TypeError, match="rows: torch.int32"):
        i8.expert_linear_fwd(X, c, e, off, rows.long())
    with pytest.raises(ValueError, match="rows: 1-D tensor"):
        i8.expert_linear_fwd(X, c, e, off, rows[:, None])
    with pytest.raises(ValueError, match="rows: 1-D tensor of 5"):
        i8.expert_linear_bwd(dY, X, c, e, off, rows)
    with pytest.raises(ValueError, match=r"out: shape \(9, 40\)"):
        i8.expert_linear_fwd(X, c, e, off, rows, out=t(5, 40))
    with pytest.raises(ValueError, match="dW: contiguous"):
        i8.expert_linear_bwd(dY, X, c, e, off, dW=t(3, 72, 40).transpose(1, 2))


def test_route_checks(lib):
    x = t(6, 8, dtype=f32)
    with pytest.raises(ValueError, match="device tensors"):
        i8.expert_route(x, 2)
    with pytest.raises(TypeError, match="logits"):
        i8.expert_route(x.double(), 2)
    with pytest.raises(ValueError, match="logits: 2-D"):
        i8.expert_route(x[0], 2)
    for k in (0, 9, -1, 2.0):
        with pytest.raises(ValueError, match="k from 1 to 8"):
            i8.expert_route(x, k)
    with pytest.raises(ValueError, match="k from 1 to 32"):
        i8.expert_route(t(2, 100), 33)
    for E in (0, 1025):
        with pytest.raises(ValueError, match="1 to 1024 experts"):
            i8.expert_route(t(2, E), 1)
    with pytest.raises(ValueError, match="score"):
        i8.expert_route(x, 2, score="relu")
    e, g = t(6, 2, dtype=i32), t(6, 2, dtype=f32)
    with pytest.raises(ValueError, match="device tensors"):
        i8.expert_route_bwd(x, e, g)
    with pytest.raises(TypeError, match="experts: torch.int32"):
        i8.expert_route_bwd(x, e.long(), g)
    with pytest.raises(TypeError, match="experts: torch.Tensor"):
        i8.expert_route_bwd(x, None, g)
    with pytest.raises(ValueError, match="dweights: shape"):
        i8.expert_route_bwd(x, e, g[:5])
    with pytest.raises(TypeError, match="dweights: torch.float32"):
        i8.expert_route_bwd(x, e, g.double())
    with pytest.raises(ValueError, match="out: shape"):
        i8.expert_route_bwd(x, e, g, out=t(6, 9, dtype=f32))


def test_combine_checks(lib):
    Y, p, w, d = t(9, 8), t(3, 2, dtype=i32), t(3, 2, dtype=f32), t(3, 8)
    with pytest.raises(ValueError, match="device tensors"):
        i8.expert_combine(Y, p, w)
    with pytest.raises(ValueError, match="device tensors"):
        i8.expert_combine_bwd(d, Y, p, w)
    with pytest.raises(TypeError, match="Y"):
        i8.expert_combine(Y.double(), p, w)
    with pytest.raises(TypeError, match="places: torch.int32"):
        i8.expert_combine(Y, p.long(), w)
    with pytest.raises(ValueError, match="at least one"):
        i8.expert_combine(Y, p[:, :0])
    with pytest.raises(ValueError, match="weights: shape"):
        i8.expert_combine(Y, p, w[:2])
    with pytest.raises(TypeError, match="residual: torch.bfloat16"):
        i8.expert_combine(Y, p, w, residual=d.float())
    with pytest.raises(ValueError, match="out: shape"):
        i8.expert_combine(Y, p, w, out=t(3, 9))
    with pytest.raises(ValueError, match="dout: shape"):
        i8.expert_combine_bwd(t(4, 8), Y, p, w)
    with pytest.raises(ValueError, match="rows: 1-D tensor of 9"):
        i8.expert_combine_bwd(d, Y, p, w, rows=t(8, dtype=i32))


# ------------------------------------------------------------------ the C ABI

A = 1 << 20


def at(n, off=0):
    return A * n + off


def block(M=5, N=40, K=72, codes=at(1), exps=at(2), experts=0, offsets=None, bits=0, rows=None, X=at(3), ldx=72, tokens=5):
    return i8._Block(M, N, K, codes, exps, experts, offsets, bits, rows, X, ldx, tokens)


def test_block_abi():
    big = 1 << 18
    f = lambda p, Y=at(4), ldy=40, ws=at(5), n=big: L.i8mp_block_fwd(p, Y, ldy, 0, ws, n, None)  # noqa: E731
    rows200 = dict(M=200, tokens=200)
    assert accepted(lambda: f(block(**rows200)))
    assert f(None) == EINVAL
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 28, tokens=1 << 28), dict(N=1 << 23), dict(K=1 << 23, ldx=1 << 23),
                dict(codes=None), dict(exps=None), dict(codes=at(1, 8)), dict(X=None), dict(X=at(3, 8)), dict(ldx=64), dict(ldx=76),
                dict(tokens=4), dict(experts=-1), dict(experts=1 << 16, offsets=at(6), bits=32), dict(experts=2), dict(offsets=at(6)),
                dict(experts=2, offsets=at(6), bits=16), dict(experts=2, offsets=at(6, 4), bits=64), dict(rows=at(7, 2)),
                dict(rows=at(7), tokens=-1), dict(rows=at(7), tokens=0)):
        assert f(block(**bad)) == EINVAL, bad
    assert f(block(), Y=None) == EINVAL and f(block(), ldy=39) == EINVAL
    for over in (at(1, 16), at(2), at(3, 64)):
        assert f(block(), Y=over) == EINVAL
    assert f(block(**rows200), ws=None) == EWORKSPACE and f(block(**rows200), n=100) == EWORKSPACE
    assert f(block(**rows200), ws=at(5, 8)) == EWORKSPACE
    assert f(block(**rows200), ws=at(4)) == EINVAL  # over Y
    assert f(block(M=0, tokens=0, X=None)) == 0
    g = lambda p, dY=at(8), ld=40, dX=at(9), ldx=72, dW=at(10), ldw=72, ws=at(5), n=big: L.i8mp_block_bwd(  # noqa: E731
        p, dY, ld, dX, ldx, dW, ldw, 0, ws, n, None)
    assert accepted(lambda: g(block()))
    assert g(block(), dY=None) == EINVAL and g(block(), dY=at(8, 2)) == EINVAL and g(block(), ld=44) == EINVAL
    assert g(block(), ldx=71) == EINVAL and g(block(), ldw=71) == EINVAL
    assert g(block(), dX=at(8)) == EINVAL and g(block(), dW=at(9)) == EINVAL and g(block(), dW=at(3)) == EINVAL
    assert g(block(), ws=None) == EWORKSPACE
    assert g(block(codes=None, exps=None)) == EINVAL and g(block(X=None)) == EINVAL
    assert accepted(lambda: g(block(codes=None, exps=None), dX=None))  # dW does not read the weights
    assert accepted(lambda: g(block(X=None), dW=None))  # dX does not read X
    assert g(block(experts=2, offsets=at(6), bits=32), ldw=80) == EINVAL
    assert g(block(), dX=None, dW=None) == 0
    q = L.i8mp_quantize_block_weight
    assert accepted(lambda: q(at(1), 2, 40, 72, 72, 40 * 72, at(2), at(3), None))
    for bad in ((None, 1, 40, 72, 72, 0), (at(1, 2), 1, 40, 72, 72, 0), (at(1), 0, 40, 72, 72, 0), (at(1), 1, 40, 72, 64, 0),
                (at(1), 1, 40, 72, 76, 0), (at(1), 2, 40, 72, 72, 2881), (at(1), 2, 40, 72, 72, -8)):
        assert q(*bad, at(2), at(3), None) == EINVAL, bad
    assert q(at(1), 1, 40, 72, 72, 0, at(2, 8), at(3), None) == EINVAL and q(at(1), 1, 40, 72, 72, 0, at(1), at(3), None) == EINVAL
    assert q(None, 1, 0, 72, 72, 0, None, None, None) == 0


def route(logits=at(1), T=6, E=8, ld=8, dtype=2, k=2, score=0, normalize=1):
    return i8._Route(logits, T, E, ld, dtype, k, score, normalize)


def test_route_abi():
    f = lambda p, w=at(2), e=at(3), pl=at(4), r=at(5), o=at(6), ws=None, n=0: L.i8mp_expert_route(p, w, e, pl, r, o, ws, n, None)  # noqa: E731
    assert accepted(lambda: f(route()))
    for bad in (dict(logits=None), dict(T=-1), dict(E=0), dict(E=1025, ld=1025), dict(ld=7), dict(dtype=3), dict(k=0), dict(k=9),
                dict(score=2), dict(T=1 << 30), dict(E=64, ld=64, k=33)):
        assert f(route(**bad)) == EINVAL, bad
    for n in ("w", "e", "pl", "r", "o"):
        assert f(route(), **{n: None}) == EINVAL and f(route(), **{n: at(9, 2)}) == EINVAL and f(route(), **{n: at(1)}) == EINVAL
    assert f(route(), w=at(3)) == EINVAL
    many = route(T=1000)
    assert L.i8mp_expert_route_workspace_bytes(256, 8, 2) == 0
    need = L.i8mp_expert_route_workspace_bytes(1000, 8, 2)
    assert need > 0 and f(many) == EWORKSPACE and f(many, ws=at(7), n=need - 1) == EWORKSPACE
    assert accepted(lambda: f(many, ws=at(7), n=need))
    assert f(many, ws=at(1), n=need) == EINVAL
    g = lambda p, e=at(3), d=at(2), out=at(8), ld=8: L.i8mp_expert_route_bwd(p, e, d, out, ld, None)  # noqa: E731
    assert accepted(lambda: g(route()))
    assert g(route(), e=None) == EINVAL and g(route(), d=None) == EINVAL and g(route(), out=None) == EINVAL
    assert g(route(), ld=7) == EINVAL and g(route(), out=at(1)) == EINVAL and g(route(), out=at(2)) == EINVAL
    assert g(route(T=0, logits=None), e=None, d=None, out=None) == 0


def combine(T=3, R=9, N=8, k=2, dtype=0, Y=at(1), ldy=8, places=at(2), weights=at(3)):
    return i8._Combine(T, R, N, k, dtype, Y, ldy, places, weights)


def test_combine_abi():
    f = lambda p, res=None, ldr=0, out=at(4), ldo=8: L.i8mp_expert_combine(p, res, ldr, out, ldo, None)  # noqa: E731
    assert accepted(lambda: f(combine())) and accepted(lambda: f(combine(weights=None), res=at(4), ldr=8))
    for bad in (dict(T=-1), dict(R=-1), dict(N=-1), dict(k=0), dict(dtype=3), dict(Y=None), dict(Y=at(1, 1)), dict(ldy=7),
                dict(places=None), dict(places=at(2, 2)), dict(weights=at(3, 2)), dict(T=1 << 30), dict(N=1 << 23, ldy=1 << 23)):
        assert f(combine(**bad)) == EINVAL, bad
    assert f(combine(), out=None) == EINVAL and f(combine(), ldo=7) == EINVAL
    for over in (at(1), at(2), at(3)):
        assert f(combine(), out=over) == EINVAL
    assert f(combine(), res=at(4, 2), ldr=8) == EINVAL and f(combine(), res=at(5), ldr=7) == EINVAL
    assert f(combine(T=0, places=None), out=None) == 0
    g = lambda p, d=at(5), ldd=8, rows=None, dY=at(6), ldg=8, dw=at(7): L.i8mp_expert_combine_bwd(p, d, ldd, rows, dY, ldg, dw, None)  # noqa: E731
    assert accepted(lambda: g(combine())) and accepted(lambda: g(combine(), rows=at(8), dw=None))
    assert g(combine(), d=None) == EINVAL and g(combine(), ldd=7) == EINVAL and g(combine(), ldg=7) == EINVAL
    assert g(combine(), dY=at(1)) == EINVAL and g(combine(), dY=at(5)) == EINVAL and g(combine(), dw=at(3)) == EINVAL
    assert g(combine(), rows=at(8, 2)) == EINVAL and g(combine(), dw=at(7, 2)) == EINVAL
    assert g(combine(), dY=None, dw=None) == 0


def test_structures_match_the_header():
    assert ctypes.sizeof(i8._Block) == 11 * 8 + 8 and ctypes.sizeof(i8._Route) == 48 and ctypes.sizeof(i8._Combine) == 64
