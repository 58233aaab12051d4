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
