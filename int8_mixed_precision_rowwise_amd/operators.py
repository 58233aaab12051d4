"""Operators around the INT8 mixed-precision linears, bound like the linears.

Linear layers with bias, activation and residual in the INT8 GEMM's epilogue
(``linear_act_fwd``, ``linear_act_fwd_train``, ``linear_act_bwd``, and over weights
quantized once ``linear_wq_fwd``), rotary positions of query and key heads
(``rotary``) and the loss of a student's logits against a teacher's top logits
(``distill_loss``, ``distill_loss_bwd``, ``distill_loss_and_grad``), with the
tensors' checks, the current stream and the errors of the package's other calls;
every step of the computation runs in the library's HIP kernels.  ``training`` holds
their autograd forms.
"""
from __future__ import annotations

import ctypes
import math

import torch

import int8_mixed_precision_rowwise_amd as _pkg

__all__ = ["ACTIVATIONS", "linear_act_fwd", "linear_act_fwd_train", "linear_act_bwd", "linear_wq_fwd",
           "linear_act_workspace_bytes", "linear_wq_workspace_bytes", "rotary", "rotary_frequencies", "distill_loss", "distill_loss_bwd", "distill_loss_and_grad"]

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_PAIRS = {"half": 0, "interleaved": 1}
_POSITIONS = {torch.int64: 64, torch.int32: 32}


def _call(dev: torch.device, name: str, *args):
    """lib.<name>(*args, stream) on dev's current stream, its status checked."""
    f, index = getattr(_pkg.lib, name), dev.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        st = f(*args, stream)
    else:  # another GPU is current
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st:
        raise _pkg.I8mpError(st, name)


def _on_gpu(first: torch.Tensor, *others) -> bool:
    """Whether all the given tensors live on one GPU (the refusal's words come from _pkg._device)."""
    dev = first.get_device()
    if dev < 0:
        return False
    for t in others:
        if t is not None and t.get_device() != dev:
            return False
    return True


# A call for a few tokens is over in a few microseconds, which is what the
# checks below cost one after the other.  So each operator first asks whether
# everything is as it should be, reading every property once, and only a call
# that is not goes through the checks that find the words for it.


# --------------------------------------------------------------------------- linears with an epilogue

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_ACT = {a: i for i, a in enumerate(ACTIVATIONS)}
_bf = torch.bfloat16


def _ld2(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _ptr(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _new_rows(rows: int, cols: int, dev) -> torch.Tensor:
    """bf16 [rows, cols], every row at a 16-byte boundary (dense where cols is a multiple of 8)."""
    ld = (cols + 7) // 8 * 8
    t = torch.empty((rows, ld), dtype=_bf, device=dev)
    return t if ld == cols else t[:, :cols]


def _activation(name: str) -> int:
    if name not in _ACT:
        raise ValueError(f"activation must be one of {ACTIVATIONS}, got {name!r}")
    return _ACT[name]


def linear_act_workspace_bytes(M: int, N: int, K: int, backward: bool) -> int:
    return _pkg.lib.i8mp_linear_act_workspace_bytes(M, N, K, int(backward))


def linear_wq_workspace_bytes(M: int, N: int, K: int) -> int:
    return _pkg.lib.i8mp_linear_wq_workspace_bytes(M, N, K)


def _space(workspace, need: int, dev) -> torch.Tensor:
    """The workspace of a call, which the caller holds until the call has returned: the
    library lets other threads run while it launches, and a block given back before
    would be theirs on the same stream."""
    return torch.empty(max(need, 1), dtype=torch.uint8, device=dev) if workspace is None else workspace


def _act_forward(X, W, w_scale, bias, activation, residual, out, workspace, keep_z=False):
    """Checks of a forward; (the C structure, device, Y, Z)."""
    try:
        (M, K), (N, KW) = X.shape, W.shape
        sx, sw, act = X.stride(), W.stride(), _ACT[activation]
        fine = (X.dtype == _bf and K == KW and K > 0 and M > 0 and sx[1] == 1 and sx[0] >= K and sw[1] == 1 and sw[0] >= K
                and W.dtype == (_bf if w_scale is None else torch.int8) and _on_gpu(X, W, w_scale, bias, residual, out, workspace))
        if w_scale is not None:
            fine = fine and w_scale.shape == (N,) and w_scale.dtype == torch.float32 and w_scale.is_contiguous()
        if bias is not None:
            fine = fine and bias.shape == (N,) and bias.dtype == _bf and bias.is_contiguous()
        for t in (residual, out):
            if t is not None:
                st = t.stride()
                fine = fine and t.shape == (M, N) and t.dtype == _bf and st[1] == 1 and st[0] >= N
        if workspace is not None:
            fine = fine and workspace.dtype == torch.uint8 and workspace.dim() == 1 and workspace.is_contiguous()
    except (AttributeError, IndexError, KeyError, TypeError, ValueError):
        fine = False
    if not fine:
        _act_forward_checks(X, W, w_scale, bias, activation, residual, out, workspace)
        (M, K), N, act = X.shape, W.shape[0], _ACT[activation]
    dev = X.device
    Y = _new_rows(M, N, dev) if out is None else out
    Z = _new_rows(M, N, dev) if keep_z and act else None
    p = _pkg._LinearAct(M, N, K, X.data_ptr(), _ld2(X), None if w_scale is not None else W.data_ptr(), _ld2(W), act, _ptr(bias),
                        _ptr(residual), 0 if residual is None else _ld2(residual), Y.data_ptr(), _ld2(Y), _ptr(Z),
                        0 if Z is None else _ld2(Z))
    return p, dev, Y, Z


def _act_forward_checks(X, W, w_scale, bias, activation, residual, out, workspace):
    _activation(activation)
    _pkg._mat(X, "X", _bf)
    M, K = X.shape
    if w_scale is None:
        _pkg._mat(W, "W", _bf)
    else:
        _pkg._mat(W, "Wq", torch.int8)
    if W.shape[1] != K:
        raise ValueError(f"W: {K} columns expected (X is {tuple(X.shape)}), got {tuple(W.shape)}")
    N = W.shape[0]
    if w_scale is not None:
        _pkg._vec(w_scale, "w_scale", N)
    if bias is not None:
        _pkg._vec(bias, "bias", N, _bf)
    if residual is not None:
        _pkg._mat(residual, "residual", _bf, (M, N))
    if out is not None:
        _pkg._mat(out, "out", _bf, (M, N))
    if workspace is not None:
        _pkg._workspace(workspace)
    _pkg._device(X, W, w_scale, bias, residual, out, workspace)


def linear_act_fwd(X: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, activation: str = "none",
                   residual: torch.Tensor | None = None, rounding="rne", seed: int = 0, offset: int = 0,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Y = act(X @ W.T + bias) + residual, X [M, K] and W [N, K] quantized row-wise over K.

    bf16 tensors; X, W and residual may have rows further apart than they are
    long (16-byte aligned).  activation: one of ACTIVATIONS.  Bias, activation and
    residual are added in fp32 and Y is rounded once.  Y's rows start every 16
    bytes unless out is given."""
    p, dev, Y, _ = _act_forward(X, W, None, bias, activation, residual, out, workspace)
    ws = _space(workspace, linear_act_workspace_bytes(p.M, p.N, p.K, False), dev)
    _call(dev, "i8mp_linear_act_fwd", p, _pkg._opts(rounding, seed, offset), None, None, ws.data_ptr(), ws.numel())
    return Y


def linear_act_fwd_train(X: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, activation: str = "none",
                         residual: torch.Tensor | None = None, rounding="rne", seed: int = 0, offset: int = 0,
                         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """linear_act_fwd that also returns what linear_act_bwd needs: (Y, Z, colmax_x,
    colmax_w), Z the pre-activation (bf16; None without an activation) and the
    column maxima of X and W (fp32 [K])."""
    p, dev, Y, Z = _act_forward(X, W, None, bias, activation, residual, out, workspace, keep_z=True)
    cx = torch.empty(p.K, dtype=torch.float32, device=dev)
    cw = torch.empty(p.K, dtype=torch.float32, device=dev)
    ws = _space(workspace, linear_act_workspace_bytes(p.M, p.N, p.K, False), dev)
    _call(dev, "i8mp_linear_act_fwd", p, _pkg._opts(rounding, seed, offset), _ptr(cx), _ptr(cw), ws.data_ptr(), ws.numel())
    return Y, Z, cx, cw


def linear_wq_fwd(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None = None,
                  activation: str = "none", residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """linear_act_fwd over weights quantized once: int8 codes Wq [N, K] and fp32 scales
    w_scale [N], for instance from quantize_rowwise.  X is quantized to nearest."""
    if not isinstance(w_scale, torch.Tensor):
        raise TypeError(f"w_scale: torch.Tensor expected, got {type(w_scale).__name__}")
    p, dev, Y, _ = _act_forward(X, Wq, w_scale, bias, activation, residual, out, workspace)
    need = linear_wq_workspace_bytes(p.M, p.N, p.K)
    ws = _space(workspace, need, dev) if need else None  # few short rows take none
    _call(dev, "i8mp_linear_wq_fwd", p, _ptr(Wq), _ld2(Wq), _ptr(w_scale), None if ws is None else ws.data_ptr(),
          0 if ws is None else ws.numel())
    return Y


def linear_act_bwd(dY: torch.Tensor, Z: torch.Tensor | None, X: torch.Tensor, W: torch.Tensor, activation: str = "none",
                   rounding="rne", seed: int = 0, offset: int = 0, want_dx: bool = True, want_dw: bool = True,
                   want_dbias: bool = False, dX: torch.Tensor | None = None, dW: torch.Tensor | None = None,
                   dbias: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   colmax_x: torch.Tensor | None = None, colmax_w: torch.Tensor | None = None):
    """Backward of linear_act_fwd: (dX, dW, dbias), None for what is not wanted.

    dZ = dY act'(Z) rounded to bf16 is quantized along each contraction as in
    linear_bwd; dbias (fp32 [N]) sums the values before that rounding.  Z: the
    pre-activation from linear_act_fwd_train (not read without an activation).
    The residual's gradient is dY itself."""
    act = _activation(activation)
    _pkg._mat(dY, "dY", _bf)
    M, N = dY.shape
    if act:
        _pkg._mat(Z, "Z", _bf, (M, N))
    else:
        Z = None
    _pkg._mat(W, "W", _bf)
    if W.shape[0] != N:
        raise ValueError(f"W: {N} rows expected (dY is {tuple(dY.shape)}), got {tuple(W.shape)}")
    K = W.shape[1]
    _pkg._mat(X, "X", _bf, (M, K))
    for t, name, shape in ((dX, "dX", (M, K)), (dW, "dW", (N, K))):
        if t is not None:
            _pkg._mat(t, name, _bf, shape)
    for t, name, n in ((dbias, "dbias", N), (colmax_x, "colmax_x", K), (colmax_w, "colmax_w", K)):
        if t is not None:
            _pkg._vec(t, name, n)
    if workspace is not None:
        _pkg._workspace(workspace)
    dev = _pkg._device(dY, Z, X, W, dX, dW, dbias, workspace, colmax_x, colmax_w)
    dX = None if not want_dx else torch.empty((M, K), dtype=_bf, device=dev) if dX is None else dX
    dW = None if not want_dw else torch.empty((N, K), dtype=_bf, device=dev) if dW is None else dW
    dbias = None if not want_dbias else torch.empty(N, dtype=torch.float32, device=dev) if dbias is None else dbias
    p = _pkg._LinearActGrad(M, N, K, _ptr(dY), _ld2(dY), _ptr(Z), 0 if Z is None else _ld2(Z), _ptr(X), _ld2(X), _ptr(W),
                            _ld2(W), act, _ptr(dX), 0 if dX is None else _ld2(dX), _ptr(dW), 0 if dW is None else _ld2(dW),
                            _ptr(dbias))
    ws = _space(workspace, linear_act_workspace_bytes(M, N, K, True), dev)
    _call(dev, "i8mp_linear_act_bwd", p, _pkg._opts(rounding, seed, offset), _ptr(colmax_x), _ptr(colmax_w), ws.data_ptr(),
          ws.numel())
    return dX, dW, dbias


# --------------------------------------------------------------------------- rotary positions


def rotary_frequencies(rot: int, theta: float = 10000.0, factor: float = 1.0, original_length: int | None = None,
                       low: float = 1.0, high: float = 4.0, device=None) -> torch.Tensor:
    """float64 [rot / 2] frequencies theta ** (-2 i / rot) for ``rotary``.

    ``factor`` > 1 stretches positions for contexts longer than the trained
    one.  Alone it divides every frequency.  With ``original_length`` (the
    trained context) a frequency is left alone where that context holds at
    least ``high`` of its turns, divided where it holds at most ``low``, and
    in between the two are mixed linearly in the number of turns."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    if not (theta > 0 and factor > 0):
        raise ValueError(f"theta and factor must be positive, got {theta} and {factor}")
    f = theta ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    if original_length is None:
        f = f / factor
    else:
        if not (original_length > 0 and 0 < low < high):
            raise ValueError(f"original_length > 0 and 0 < low < high expected, got {original_length}, {low}, {high}")
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f.to(device) if device is not None else f


def _heads(t, name: str, dtype, lead=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: torch.Tensor expected, got {type(t).__name__}")
    if t.dtype != dtype or dtype not in _DTYPE:
        raise TypeError(f"{name}: {'bfloat16, float16 or float32' if dtype not in _DTYPE else dtype} tensor expected, got {t.dtype}")
    if t.dim() != 4:
        raise ValueError(f"{name}: 4-D tensor [batch, positions, heads, head size] expected, got {t.dim()}-D")
    if lead is not None and (t.shape[0], t.shape[1], t.shape[3]) != lead:
        raise ValueError(f"{name}: shape {(lead[0], lead[1], 'heads', lead[2])} expected, got {tuple(t.shape)}")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{name}: elements of a head must be adjacent (stride 1)")
    return t


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, freqs: torch.Tensor,
           pairs: str = "half", inverse: bool = False, out_q: torch.Tensor | None = None,
           out_k: torch.Tensor | None = None):
    """Query and key heads turned by their positions: (q', k').

    q [B, S, HQ, D] and k [B, S, HK, D] (bf16, fp16 or fp32; k may be None) may
    be views of a packed projection: only a head's own elements have to be
    adjacent.  positions: int64 or int32, [B, S] or [S].  freqs: float64
    [rot / 2], rot <= D (``rotary_frequencies``); elements from rot on are
    copied.  pairs: "half" pairs element i with i + rot / 2, "interleaved" 2i
    with 2i + 1.  ``inverse`` turns back, which is also the backward: it takes
    the gradients of q' and k' to those of q and k.  out_q / out_k: where to
    write, any strides; q and k themselves for a rotation in place."""
    try:
        B, S, HQ, D = q.shape
        dtype, half = q.dtype, freqs.shape[0]
        at = positions.shape
        fine = (dtype in _DTYPE and pairs in _PAIRS and 1 <= half and 2 * half <= D <= 4096 and D % 2 == 0
                and freqs.dtype == torch.float64 and freqs.dim() == 1 and freqs.is_contiguous() and positions.dtype in _POSITIONS
                and (at == (B, S) or at == (S,)) and _on_gpu(q, k, positions, freqs, out_q, out_k))
        xq = q.stride()
        fine = fine and xq[3] == 1
        HK = 0
        if k is not None:
            HK, xk = k.shape[2], k.stride()
            fine = fine and k.shape == (B, S, HK, D) and k.dtype == dtype and xk[3] == 1
        for out, heads in ((out_q, HQ), (out_k, HK if k is not None else -1)):
            if out is not None:
                fine = fine and out.shape == (B, S, heads, D) and out.dtype == dtype and out.stride(3) == 1
    except (AttributeError, IndexError, TypeError, ValueError):
        fine = False
    if not fine:
        _rotary_checks(q, k, positions, freqs, pairs, out_q, out_k)
        B, S, HQ, D = q.shape
        dtype, half, at, xq = q.dtype, freqs.shape[0], positions.shape, q.stride()
        HK, xk = (0, None) if k is None else (k.shape[2], k.stride())
    if out_q is None:
        out_q = torch.empty_like(q, memory_format=torch.contiguous_format)
    y = out_q.stride()
    hq = _pkg._Heads(q.data_ptr(), out_q.data_ptr(), HQ, xq[0], xq[1], xq[2], y[0], y[1], y[2])
    hk = None
    if k is not None:
        if out_k is None:
            out_k = torch.empty_like(k, memory_format=torch.contiguous_format)
        y = out_k.stride()
        hk = _pkg._Heads(k.data_ptr(), out_k.data_ptr(), HK, xk[0], xk[1], xk[2], y[0], y[1], y[2])
    p = positions.stride()
    _call(q.device, "i8mp_rotary", hq, hk, B, S, D, 2 * half, _DTYPE[dtype], _PAIRS[pairs], 1 if inverse else 0, positions.data_ptr(),
          _POSITIONS[positions.dtype], p[0] if len(at) == 2 else 0, p[-1], freqs.data_ptr())
    return out_q, out_k


def _rotary_checks(q, k, positions, freqs, pairs, out_q, out_k):
    """rotary's checks one by one: raises what is wrong with the first that fails."""
    dtype = q.dtype if isinstance(q, torch.Tensor) else None
    _heads(q, "q", dtype)
    B, S, HQ, D = q.shape
    HK = 0
    if k is not None:
        _heads(k, "k", dtype, (B, S, D))
        HK = k.shape[2]
    elif out_k is not None:
        raise ValueError("out_k given without k")
    if pairs not in _PAIRS:
        raise ValueError(f"pairs must be 'half' or 'interleaved', got {pairs!r}")
    if not isinstance(freqs, torch.Tensor) or freqs.dtype != torch.float64:
        raise TypeError("freqs: torch.float64 tensor expected")
    if freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError(f"freqs: contiguous 1-D tensor expected, got shape {tuple(freqs.shape)}")
    rot = 2 * freqs.shape[0]
    if D % 2 or D > 4096 or not 2 <= rot <= D:
        raise ValueError(f"an even head size of at most 4096 and 1 to {D // 2} frequencies expected, got {D} and {rot // 2}")
    if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int64, torch.int32):
        raise TypeError("positions: torch.int64 or torch.int32 tensor expected")
    if tuple(positions.shape) not in ((B, S), (S,)):
        raise ValueError(f"positions: shape {(B, S)} or {(S,)} expected, got {tuple(positions.shape)}")
    if out_q is not None:
        _heads(out_q, "out_q", dtype, (B, S, D))
        if out_q.shape[2] != HQ:
            raise ValueError(f"out_q: {HQ} heads expected, got {out_q.shape[2]}")
    if out_k is not None:
        _heads(out_k, "out_k", dtype, (B, S, D))
        if out_k.shape[2] != HK:
            raise ValueError(f"out_k: {HK} heads expected, got {out_k.shape[2]}")
    _pkg._device(q, k, positions, freqs, out_q, out_k)


# --------------------------------------------------------------------------- distillation loss

DISTILL_STATS = 8
DISTILL_MAX_KEPT = 1024


def _rows(t, name: str, dtypes, shape=None):
    """2-D tensor of one of `dtypes` with adjacent columns (any row stride that spans a row)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: torch.Tensor expected, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: {' or '.join(str(d) for d in dtypes)} tensor expected, got {t.dtype}")
    return _pkg._mat(t, name, t.dtype, shape)


def _per_row(t, name: str, dtypes, T: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: torch.Tensor expected, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: {' or '.join(str(d) for d in dtypes)} tensor expected, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != T:
        raise ValueError(f"{name}: 1-D tensor of {T} elements expected, got shape {tuple(t.shape)}")


def _distill(logits, teacher, idx, temperature, teacher_lse, labels, ce_weight, ignore_index, grad=None, stats=None,
             out=None, workspace=None, backward=False):
    """Checks of the loss's inputs: (the C structure, device, T, V)."""
    try:
        (T, V), (_, k) = logits.shape, teacher.shape
        sl, st, si = logits.stride(), teacher.stride(), idx.stride()
        fine = (T > 0 and 0 < k <= DISTILL_MAX_KEPT and V > 0 and teacher.shape[0] == T and idx.shape == teacher.shape
                and logits.dtype in _DTYPE and teacher.dtype in _DTYPE and idx.dtype in _POSITIONS
                and sl[1] == 1 and st[1] == 1 and si[1] == 1 and sl[0] >= V and st[0] >= k and si[0] >= k
                and 0 < temperature < math.inf and math.isfinite(ce_weight)
                and _on_gpu(logits, teacher, idx, teacher_lse, labels, grad, stats, out, workspace))
        if teacher_lse is not None:
            fine = fine and teacher_lse.shape == (T,) and teacher_lse.dtype == torch.float32 and teacher_lse.is_contiguous()
        if labels is not None:
            fine = fine and labels.shape == (T,) and labels.dtype in _POSITIONS and labels.is_contiguous()
        elif ce_weight:
            fine = False
        if backward:
            fine = fine and grad.shape == (T,) and grad.dtype == torch.float32
            if stats is not None:
                fine = fine and stats.shape == (T, DISTILL_STATS) and stats.dtype == torch.float64 and stats.is_contiguous()
            if out is not None:
                so = out.stride()
                fine = fine and out.shape == (T, V) and out.dtype == logits.dtype and so[1] == 1 and so[0] >= V
        if workspace is not None:
            fine = fine and workspace.dtype == torch.uint8 and workspace.dim() == 1 and workspace.is_contiguous()
    except (AttributeError, IndexError, TypeError, ValueError):
        fine = False
    if not fine:
        _distill_checks(logits, teacher, idx, temperature, teacher_lse, labels, ce_weight, grad, stats, out, workspace, backward)
        (T, V), k = logits.shape, teacher.shape[1]
    p = _pkg._Distill(logits.data_ptr(), T, V, _ld2(logits), _DTYPE[logits.dtype], teacher.data_ptr(), _ld2(teacher),
                      _DTYPE[teacher.dtype], idx.data_ptr(), _ld2(idx), _POSITIONS[idx.dtype], k,
                      temperature, None if teacher_lse is None else teacher_lse.data_ptr(),
                      None if labels is None else labels.data_ptr(),
                      0 if labels is None else _POSITIONS[labels.dtype], ignore_index, ce_weight)
    return p, logits.device, T, V


def _distill_checks(logits, teacher, idx, temperature, teacher_lse, labels, ce_weight, grad, stats, out, workspace, backward):
    _rows(logits, "logits", tuple(_DTYPE))
    T, V = logits.shape
    _rows(teacher, "teacher", tuple(_DTYPE))
    if teacher.shape[0] != T:
        raise ValueError(f"teacher: {T} rows expected (logits are {tuple(logits.shape)}), got {tuple(teacher.shape)}")
    k = teacher.shape[1]
    _rows(idx, "idx", (torch.int32, torch.int64), (T, k))
    if k > DISTILL_MAX_KEPT:
        raise ValueError(f"teacher: at most {DISTILL_MAX_KEPT} kept entries a row, got {k}")
    if V == 0 and T > 0:
        raise ValueError("logits: rows without classes")
    if not (0 < temperature < math.inf):
        raise ValueError(f"temperature must be positive and finite, got {temperature}")
    if not math.isfinite(ce_weight):
        raise ValueError(f"ce_weight must be finite, got {ce_weight}")
    if teacher_lse is not None:
        _pkg._vec(teacher_lse, "teacher_lse", T)
    if labels is not None:
        _per_row(labels, "labels", (torch.int64, torch.int32), T)
        if T > 1 and labels.stride(0) != 1:
            raise ValueError("labels: contiguous tensor expected")
    elif ce_weight:
        raise ValueError("ce_weight given without labels")
    if backward:
        _per_row(grad, "grad", (torch.float32,), T)
        if stats is not None:
            _pkg._mat(stats, "stats", torch.float64, (T, DISTILL_STATS), dense=True)
        if out is not None:
            _pkg._mat(out, "out", logits.dtype, (T, V))
    if workspace is not None:
        _pkg._workspace(workspace)
    _pkg._device(logits, teacher, idx, teacher_lse, labels, grad, stats, out, workspace)


def _distill_ws(p, dev, workspace):
    """The workspace to hold until the call has returned, or None."""
    need = _pkg.lib.i8mp_distill_workspace_bytes(p.T, p.V, p.kept, p.dtype)
    return _space(workspace, need, dev) if need else workspace


def _grad_out(logits, out, dev):
    """Where the gradient goes: rows as far apart as the logits', so that both sides start at the same place in a chunk."""
    if out is not None:
        return out
    T, V = logits.shape
    ld = _ld2(logits)
    if ld == V or ld > 2 * V:
        return torch.empty((T, V), dtype=logits.dtype, device=dev)
    return torch.empty((T, ld), dtype=logits.dtype, device=dev)[:, :V]


def distill_loss(logits: torch.Tensor, teacher: torch.Tensor, idx: torch.Tensor, temperature: float = 1.0,
                 teacher_lse: torch.Tensor | None = None, labels: torch.Tensor | None = None, ce_weight: float = 0.0,
                 ignore_index: int = -100, workspace: torch.Tensor | None = None):
    """Loss of each row of a student's logits against a teacher's kept top logits: (loss fp32 [T], stats).

    logits [T, V] (bf16, fp16 or fp32); teacher [T, k] (the same types) the
    teacher's logits of the classes idx [T, k] (int32 or int64; negative: no
    entry; distinct within a row; at most 1024).  With q = softmax(logits /
    temperature) and p the softmax of teacher / temperature over the kept
    classes, the loss is temperature^2 KL(p || q).  teacher_lse (fp32 [T], the
    log-sum-exp of all the teacher's logits / temperature) makes p the
    teacher's own probabilities and the classes not kept one more class.
    labels ([T], int64 or int32) with ce_weight add ce_weight times the cross
    entropy; rows labelled ignore_index (or outside the classes) add none, and
    rows without kept entries have no other part.  stats: float64 [T, 8], what
    distill_loss_bwd needs."""
    p, dev, T, _ = _distill(logits, teacher, idx, temperature, teacher_lse, labels, ce_weight, ignore_index, workspace=workspace)
    loss = torch.empty(T, dtype=torch.float32, device=dev)
    stats = torch.empty((T, DISTILL_STATS), dtype=torch.float64, device=dev)
    ws = _distill_ws(p, dev, workspace)
    _call(dev, "i8mp_distill_fwd", p, loss.data_ptr(), stats.data_ptr(), None if ws is None else ws.data_ptr(),
          0 if ws is None else ws.numel())
    return loss, stats


def distill_loss_bwd(logits: torch.Tensor, teacher: torch.Tensor, idx: torch.Tensor, stats: torch.Tensor,
                     grad: torch.Tensor, temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                     labels: torch.Tensor | None = None, ce_weight: float = 0.0, ignore_index: int = -100,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of sum(grad * loss) at the logits, in their type, from distill_loss's stats.

    grad: fp32 [T], any stride (an expanded scalar too); the other arguments as
    in the forward."""
    if not isinstance(stats, torch.Tensor):
        raise TypeError(f"stats: torch.Tensor expected, got {type(stats).__name__}")
    p, dev, T, V = _distill(logits, teacher, idx, temperature, teacher_lse, labels, ce_weight, ignore_index, grad, stats, out,
                            backward=True)
    d = _grad_out(logits, out, dev)
    _call(dev, "i8mp_distill_bwd", p, stats.data_ptr(), grad.data_ptr(), grad.stride(0), d.data_ptr(), _ld2(d))
    return d


def distill_loss_and_grad(logits: torch.Tensor, teacher: torch.Tensor, idx: torch.Tensor, grad: torch.Tensor,
                          temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                          labels: torch.Tensor | None = None, ce_weight: float = 0.0, ignore_index: int = -100,
                          out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """distill_loss and the gradient of sum(grad * loss) at the logits with one
    read of them: (loss, dlogits).  For training, where the rows' weights (1 / T
    for a mean) are known before the loss is."""
    p, dev, T, V = _distill(logits, teacher, idx, temperature, teacher_lse, labels, ce_weight, ignore_index, grad, None, out,
                            workspace, backward=True)
    d = _grad_out(logits, out, dev)
    loss = torch.empty(T, dtype=torch.float32, device=dev)
    ws = _distill_ws(p, dev, workspace)
    _call(dev, "i8mp_distill_step", p, grad.data_ptr(), grad.stride(0), loss.data_ptr(), d.data_ptr(), _ld2(d),
          None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    return loss, d
