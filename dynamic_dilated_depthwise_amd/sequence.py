"""Sequence operators on the GPU: layer norm, short causal convolution, selective scan.

They carry a state space mixer over the pixels of a feature map (or any tokens): the layer
norm before it, the convolution of a few neighbours along the sequence and the scan
(``mixer.PixelMixer`` runs them together).  Each function has the name of its C entry point
in ``include/ddpm_seq.h`` without the prefix: it checks its arguments, allocates the outputs
and the workspace, and enqueues the library's kernels on ``stream`` (the current stream by
default).  The functions here know nothing of autograd; ``layer_norm``, ``causal_conv`` and
``selective_scan`` are their differentiable forms.  There is no CPU or PyTorch fallback.

Layouts (float32 or bfloat16 unless stated; ``L`` tokens, ``H`` heads in ``G`` groups):
  x of the norm [..., C], weight and bias [C]
  x of the convolution [batch, L, D], weight [D, W], bias [D], states [batch, W - 1, D]
  x of the scan [batch, L, H, P], dt [batch, L, H], B and C [batch, L, G, N];
  A, D, dt_bias [H] and states [batch, H, P, N] float32
Inputs along a sequence may be views whose last axis (scan: all but the first two) is
contiguous, such as the slices of one projection.  lengths and slots are int32 [batch]; see
the header for what they mean, and for widths (to 8) and state columns (to 128).
"""
import ctypes

import torch

from . import _DTYPES, _check, raw_library

__all__ = [
    "layer_norm_fwd", "layer_norm_bwd", "layer_norm",
    "causal_conv_fwd", "causal_conv_bwd", "causal_conv_step", "causal_conv",
    "selective_scan_fwd", "selective_scan_bwd", "selective_scan_step", "selective_scan",
    "MAX_WIDTH", "MAX_STATE",
]

MAX_WIDTH = 8
MAX_STATE = 128

_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_F32, _I32 = torch.float32, torch.int32


class _Scan(ctypes.Structure):
    """ddpm_scan of the C header."""
    _fields_ = ([(n, _P) for n in ("x", "dt", "B", "C", "A", "D", "dt_bias", "initial_state", "lengths")] +
                [(n, _I64) for n in ("batch", "length", "x_batch", "x_token", "dt_batch", "dt_token", "B_batch", "B_token",
                                     "C_batch", "C_token")] +
                [(n, ctypes.c_int32) for n in ("heads", "P", "groups", "N", "dtype")])


_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = raw_library()
        scan = ctypes.POINTER(_Scan)
        types = {
            "ddpm_layer_norm_fwd": [_P] * 6 + [_I64] * 3 + [ctypes.c_float, _I, _P],
            "ddpm_layer_norm_bwd": [_P] * 9 + [_I64] * 4 + [_I, _P],
            "ddpm_causal_conv_fwd": [_P] * 7 + [_I64] * 3 + [_I] + [_I64] * 2 + [_I, _P],
            "ddpm_causal_conv_bwd": [_P] * 12 + [_I64] * 3 + [_I] + [_I64] * 4 + [_I, _P],
            "ddpm_causal_conv_step": [_P] * 6 + [_I64] * 3 + [_I, _I64, _I, _P],
            "ddpm_selective_scan_fwd": [scan, _P, _P, _I, _P, _P],
            "ddpm_selective_scan_bwd": [scan, _P, _P, _I64, _I64] + [_P] * 11,
            "ddpm_selective_scan_step": [scan, _P, _P, _I64, _P, _P],
            "ddpm_layer_norm_bwd_workspace": [_I64, _I64, _I],
            "ddpm_causal_conv_bwd_workspace": [_I64, _I64, _I64, _I, _I],
            "ddpm_selective_scan_fwd_workspace": [scan],
            "ddpm_selective_scan_bwd_workspace": [scan],
        }
        for name, args in types.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = _I64 if name.endswith("_workspace") else _I
        _lib = lib
    return _lib


# ----------------------------------------------------------------------------- arguments
def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")


def _like(t, name, x, dtype, shape):
    """The pointer of a contiguous tensor of this dtype and shape on x's device."""
    _tensor(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != x.device:
        raise ValueError(f"{name} must be on {x.device} (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _maybe(t, name, x, dtype, shape):
    return None if t is None else _like(t, name, x, dtype, shape)


def _view(t, name, x, dtype, shape, axes):
    """Checks a tensor whose first `axes` axes may have any strides and whose others are contiguous."""
    _tensor(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != x.device:
        raise ValueError(f"{name} must be on {x.device} (got {t.device})")
    if not t.is_contiguous():
        want = 1
        for size, stride in zip(reversed(t.shape[axes:]), reversed(t.stride()[axes:])):
            if size != 1 and stride != want:
                raise ValueError(f"{name} must be contiguous after its first {axes} axes (got strides {t.stride()})")
            want *= size
    return t


def _dtype(x):
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {x.dtype}; use float32 or bfloat16")
    return code


def _dims(x, name, n):
    _tensor(x, name)
    if x.dim() != n:
        raise ValueError(f"{name} must have {n} axes (got shape {tuple(x.shape)})")
    if x.numel() == 0:
        raise ValueError(f"{name} must not be empty (got shape {tuple(x.shape)})")
    return x.shape


def _on_stream(f):
    """Adds `stream`: the call's tensors are allocated for it and its kernels run on it, with
    the device of the first argument current."""
    def call(x, *args, stream=None, **kw):
        if stream is not None:
            with torch.cuda.stream(stream):
                return f(x, *args, **kw)
        if isinstance(x, torch.Tensor) and x.is_cuda and x.device.index != torch.cuda.current_device():
            with torch.cuda.device(x.device):
                return f(x, *args, **kw)
        return f(x, *args, **kw)
    call.__name__ = call.__qualname__ = f.__name__
    call.__doc__ = f.__doc__
    return call


def _current():
    return torch.cuda.current_stream().cuda_stream


def _bytes(n, x):
    return torch.empty(n, device=x.device, dtype=torch.uint8)


# ---------------------------------------------------------------------------- layer norm
def _rows(x, name):
    """(rows, C, row stride) of [..., C]: contiguous, or two axes with contiguous rows."""
    _tensor(x, name)
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError(f"{name} must have a last axis and not be empty (got shape {tuple(x.shape)})")
    C = x.shape[-1]
    if x.is_contiguous():
        return x.numel() // C, C, C
    if x.dim() == 2 and (x.stride(1) == 1 or C == 1):
        return x.shape[0], C, x.stride(0)
    raise ValueError(f"{name} must be contiguous, or have two axes with contiguous rows (got strides {x.stride()})")


@_on_stream
def layer_norm_fwd(x, weight, bias, eps=1e-5, stats=False):
    """(y, mean, rstd) of the layer norm over the last axis; mean and rstd (float32, the shape
    of x without its last axis) are None unless stats, and are what layer_norm_bwd takes."""
    rows, C, row = _rows(x, "x")
    code = _dtype(x)
    w, b = _like(weight, "weight", x, x.dtype, (C,)), _like(bias, "bias", x, x.dtype, (C,))
    y = torch.empty(x.shape, device=x.device, dtype=x.dtype)
    mean = rstd = None
    if stats:
        mean = torch.empty(x.shape[:-1], device=x.device, dtype=_F32)
        rstd = torch.empty_like(mean)
    _check("ddpm_layer_norm_fwd", _load().ddpm_layer_norm_fwd(
        x.data_ptr(), w, b, y.data_ptr(), mean.data_ptr() if stats else None, rstd.data_ptr() if stats else None, rows, C,
        row, eps, code, _current()))
    return y, mean, rstd


@_on_stream
def layer_norm_bwd(grad, x, weight, mean, rstd):
    """(grad_x, grad_weight, grad_bias) from grad, of the shape of x, and the forward's statistics."""
    rows, C, row = _rows(x, "x")
    code = _dtype(x)
    if _rows(grad, "grad")[:2] != (rows, C) or grad.shape != x.shape or grad.dtype != x.dtype or grad.device != x.device:
        raise ValueError(f"grad must be as x, {x.dtype} {tuple(x.shape)} (got {grad.dtype} {tuple(grad.shape)})")
    w = _like(weight, "weight", x, x.dtype, (C,))
    m, r = _like(mean, "mean", x, _F32, x.shape[:-1]), _like(rstd, "rstd", x, _F32, x.shape[:-1])
    lib = _load()
    gx = torch.empty(x.shape, device=x.device, dtype=x.dtype)
    gw, gb = torch.empty_like(weight), torch.empty_like(weight)
    work = _bytes(lib.ddpm_layer_norm_bwd_workspace(rows, C, code), x)
    _check("ddpm_layer_norm_bwd", lib.ddpm_layer_norm_bwd(
        grad.data_ptr(), x.data_ptr(), w, m, r, gx.data_ptr(), gw.data_ptr(), gb.data_ptr(), work.data_ptr(), rows, C, row,
        _rows(grad, "grad")[2], code, _current()))
    return gx, gw, gb


# ----------------------------------------------------------------------- causal convolution
def _taps(x, weight, bias, D):
    _tensor(weight, "weight")
    if weight.dim() != 2 or weight.shape[0] != D or weight.shape[1] < 1:
        raise ValueError(f"weight must have shape ({D}, width) (got {tuple(weight.shape)})")
    W = weight.shape[1]
    return W, _like(weight, "weight", x, x.dtype, (D, W)), _like(bias, "bias", x, x.dtype, (D,))


def _conv_state(t, name, x, shape):
    if t is not None and shape[1] == 0:
        raise ValueError(f"{name} must be None with one tap")
    return _maybe(t, name, x, x.dtype, shape)


@_on_stream
def causal_conv_fwd(x, weight, bias, initial_state=None, lengths=None, return_state=False):
    """(y, state): silu of the causal convolution along the sequence, and the last W - 1 inputs
    (None unless return_state) that a later call takes as initial_state."""
    batch, L, D = _dims(x, "x", 3)
    code = _dtype(x)
    _view(x, "x", x, x.dtype, x.shape, 2)
    W, w, b = _taps(x, weight, bias, D)
    init = _conv_state(initial_state, "initial_state", x, (batch, W - 1, D))
    n = _maybe(lengths, "lengths", x, _I32, (batch,))
    y = torch.empty((batch, L, D), device=x.device, dtype=x.dtype)
    last = torch.empty((batch, W - 1, D), device=x.device, dtype=x.dtype) if return_state else None
    _check("ddpm_causal_conv_fwd", _load().ddpm_causal_conv_fwd(
        x.data_ptr(), w, b, init, n, y.data_ptr(), last.data_ptr() if return_state and W > 1 else None, batch, L, D, W,
        x.stride(0), x.stride(1), code, _current()))
    return y, last


@_on_stream
def causal_conv_bwd(grad, x, weight, bias, initial_state=None, lengths=None, grad_state=None):
    """(grad_x, grad_weight, grad_bias, grad_initial): the last is None without an initial_state.
    grad_state is the gradient of the state that the forward returned."""
    batch, L, D = _dims(x, "x", 3)
    code = _dtype(x)
    _view(x, "x", x, x.dtype, x.shape, 2)
    _view(grad, "grad", x, x.dtype, x.shape, 2)
    W, w, b = _taps(x, weight, bias, D)
    init = _conv_state(initial_state, "initial_state", x, (batch, W - 1, D))
    gs = _conv_state(grad_state, "grad_state", x, (batch, W - 1, D))
    n = _maybe(lengths, "lengths", x, _I32, (batch,))
    lib = _load()
    gx = torch.empty((batch, L, D), device=x.device, dtype=x.dtype)
    gw, gb = torch.empty_like(weight), torch.empty_like(bias)
    gi = torch.empty_like(initial_state) if initial_state is not None else None
    work = _bytes(lib.ddpm_causal_conv_bwd_workspace(batch, L, D, W, code), x)
    _check("ddpm_causal_conv_bwd", lib.ddpm_causal_conv_bwd(
        grad.data_ptr(), x.data_ptr(), w, b, init, n, gs, gx.data_ptr(), gw.data_ptr(), gb.data_ptr(),
        gi.data_ptr() if gi is not None else None, work.data_ptr(), batch, L, D, W, x.stride(0), x.stride(1),
        grad.stride(0), grad.stride(1), code, _current()))
    return gx, gw, gb, gi


@_on_stream
def causal_conv_step(x, weight, bias, state, slots=None):
    """y [batch, D] of one token x [batch, D] of each sequence; state [S, W - 1, D] (of sequence
    b at slots[b], or at b) is moved on by the token in place."""
    batch, D = _dims(x, "x", 2)
    code = _dtype(x)
    _view(x, "x", x, x.dtype, x.shape, 1)
    W, w, b = _taps(x, weight, bias, D)
    _tensor(state, "state")
    S = state.shape[0] if state.dim() == 3 else 0
    st = _like(state, "state", x, x.dtype, (S, W - 1, D))
    n = _maybe(slots, "slots", x, _I32, (batch,))
    y = torch.empty((batch, D), device=x.device, dtype=x.dtype)
    _check("ddpm_causal_conv_step", _load().ddpm_causal_conv_step(
        x.data_ptr(), w, b, st if W > 1 else None, n, y.data_ptr(), batch, S, D, W, x.stride(0), code, _current()))
    return y


# --------------------------------------------------------------------------- selective scan
def _scan(x, dt, A, B, C, D, dt_bias, initial_state, lengths, token):
    """The C call's struct; `token` for the single-token shapes, which lack the second axis."""
    lead = 1 if token else 2
    shape = _dims(x, "x", lead + 2)
    code = _dtype(x)
    H, P = shape[lead:]
    _dims(B, "B", lead + 2)
    G, N = B.shape[lead:]
    front = shape[:lead]
    if H % G:
        raise ValueError(f"{H} heads do not divide into {G} groups")
    for t, name, s in ((x, "x", (H, P)), (dt, "dt", (H,)), (B, "B", (G, N)), (C, "C", (G, N))):
        _view(t, name, x, x.dtype, front + s, lead)
    a, d, bias = (_like(t, name, x, _F32, (H,)) for t, name in ((A, "A"), (D, "D"), (dt_bias, "dt_bias")))
    batch, L = front[0], 1 if token else front[1]
    init = _maybe(initial_state, "initial_state", x, _F32, (batch, H, P, N))
    n = _maybe(lengths, "lengths", x, _I32, (batch,))

    def strides(t):
        return (t.stride(0), 0 if token else t.stride(1))

    return _Scan(x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(), a, d, bias, init, n, batch, L, *strides(x),
                 *strides(dt), *strides(B), *strides(C), H, P, G, N, code)


@_on_stream
def selective_scan_fwd(x, dt, A, B, C, D, dt_bias, initial_state=None, lengths=None, return_state=False, save=False):
    """(y, state, saved): the scan's output, the states behind the last tokens (None unless
    return_state) and, with save, what selective_scan_bwd needs from this call (else None)."""
    s = _scan(x, dt, A, B, C, D, dt_bias, initial_state, lengths, False)
    lib = _load()
    y = torch.empty(x.shape, device=x.device, dtype=x.dtype)
    last = torch.empty((s.batch, s.heads, s.P, s.N), device=x.device, dtype=_F32) if return_state else None
    work = _bytes(lib.ddpm_selective_scan_fwd_workspace(s), x)
    _check("ddpm_selective_scan_fwd", lib.ddpm_selective_scan_fwd(
        s, y.data_ptr(), last.data_ptr() if return_state else None, 1 if save else 0, work.data_ptr(), _current()))
    return y, last, work if save else None


@_on_stream
def selective_scan_bwd(grad, x, dt, A, B, C, D, dt_bias, saved, initial_state=None, lengths=None, grad_state=None):
    """(grad_x, grad_dt, grad_A, grad_B, grad_C, grad_D, grad_dt_bias, grad_initial): the last is
    None without an initial_state.  initial_state and lengths are the forward's, saved what it
    returned; grad_state is the gradient of the state that it returned."""
    s = _scan(x, dt, A, B, C, D, dt_bias, initial_state, lengths, False)
    _view(grad, "grad", x, x.dtype, x.shape, 2)
    gs = _maybe(grad_state, "grad_state", x, _F32, (s.batch, s.heads, s.P, s.N))
    lib = _load()
    sv = _like(saved, "saved", x, torch.uint8, (lib.ddpm_selective_scan_fwd_workspace(s),))

    def out(t):
        return torch.empty(t.shape, device=t.device, dtype=t.dtype)

    gx, gdt, gA, gB, gC, gD, gbias = out(x), out(dt), out(A), out(B), out(C), out(D), out(dt_bias)
    gi = out(initial_state) if initial_state is not None else None
    work = _bytes(lib.ddpm_selective_scan_bwd_workspace(s), x)
    _check("ddpm_selective_scan_bwd", lib.ddpm_selective_scan_bwd(
        s, sv, grad.data_ptr(), grad.stride(0), grad.stride(1), gs, gx.data_ptr(), gdt.data_ptr(), gA.data_ptr(),
        gB.data_ptr(), gC.data_ptr(), gD.data_ptr(), gbias.data_ptr(), gi.data_ptr() if gi is not None else None,
        work.data_ptr(), _current()))
    return gx, gdt, gA, gB, gC, gD, gbias, gi


@_on_stream
def selective_scan_step(x, dt, A, B, C, D, dt_bias, state, slots=None):
    """y [batch, H, P] of one token of each sequence (x [batch, H, P], dt [batch, H], B and C
    [batch, G, N]); state [S, H, P, N] float32 (of sequence b at slots[b], or at b) is moved on
    by the token in place."""
    s = _scan(x, dt, A, B, C, D, dt_bias, None, None, True)
    _tensor(state, "state")
    S = state.shape[0] if state.dim() == 4 else 0
    st = _like(state, "state", x, _F32, (S, s.heads, s.P, s.N))
    n = _maybe(slots, "slots", x, _I32, (s.batch,))
    y = torch.empty(x.shape, device=x.device, dtype=x.dtype)
    _check("ddpm_selective_scan_step", _load().ddpm_selective_scan_step(s, st, n, S, y.data_ptr(), _current()))
    return y


# ------------------------------------------------------------------------------- autograd
def _rowwise(t, axes):
    """t itself if its axes after the first `axes` are contiguous, else a contiguous copy."""
    want = 1
    for size, stride in zip(reversed(t.shape[axes:]), reversed(t.stride()[axes:])):
        if size != 1 and stride != want:
            return t.contiguous()
        want *= size
    return t


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps, stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, grad):
        return (*layer_norm_bwd(grad.contiguous(), *ctx.saved_tensors), None)


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, lengths):
        ctx.save_for_backward(x, weight, bias, initial_state, lengths)
        ctx.set_materialize_grads(False)
        return causal_conv_fwd(x, weight, bias, initial_state, lengths, return_state=True)

    @staticmethod
    def backward(ctx, grad, grad_state):
        x, weight, bias, initial_state, lengths = ctx.saved_tensors
        if grad is None:
            grad = torch.zeros_like(x, memory_format=torch.contiguous_format)
        gs = grad_state.contiguous() if grad_state is not None and weight.shape[1] > 1 else None
        return (*causal_conv_bwd(_rowwise(grad, 2), x, weight, bias, initial_state, lengths, gs), None)


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, dt_bias, initial_state, lengths):
        args = (x, dt, A, B, C, D, dt_bias)
        y, state, saved = selective_scan_fwd(*args, initial_state, lengths, return_state=True, save=True)
        ctx.save_for_backward(*args, saved, initial_state, lengths)
        ctx.set_materialize_grads(False)
        return y, state

    @staticmethod
    def backward(ctx, grad, grad_state):
        saved = ctx.saved_tensors
        if grad is None:
            grad = torch.zeros_like(saved[0], memory_format=torch.contiguous_format)
        gs = grad_state.contiguous() if grad_state is not None else None
        return (*selective_scan_bwd(_rowwise(grad, 2), *saved, gs), None)


def layer_norm(x, weight, bias, eps=1e-5):
    """Differentiable layer norm over the last axis."""
    return _LayerNorm.apply(x if x.dim() == 2 and x.stride(-1) == 1 else x.contiguous(), weight, bias, eps)


def causal_conv(x, weight, bias, initial_state=None, lengths=None):
    """Differentiable (y, state) of causal_conv_fwd."""
    return _CausalConv.apply(_rowwise(x, 2), weight, bias, initial_state, lengths)


def selective_scan(x, dt, A, B, C, D, dt_bias, initial_state=None, lengths=None):
    """Differentiable (y, state) of selective_scan_fwd."""
    return _SelectiveScan.apply(_rowwise(x, 2), _rowwise(dt, 2), A, _rowwise(B, 2), _rowwise(C, 2), D, dt_bias,
                                initial_state, lengths)
