"""Sequence operators on the GPU: layer norm, short causal convolution, selective scan.

They carry a state space mixer over the pixels of a feature map (or any tokens): the layer
norm before it, the convolution of a few neighbours along the sequence and the scan
(``mixer.PixelMixer`` runs them together).  Each function has the name of its C entry point
in ``include/ddpm_seq.h`` without the prefix: it checks its arguments, allocates the outputs
and the workspace, and enqueues the library's kernels on ``stream`` (the current stream by
default).  Wrong arguments raise TypeError or ValueError, what the library refuses
``DDPMError``.  The functions know nothing of autograd; ``layer_norm``, ``causal_conv`` and
``selective_scan`` are their differentiable forms (once, in reverse mode; inputs with a
forward-mode tangent raise).  There is no CPU or PyTorch fallback.

Layouts (float32 or bfloat16 unless stated; ``L`` tokens, ``H`` heads in ``G`` groups):
  x of the norm [..., C], weight and bias [C]
  x of the convolution [batch, L, D], weight [D, W], bias [D], states [batch, W - 1, D]
  x of the scan [batch, L, H, P], dt [batch, L, H], B and C [batch, L, G, N];
  A, D, dt_bias [H] and states [batch, H, P, N] float32
Inputs along a sequence may be views whose last axis (scan: all but the first two) is
contiguous, such as the slices of one projection.  Every size is at least one (a sequence of a
ragged batch may have no tokens).  lengths and slots are int32 [batch]; see
the header for what they mean, and for widths (to 8) and state columns (to 128).

The step functions write `state` in place as torch's in-place forms do: a state that requires grad
is refused in grad mode, and a backward pass that has kept the state raises after the step.

Streams: a call on a given `stream` does not wait for work on the current one that makes its
arguments; it keeps their memory from reuse until its own work is done.  All calls may be
captured into a graph.  Before a training step is captured, let go of every eager result that
still holds a graph of the same leaves: torch's engine joins the stream on which such a graph
was made, which a capture does not allow and which ends the process.

The checks and allocations are native (``csrc/seq_binding.cpp``): a single token's kernel
takes 3 us, the same checks in Python four times that.
"""
import os

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import raw_library

__all__ = [
    "layer_norm_fwd", "layer_norm_bwd", "layer_norm",
    "causal_conv_fwd", "causal_conv_bwd", "causal_conv_step", "causal_conv",
    "selective_scan_fwd", "selective_scan_bwd", "selective_scan_step", "selective_scan",
    "MAX_WIDTH", "MAX_STATE",
]

MAX_WIDTH = 8
MAX_STATE = 128

raw_library()  # the extension's own library, or the error that says how to build it
try:
    from . import _sequence
except ImportError as e:
    raise RuntimeError(f"the sequence operators' extension does not load from {os.path.dirname(__file__)} ({e}); build it "
                       "with `python -m dynamic_dilated_depthwise_amd.build`") from e


def layer_norm_fwd(x, weight, bias, eps=1e-5, stats=False, stream=None):
    """(y, mean, rstd) of the layer norm over the last axis; mean and rstd (float32, the shape
    of x without its last axis) are None unless stats, and are what layer_norm_bwd takes."""
    return _sequence.layer_norm_fwd(x, weight, bias, eps, stats, stream)


def layer_norm_bwd(grad, x, weight, mean, rstd, stream=None):
    """(grad_x, grad_weight, grad_bias) from grad, of the shape of x, and the forward's statistics."""
    return _sequence.layer_norm_bwd(grad, x, weight, mean, rstd, stream)


def causal_conv_fwd(x, weight, bias, initial_state=None, lengths=None, return_state=False, stream=None):
    """(y, state): silu of the causal convolution along the sequence, and the last W - 1 inputs
    (None unless return_state) that a later call takes as initial_state."""
    return _sequence.causal_conv_fwd(x, weight, bias, initial_state, lengths, return_state, stream)


def causal_conv_bwd(grad, x, weight, bias, initial_state=None, lengths=None, grad_state=None, stream=None):
    """(grad_x, grad_weight, grad_bias, grad_initial): the last is None without an initial_state.
    grad_state is the gradient of the state that the forward returned."""
    return _sequence.causal_conv_bwd(grad, x, weight, bias, initial_state, lengths, grad_state, stream)


def causal_conv_step(x, weight, bias, state, slots=None, stream=None):
    """y [batch, D] of one token x [batch, D] of each sequence; state [S, W - 1, D] (of sequence
    b at slots[b], or at b) is moved on by the token in place."""
    return _sequence.causal_conv_step(x, weight, bias, state, slots, stream)


def selective_scan_fwd(x, dt, A, B, C, D, dt_bias, initial_state=None, lengths=None, return_state=False, save=False,
                       stream=None):
    """(y, state, saved): the scan's output, the states behind the last tokens (None unless
    return_state) and, with save, what selective_scan_bwd needs from this call (else None)."""
    return _sequence.selective_scan_fwd(x, dt, A, B, C, D, dt_bias, initial_state, lengths, return_state, save, stream)


def selective_scan_bwd(grad, x, dt, A, B, C, D, dt_bias, saved, initial_state=None, lengths=None, grad_state=None,
                       stream=None):
    """(grad_x, grad_dt, grad_A, grad_B, grad_C, grad_D, grad_dt_bias, grad_initial): the last is
    None without an initial_state.  initial_state and lengths are the forward's, saved what it
    returned; grad_state is the gradient of the state that it returned."""
    return _sequence.selective_scan_bwd(grad, x, dt, A, B, C, D, dt_bias, saved, initial_state, lengths, grad_state, stream)


def selective_scan_step(x, dt, A, B, C, D, dt_bias, state, slots=None, stream=None):
    """y [batch, H, P] of one token of each sequence (x [batch, H, P], dt [batch, H], B and C
    [batch, G, N]); state [S, H, P, N] float32 (of sequence b at slots[b], or at b) is moved on
    by the token in place."""
    return _sequence.selective_scan_step(x, dt, A, B, C, D, dt_bias, state, slots, stream)


# ------------------------------------------------------------------------------- autograd
def _differentiated(*ts):
    """Whether autograd has to see the call.  A tangent counts in any grad mode: the autograd forms
    have no forward-mode rule and raise, where the plain call would drop it."""
    ts = [t for t in ts if t is not None]
    return (torch.is_grad_enabled() and any(t.requires_grad for t in ts) or
            forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in ts))


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
    @once_differentiable
    def backward(ctx, grad):
        return (*layer_norm_bwd(grad.contiguous(), *ctx.saved_tensors), None)


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, lengths):
        ctx.save_for_backward(x, weight, bias, initial_state, lengths)
        ctx.set_materialize_grads(False)
        return causal_conv_fwd(x, weight, bias, initial_state, lengths, return_state=True)

    @staticmethod
    @once_differentiable
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
    @once_differentiable
    def backward(ctx, grad, grad_state):
        saved = ctx.saved_tensors
        if grad is None:
            grad = torch.zeros_like(saved[0], memory_format=torch.contiguous_format)
        gs = grad_state.contiguous() if grad_state is not None else None
        return (*selective_scan_bwd(_rowwise(grad, 2), *saved, gs), None)


def layer_norm(x, weight, bias, eps=1e-5):
    """Differentiable layer norm over the last axis."""
    x = x if x.dim() == 2 and x.stride(-1) == 1 else x.contiguous()
    if not _differentiated(x, weight, bias):
        return layer_norm_fwd(x, weight, bias, eps)[0]
    return _LayerNorm.apply(x, weight, bias, eps)


def causal_conv(x, weight, bias, initial_state=None, lengths=None):
    """Differentiable (y, state) of causal_conv_fwd."""
    args = _rowwise(x, 2), weight, bias, initial_state
    if not _differentiated(*args):
        return causal_conv_fwd(*args, lengths, return_state=True)
    return _CausalConv.apply(*args, lengths)


def selective_scan(x, dt, A, B, C, D, dt_bias, initial_state=None, lengths=None):
    """Differentiable (y, state) of selective_scan_fwd."""
    args = _rowwise(x, 2), _rowwise(dt, 2), A, _rowwise(B, 2), _rowwise(C, 2), D, dt_bias, initial_state
    if not _differentiated(*args):
        return selective_scan_fwd(*args, lengths, return_state=True)[:2]
    return _SelectiveScan.apply(*args, lengths)
