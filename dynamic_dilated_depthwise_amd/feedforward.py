"""Feed-forward operators on the GPU: products with an epilogue and the gated projection.

They mix the channels of a token as the sequence operators mix tokens (``mixer.PixelFeedForward``
and ``mixer.PixelBlock`` run both).  Each function has the name of its C entry point in
``include/ddpm_ff.h`` without the prefix: it checks its arguments, allocates the outputs and the
workspace, and enqueues the library's kernels on ``stream`` (the current stream by default).
Wrong arguments raise TypeError or ValueError, what the library refuses ``DDPMError``.  The
functions know nothing of autograd; ``linear`` and ``gated_linear`` are their differentiable forms
(once, in reverse mode; inputs with a forward-mode tangent raise).  There is no CPU or PyTorch
fallback.

    linear         z = x weight^T + bias;  y = act(z) + residual
    gated_linear   [g, u] = x weight^T + bias;  y = act(g) * u

Layouts (float32 or bfloat16): x [..., C], y, residual and grad [..., N]; weight [N, C] and bias
[N], of gated_linear [2 N, C] (the gate's rows first) and [2 N].  x, residual and grad are
contiguous or have two axes with contiguous rows; weight and bias are contiguous.  Every size is at
least one.  activation is "none", "relu", "silu" or "gelu" (z times the normal distribution at z).

Sums are float32; outputs are rounded once, and nothing on the way.  Where an activation or a gate
lies between, its input is kept in float32 by the forward, or made again by the backward, and the
gradient of it enters the backward's two products in float32 or as two bfloat16 terms.

An infinity or NaN in a row of x or grad reaches that row of y or of grad_x and the parameters'
gradients, and no other row.  In float32 a sum that is infinite may come out as NaN.

Streams, captured graphs and training steps in them are as in ``sequence``.
"""
import os

import torch
from torch.autograd.function import once_differentiable

from . import raw_library
from .sequence import _differentiated

__all__ = ["linear_fwd", "linear_bwd", "linear", "gated_linear_fwd", "gated_linear_bwd", "gated_linear", "ACTIVATIONS"]

ACTIVATIONS = ("none", "relu", "silu", "gelu")

raw_library()  # the extension's own library, or the error that says how to build it
try:
    from . import _feedforward
except ImportError as e:
    raise RuntimeError(f"the feed-forward operators' extension does not load from {os.path.dirname(__file__)} ({e}); build it "
                       "with `python -m dynamic_dilated_depthwise_amd.build`") from e


def linear_fwd(x, weight, bias=None, residual=None, activation="none", save=False, stream=None):
    """(y, saved): saved is what linear_bwd needs from this call (None unless save, and without an activation)."""
    return _feedforward.linear_fwd(x, weight, bias, residual, activation, save, stream)


def linear_bwd(grad, x, weight, saved=None, activation="none", need_x=True, need_weight=True, stream=None):
    """(grad_x, grad_weight, grad_bias); grad_x is None unless need_x, the others unless need_weight.
    The residual's gradient is grad."""
    return _feedforward.linear_bwd(grad, x, weight, saved, activation, need_x, need_weight, stream)


def gated_linear_fwd(x, weight, bias=None, activation="silu", save=False, stream=None):
    """(y, saved): saved is what gated_linear_bwd needs from this call (None unless save)."""
    return _feedforward.gated_linear_fwd(x, weight, bias, activation, save, stream)


def gated_linear_bwd(grad, x, weight, saved, activation="silu", need_x=True, need_weight=True, stream=None):
    """(grad_x, grad_weight, grad_bias); grad_x is None unless need_x, the others unless need_weight."""
    return _feedforward.gated_linear_bwd(grad, x, weight, saved, activation, need_x, need_weight, stream)


# ------------------------------------------------------------------------------- autograd
def _rows(t):
    """t itself if it is contiguous or its rows are, else a contiguous copy."""
    return t if t.dim() == 2 and t.stride(-1) == 1 else t.contiguous()


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation):
        product = any(ctx.needs_input_grad[:3])  # the residual's gradient needs nothing
        y, saved = linear_fwd(x, weight, bias, residual, activation, save=product)
        if product:
            ctx.save_for_backward(x, weight, saved)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        nx, nw, nb, nr, _ = ctx.needs_input_grad
        gx = gw = gb = None
        if nx or nw or nb:
            x, weight, saved = ctx.saved_tensors
            gx, gw, gb = linear_bwd(_rows(grad), x, weight, saved, ctx.activation, nx, nw or nb)
        return gx, gw if nw else None, gb if nb else None, grad if nr else None, None


class _GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, activation):
        y, saved = gated_linear_fwd(x, weight, bias, activation, save=True)
        ctx.save_for_backward(x, weight, saved)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        nx, nw, nb, _ = ctx.needs_input_grad
        gx, gw, gb = gated_linear_bwd(_rows(grad), *ctx.saved_tensors, ctx.activation, nx, nw or nb)
        return gx, gw if nw else None, gb if nb else None, None


def linear(x, weight, bias=None, residual=None, activation="none"):
    """Differentiable product with its epilogue."""
    x, residual = _rows(x), _rows(residual) if residual is not None else None
    if not _differentiated(x, weight, bias, residual):
        return linear_fwd(x, weight, bias, residual, activation)[0]
    return _Linear.apply(x, weight, bias, residual, activation)


def gated_linear(x, weight, bias=None, activation="silu"):
    """Differentiable gated projection."""
    x = _rows(x)
    if not _differentiated(x, weight, bias):
        return gated_linear_fwd(x, weight, bias, activation)[0]
    return _GatedLinear.apply(x, weight, bias, activation)
