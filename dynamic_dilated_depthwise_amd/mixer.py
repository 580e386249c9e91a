"""Blocks over the pixels of a feature map: a state space mixer, ``PixelMixer(dim)(x)``, a gated
feed-forward, ``PixelFeedForward(dim, hidden)(x)``, and both, ``PixelBlock(dim, hidden)(x)``.

The feature maps that DDPM filters, [N, dim, H, W], mix neighbours by their taps; the mixer
carries information along the whole map.  Its pixels in row order are a sequence of H * W
tokens of ``dim`` channels:

    t = layer_norm(tokens)
    z, u, raw = split(in_proj(t))              z the gate, u = [v, B, C] channels, raw per head
    v, B, C = split(silu(causal_conv(u)))
    tokens + out_proj(selective_scan(v, raw, A, B, C, D, dt_bias) * silu(z))

with the norm, the convolution and the scan from ``sequence`` (HIP kernels, forward and
backward) and the two projections and the gate from torch.  A prompt that arrives in parts,
or token by token, runs through ``prompt`` and ``step`` with the states of the convolution and
the scan kept between calls; both give what one call over the whole sequence gives.

The feed-forward mixes the channels of each token by itself, all of it in HIP kernels (``sequence``
and ``feedforward``), forward and backward:

    h = gated_linear(layer_norm(tokens))       act(gate) * up, hidden channels
    tokens + h down^T + bias                   the residual in the product's epilogue
"""
import math

import torch
import torch.nn as nn
import torch.nn.functional as F

from . import feedforward as ff
from . import sequence as seq

__all__ = ["PixelMixer", "PixelFeedForward", "PixelBlock"]


def _inside(tokens, lengths):
    """[batch, L, 1] truth values: the tokens [batch, L, dim] before each sequence's length."""
    if lengths.dtype != torch.int32 or lengths.shape != tokens.shape[:1] or lengths.device != tokens.device:
        raise ValueError(f"lengths must be int32 of shape ({tokens.shape[0]},) on {tokens.device} (got "
                         f"{lengths.dtype}, {tuple(lengths.shape)}, {lengths.device})")
    return (torch.arange(tokens.shape[1], device=tokens.device) < lengths[:, None])[..., None]


def _over_map(x, dim, prompt):
    """prompt over the pixels of a map [N, dim, H, W] in row order."""
    if x.dim() != 4 or x.shape[1] != dim:
        raise ValueError(f"x must have shape (N, {dim}, H, W) (got {tuple(x.shape)})")
    out = prompt(x.flatten(2).transpose(1, 2).contiguous())
    return out.transpose(1, 2).unflatten(2, x.shape[2:])


class PixelMixer(nn.Module):
    """heads of head_dim channels each keep a [head_dim, state_dim] state; the heads of one of
    ``groups`` share B and C; width is the convolution's.  float32 or bfloat16, on the GPU;
    A, D and dt_bias enter the scan in float32 whatever the module's type.  Under autocast the
    projections run in its type, the operators between them and the states stay in the module's."""

    def __init__(self, dim=64, heads=2, head_dim=64, state_dim=64, groups=1, width=4, eps=1e-5):
        super().__init__()
        if heads % groups:
            raise ValueError(f"{heads} heads do not divide into {groups} groups")
        if not 2 <= width <= seq.MAX_WIDTH:
            raise ValueError(f"width must be 2 to {seq.MAX_WIDTH} (got {width})")
        if not 1 <= state_dim <= seq.MAX_STATE:
            raise ValueError(f"state_dim must be 1 to {seq.MAX_STATE} (got {state_dim})")
        self.dim, self.heads, self.head_dim = dim, heads, head_dim
        self.state_dim, self.groups, self.width, self.eps = state_dim, groups, width, eps
        self.inner, self.shared = heads * head_dim, groups * state_dim
        self.channels = self.inner + 2 * self.shared  # of the convolution
        self.norm_weight = nn.Parameter(torch.ones(dim))
        self.norm_bias = nn.Parameter(torch.zeros(dim))
        self.in_proj = nn.Linear(dim, self.inner + self.channels + heads, bias=False)
        self.conv_weight = nn.Parameter((torch.rand(self.channels, width) * 2 - 1) / math.sqrt(width))
        self.conv_bias = nn.Parameter(torch.zeros(self.channels))
        self.A_log = nn.Parameter(torch.log(1 + 15 * torch.rand(heads)))  # A = -exp(A_log), from -1 to -16
        self.D = nn.Parameter(torch.ones(heads))
        step = torch.exp(torch.rand(heads) * math.log(100)) * 1e-3  # softplus(dt_bias), from 1e-3 to 1e-1
        self.dt_bias = nn.Parameter(torch.log(torch.expm1(step)))
        self.out_proj = nn.Linear(self.inner, dim, bias=False)

    def new_state(self, slots):
        """(convolution's, scan's) states of `slots` sequences before their first token."""
        w = self.conv_weight
        return (w.new_zeros(slots, self.width - 1, self.channels),
                torch.zeros(slots, self.heads, self.head_dim, self.state_dim, device=w.device, dtype=torch.float32))

    def _enter(self, tokens):
        dtype = self.norm_weight.dtype
        if torch.is_autocast_enabled("cuda"):
            tokens = tokens.to(dtype)
        t = seq.layer_norm(tokens, self.norm_weight, self.norm_bias, self.eps)
        z, u, raw = self.in_proj(t).split([self.inner, self.channels, self.heads], -1)
        return z, u.to(dtype), raw.to(dtype)

    def _per_head(self, u):
        v, B, C = u.split([self.inner, self.shared, self.shared], -1)
        per_group = (self.groups, self.state_dim)
        return v.unflatten(-1, (self.heads, self.head_dim)), B.unflatten(-1, per_group), C.unflatten(-1, per_group)

    def _scan_parameters(self):
        return -torch.exp(self.A_log.float()), self.D.float(), self.dt_bias.float()

    def _leave(self, tokens, y, z):
        return tokens + self.out_proj(y.flatten(-2) * F.silu(z))

    def prompt(self, tokens, state=None, lengths=None):
        """(out, state): tokens [batch, L, dim], of which sequence b has lengths[b] (int32; L
        without lengths); state from new_state or an earlier call.  Past a length out repeats
        the tokens, which take part in nothing else: neither they nor gradients there need be finite."""
        if tokens.dim() != 3 or tokens.shape[2] != self.dim:
            raise ValueError(f"tokens must have shape (batch, length, {self.dim}) (got {tuple(tokens.shape)})")
        first, h = state if state is not None else (None, None)
        inside = _inside(tokens, lengths) if lengths is not None else None
        z, u, raw = self._enter(tokens if inside is None else torch.where(inside, tokens, 0))
        u, last = seq.causal_conv(u, self.conv_weight, self.conv_bias, first, lengths)
        v, B, C = self._per_head(u)
        A, D, bias = self._scan_parameters()
        y, h = seq.selective_scan(v, raw, A, B, C, D, bias, h, lengths)
        out = self._leave(tokens, y, z)
        return out if inside is None else torch.where(inside, out, tokens), (last, h)

    @torch.no_grad()
    def step(self, tokens, state, slots=None):
        """out [batch, dim] of one token of each sequence; sequence b's states, at slots[b]
        (int32; b without slots) of `state`, are moved on in place.  Inference only."""
        if tokens.dim() != 2 or tokens.shape[1] != self.dim:
            raise ValueError(f"tokens must have shape (batch, {self.dim}) (got {tuple(tokens.shape)})")
        line, h = state
        z, u, raw = self._enter(tokens)
        u = seq.causal_conv_step(u, self.conv_weight, self.conv_bias, line, slots)
        v, B, C = self._per_head(u)
        A, D, bias = self._scan_parameters()
        y = seq.selective_scan_step(v, raw, A, B, C, D, bias, h, slots)
        return self._leave(tokens, y, z)

    def forward(self, x):
        return _over_map(x, self.dim, lambda tokens: self.prompt(tokens)[0])


class PixelFeedForward(nn.Module):
    """Layer norm, a gated projection to ``hidden`` channels and the projection back, added to its input.
    float32 or bfloat16, on the GPU.  Under autocast everything runs in the module's type, and so does
    what comes out."""

    def __init__(self, dim=64, hidden=128, activation="silu", bias=True, eps=1e-5):
        super().__init__()
        if activation not in ff.ACTIVATIONS:
            raise ValueError(f"activation must be one of {', '.join(ff.ACTIVATIONS)} (got {activation!r})")
        if dim < 1 or hidden < 1:
            raise ValueError(f"dim and hidden must be at least one (got {dim}, {hidden})")
        self.dim, self.hidden, self.activation, self.eps = dim, hidden, activation, eps
        self.norm_weight = nn.Parameter(torch.ones(dim))
        self.norm_bias = nn.Parameter(torch.zeros(dim))
        self.up_weight = nn.Parameter((torch.rand(2 * hidden, dim) * 2 - 1) / math.sqrt(dim))  # the gate's rows first
        self.down_weight = nn.Parameter((torch.rand(dim, hidden) * 2 - 1) / math.sqrt(hidden))
        self.up_bias = nn.Parameter(torch.zeros(2 * hidden)) if bias else None
        self.down_bias = nn.Parameter(torch.zeros(dim)) if bias else None

    def tokens(self, tokens, lengths=None):
        """tokens [..., dim]; with lengths (int32) [batch, L, dim], of which sequence b has lengths[b]:
        past them out repeats the tokens, which take part in nothing else."""
        if tokens.dim() < 1 or tokens.shape[-1] != self.dim or lengths is not None and tokens.dim() != 3:
            raise ValueError(f"tokens must have shape ({'batch, length' if lengths is not None else '...'}, {self.dim}) "
                             f"(got {tuple(tokens.shape)})")
        inside = _inside(tokens, lengths) if lengths is not None else None
        x = tokens if inside is None else torch.where(inside, tokens, 0)
        if torch.is_autocast_enabled("cuda"):
            x = x.to(self.norm_weight.dtype)
        h = seq.layer_norm(x, self.norm_weight, self.norm_bias, self.eps)
        h = ff.gated_linear(h, self.up_weight, self.up_bias, self.activation)
        out = ff.linear(h, self.down_weight, self.down_bias, x)
        return out if inside is None else torch.where(inside, out, tokens.to(out.dtype))

    def forward(self, x):
        return _over_map(x, self.dim, self.tokens)


class PixelBlock(nn.Module):
    """A PixelMixer, then a PixelFeedForward: maps, prompts in parts and single tokens as the mixer
    takes them.  mixer: further arguments of PixelMixer."""

    def __init__(self, dim=64, hidden=128, activation="silu", bias=True, eps=1e-5, **mixer):
        super().__init__()
        self.dim = dim
        self.mixer = PixelMixer(dim, eps=eps, **mixer)
        self.feed_forward = PixelFeedForward(dim, hidden, activation, bias, eps)

    def new_state(self, slots):
        """The mixer's states of `slots` sequences before their first token."""
        return self.mixer.new_state(slots)

    def prompt(self, tokens, state=None, lengths=None):
        """(out, state) as PixelMixer.prompt; past a length out repeats the tokens."""
        mixed, state = self.mixer.prompt(tokens, state, lengths)
        return self.feed_forward.tokens(mixed, lengths), state

    @torch.no_grad()
    def step(self, tokens, state, slots=None):
        """out [batch, dim] of one token of each sequence, as PixelMixer.step."""
        return self.feed_forward.tokens(self.mixer.step(tokens, state, slots))

    def forward(self, x):
        return _over_map(x, self.dim, lambda tokens: self.prompt(tokens)[0])
