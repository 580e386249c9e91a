"""A state space mixer over the pixels of a feature map: ``PixelMixer(dim)(x)``.

The feature maps that DDPM filters, [N, dim, H, W], mix neighbours by their taps; this module
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
"""
import math

import torch
import torch.nn as nn
import torch.nn.functional as F

from . import sequence as seq

__all__ = ["PixelMixer"]


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
        inside = None
        if lengths is not None:
            if lengths.dtype != torch.int32 or lengths.shape != tokens.shape[:1] or lengths.device != tokens.device:
                raise ValueError(f"lengths must be int32 of shape ({tokens.shape[0]},) on {tokens.device} (got "
                                 f"{lengths.dtype}, {tuple(lengths.shape)}, {lengths.device})")
            inside = (torch.arange(tokens.shape[1], device=tokens.device) < lengths[:, None])[..., None]
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
        if x.dim() != 4 or x.shape[1] != self.dim:
            raise ValueError(f"x must have shape (N, {self.dim}, H, W) (got {tuple(x.shape)})")
        out, _ = self.prompt(x.flatten(2).transpose(1, 2).contiguous())
        return out.transpose(1, 2).unflatten(2, x.shape[2:])
