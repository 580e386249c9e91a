"""The feed-forward operators from their definitions, in 64 bits with torch's own products.

Besides each result comes its size: the same sums over the terms' absolute values, which is what a
rounding error of one term is relative to, and what follows from the errors of what the sum is made of.
"""
import math

import torch

F64 = torch.float64
SLOPE, BEND = 1.13, 1.2  # the largest first (gelu 1.129, silu 1.100) and, doubled for room, second derivatives (0.80, 0.50)


def u(dtype):
    """Half a step of a type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def curve(z, act):
    """The activation and its derivative."""
    if act == "relu":
        on = (z > 0).to(F64)
        return z * on, on
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def run(x, weight, bias=None, residual=None, activation="none", grad=None, gated=False):
    """{name: (result, size, operand's size)}: the last is zero where no operand of the sum is rounded first."""
    x, weight, bias, residual, grad = (t.detach().to(F64) if t is not None else None for t in (x, weight, bias, residual, grad))
    lead = x.shape[:-1]
    x = x.reshape(-1, x.shape[-1])
    z, zs = x @ weight.t(), x.abs() @ weight.abs().t()
    if bias is not None:
        z, zs = z + bias, zs + bias.abs()
    N = z.shape[1] // (2 if gated else 1)
    a, da = curve(z[:, :N], activation)
    sa = a.abs() + SLOPE * zs[:, :N]
    if gated:
        y, ys = a * z[:, N:], sa * (z[:, N:].abs() + zs[:, N:])
    else:
        y, ys = a, sa
        if residual is not None:
            y, ys = y + residual.reshape(-1, N), ys + residual.reshape(-1, N).abs()
    out = {"y": (y, ys, torch.zeros_like(y))}
    if grad is not None:
        g = grad.reshape(-1, N)
        sd = g.abs() * (da.abs() + BEND * zs[:, :N])
        if gated:
            dz = torch.cat([g * z[:, N:] * da, g * a], 1)
            ds = torch.cat([sd * (z[:, N:].abs() + zs[:, N:]), g.abs() * sa], 1)
        else:
            dz, ds = g * da, sd
        rounded = dz.abs() if gated or activation != "none" else torch.zeros_like(dz)
        w, ax, dt = weight.abs(), x.abs(), dz.t().contiguous()
        out["grad_x"] = (dz @ weight, ds @ w, rounded @ w)
        out["grad_weight"] = (dt @ x, ds.t().contiguous() @ ax, rounded.t().contiguous() @ ax)
        out["grad_bias"] = (dz.sum(0), ds.sum(0), rounded.sum(0))
        out["grad_x"] = tuple(t.reshape(*lead, -1) for t in out["grad_x"])
    out["y"] = tuple(t.reshape(*lead, N) for t in out["y"])
    return out


def check(got, want, dtype, name, count):
    """|got - want| within: one rounding of the output to its type, `count` roundings of float32 relative
    to the size (twice the terms of the sums that lead to it and 64 for the functions between are more
    than enough in any order) and one rounding of the operand to the type where there is one."""
    want, size, operand = want
    assert got.dtype == dtype, f"{name}: {got.dtype}"
    got = got.detach().to(F64)
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)}, want {tuple(want.shape)}"
    tol = u(dtype) * (want.abs() + operand) + count * u(torch.float32) * size
    over = (got - want).abs() - (tol * (1 + u(dtype)) + 1e-37)  # beyond that the types' own smallest numbers
    assert bool((over <= 0).all()), (
        f"{name}: off by {float((got - want).abs().max()):.3g}, over the bound by {float(over.max()):.3g} "
        f"at {tuple(int(i) for i in torch.unravel_index(over.argmax(), over.shape))}")
