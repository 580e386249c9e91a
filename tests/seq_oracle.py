"""The sequence operators from their definitions, token by token, in 64 bits on the CPU.

Besides each result comes its size: the same sums over the terms' absolute values, which is
what a rounding error of one term is relative to.
"""
import torch

F64 = torch.float64


def u(dtype):
    """Half a step of a type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def norm(x, weight, bias, eps, grad):
    """(y, grad_x, grad_weight, grad_bias) and their sizes."""
    x, weight, bias, grad = (t.detach().to(F64).cpu() for t in (x, weight, bias, grad))
    C = x.shape[-1]
    mean = x.mean(-1, keepdim=True)
    rs = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - mean) * rs
    gw = grad * weight
    gx = rs * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
    red = tuple(range(x.dim() - 1))
    out = (xh * weight + bias, gx, (grad * xh).sum(red), grad.sum(red))
    # x and the mean are both rounded relative to the row's largest values before they cancel
    big = x.abs().mean(-1, keepdim=True) + x.abs()
    xs = big * rs
    agw = gw.abs()
    sizes = (xs * weight.abs() + bias.abs(),
             rs * (agw + agw.mean(-1, keepdim=True) + xs * (agw * xs).mean(-1, keepdim=True)),
             (grad.abs() * xs).sum(red), grad.abs().sum(red))
    return out, sizes, C


def _conv(x, weight, bias, initial, lengths, positive=False):
    """y and the final state, differentiable; sequence by sequence."""
    B, L, D = x.shape
    W = weight.shape[1]
    ys, lasts = [], []
    for b in range(B):
        n = max(0, min(L, int(lengths[b]))) if lengths is not None else L
        front = initial[b] if initial is not None else torch.zeros(W - 1, D, dtype=F64)
        line = torch.cat([front, x[b, :n]])
        u_ = bias.expand(n, D)
        for j in range(W):
            u_ = u_ + weight[:, j] * line[j:j + n]
        y = u_ if positive else u_ * torch.sigmoid(u_)
        ys.append(torch.cat([y, torch.zeros(L - n, D, dtype=F64)]))
        lasts.append(line[n:])
    return torch.stack(ys), torch.stack(lasts)


def conv(x, weight, bias, initial=None, lengths=None, grad=None, grad_state=None):
    """dict of results and dict of sizes: y, state and, with grad, the gradients."""
    leaves = [t.detach().to(F64).cpu().requires_grad_() if t is not None else None for t in (x, weight, bias, initial)]
    y, last = _conv(*leaves, lengths)
    out = {"y": y.detach(), "state": last.detach()}
    ab = [t.detach().abs().requires_grad_() if t is not None else None for t in leaves]
    us, ls = _conv(*ab, lengths, positive=True)  # sum of the absolute terms of u
    size = {"y": us.detach(), "state": ls.detach()}  # |silu'| < 1.1
    if grad is not None:
        names = [n for n, t in zip(("grad_x", "grad_weight", "grad_bias", "grad_initial"), leaves) if t is not None]
        g = grad.detach().to(F64).cpu()
        total, stotal = (y * g).sum(), (us * g.abs() * (1 + us.detach())).sum()  # an error of u moves du by at most |g| of it
        if grad_state is not None and last.numel():
            gs = grad_state.detach().to(F64).cpu()
            total, stotal = total + (last * gs).sum(), stotal + (ls * gs.abs()).sum()
        live, alive = [t for t in leaves if t is not None], [t for t in ab if t is not None]
        out |= dict(zip(names, torch.autograd.grad(total, live, allow_unused=True)))
        size |= dict(zip(names, torch.autograd.grad(stotal, alive, allow_unused=True)))
        for d in (out, size):
            for k, t in zip(names, live):
                if d[k] is None:
                    d[k] = torch.zeros_like(t)
    return out, size


def conv_step(x, weight, bias, state, slots):
    """(y, size of y, the moved state)."""
    x, weight, bias, state = (t.detach().to(F64).cpu() for t in (x, weight, bias, state))
    state = state.clone()
    y, size = torch.zeros_like(x), torch.zeros_like(x)
    for b in range(x.shape[0]):
        at = int(slots[b]) if slots is not None else b
        if not 0 <= at < state.shape[0]:
            continue
        line = torch.cat([state[at], x[b:b + 1]])
        v = bias + (line * weight.t()).sum(0)
        y[b] = v * torch.sigmoid(v)
        size[b] = bias.abs() + (line * weight.t()).abs().sum(0)
        state[at] = line[1:]
    return y, size, state


def _scan(x, dt, dt_decay, A, B, C, D, initial, on):
    """y and the final state; dt where it scales the input and dt_decay where it decays, both
    already through softplus; `on` [batch, L] truth values."""
    Bt, L, H, P = x.shape
    per = H // B.shape[2]
    h = initial if initial is not None else torch.zeros(Bt, H, P, B.shape[3], dtype=F64)
    ys = []
    for t in range(L):
        Bh, Ch = B[:, t].repeat_interleave(per, 1), C[:, t].repeat_interleave(per, 1)
        new = (torch.exp(dt_decay[:, t] * A)[..., None, None] * h +
               (dt[:, t, :, None] * x[:, t])[..., None] * Bh[:, :, None])
        live = on[:, t, None, None, None]
        h = torch.where(live, new, h)
        y = (h * Ch[:, :, None]).sum(-1) + D[:, None] * x[:, t]
        ys.append(torch.where(live[..., 0], y, 0))
    return torch.stack(ys, 1), h


def scan(x, dt, A, B, C, D, dt_bias, initial=None, lengths=None, grad=None, grad_state=None):
    """dict of results and dict of sizes: y, state and, with grad, the gradients."""
    c = [t.detach().to(F64).cpu() if t is not None else None for t in (x, dt, A, B, C, D, dt_bias, initial)]
    x, dt, A, B, C, D, dt_bias, initial = c
    Bt, L, H, _ = x.shape
    on = torch.ones(Bt, L, dtype=torch.bool)
    if lengths is not None:
        on = torch.arange(L)[None] < lengths.cpu().clamp(0, L)[:, None]
    raw = dt + dt_bias
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    sig = torch.sigmoid(raw)

    def run(v):
        x, A, B, C, D, initial = v
        leaves = [t.clone().requires_grad_() if t is not None else None for t in (x, step, step, A, B, C, D, initial)]
        y, h = _scan(*leaves, on)
        if grad is None:
            return y.detach(), h.detach(), None
        g = grad.detach().to(F64).cpu()
        gs = grad_state.detach().to(F64).cpu() if grad_state is not None else None
        if v[0] is not vals[0]:
            g, gs = g.abs(), gs.abs() if gs is not None else None
        total = (y * g).sum() + ((h * gs).sum() if gs is not None else 0)
        live = [t for t in leaves if t is not None]
        got = torch.autograd.grad(total, live, allow_unused=True)
        got = [torch.zeros_like(t) if q is None else q for q, t in zip(got, live)]
        return y.detach(), h.detach(), got + ([None] if initial is None else [])

    vals = [x, A, B, C, D, initial]
    y, h, g = run(vals)
    ys, hs, gs_ = run([t.abs() if t is not None and t is not A else t for t in vals])
    out, size = {"y": y, "state": h}, {"y": ys, "state": hs}
    if grad is not None:
        def named(q):
            gx, g1, g2, gA, gB, gC, gD, gi = q
            return {"grad_x": gx, "grad_A": gA, "grad_B": gB, "grad_C": gC, "grad_D": gD, "grad_initial": gi}
        out |= named(g)
        size |= named(gs_)
        onf = on[..., None].to(F64)
        out["grad_dt"] = (g[1] + g[2]) * sig * onf
        # the decay's gradient is summed from differences inside a stretch of tokens: a
        # rounding is relative to all of what flows at this token or after it
        flow = (step * gs_[1]).flip(1).cumsum(1).flip(1)
        size["grad_dt"] = (gs_[1] + gs_[2].abs() + A.abs() * 2 * flow) * sig * onf
        size["grad_A"] = size["grad_A"].abs() + (2 * step * flow * onf).sum((0, 1))
        out["grad_dt_bias"], size["grad_dt_bias"] = out["grad_dt"].sum((0, 1)), size["grad_dt"].sum((0, 1))
    return out, size


def scan_step(x, dt, A, B, C, D, dt_bias, state, slots):
    """(y, size of y, the moved state, its size)."""
    x, dt, A, B, C, D, dt_bias, state = (t.detach().to(F64).cpu() for t in (x, dt, A, B, C, D, dt_bias, state))
    state = state.clone()
    size_s = state.abs()
    per = x.shape[1] // B.shape[1]
    y, size = torch.zeros_like(x), torch.zeros_like(x)
    for b in range(x.shape[0]):
        at = int(slots[b]) if slots is not None else b
        if not 0 <= at < state.shape[0]:
            continue
        raw = dt[b] + dt_bias
        step = torch.logaddexp(raw, torch.zeros_like(raw))
        Bh, Ch = B[b].repeat_interleave(per, 0), C[b].repeat_interleave(per, 0)
        a = torch.exp(step * A)[:, None, None]
        add = (step[:, None] * x[b])[..., None] * Bh[:, None]
        size_s[at] = a * state[at].abs() + add.abs()
        state[at] = a * state[at] + add
        y[b] = (state[at] * Ch[:, None]).sum(-1) + D[:, None] * x[b]
        size[b] = (size_s[at] * Ch[:, None].abs()).sum(-1) + (D[:, None] * x[b]).abs()
    return y, size, state, size_s


def check(got, want, size, dtype, name, operand=None, count=512):
    """|got - want| within: one rounding of the output to its type, `count` roundings of
    float32 (the longest sums here have a few hundred terms) and, where an operand of the
    terms is rounded to the type first, one such rounding, both relative to the size."""
    assert got.dtype == dtype, f"{name}: {got.dtype}"
    got = got.detach().to(F64).cpu()
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)}, want {tuple(want.shape)}"
    tol = u(dtype) * want.abs() + (count * u(torch.float32) + (u(operand) if operand is not None else 0)) * size
    # beyond that the types' own smallest numbers
    over = (got - want).abs() - (tol * (1 + u(dtype)) + 1e-37)
    assert bool((over <= 0).all()), (
        f"{name}: off by {float((got - want).abs().max()):.3g}, over the bound by {float(over.max()):.3g} "
        f"at {tuple(int(i) for i in torch.unravel_index(over.argmax(), over.shape)) if over.dim() else ()}")
