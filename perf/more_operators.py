"""The feed-forward operators' workloads: products with an epilogue and the gated feed-forward projection.

A case names an operator (``op``), a form (``forward``, or ``train``: forward and backward) and its sizes: ``rows``
tokens, ``C`` channels in, ``N`` out.  ``run`` computes it in plain torch, or through the package's own entry points where
``own`` is true; ``exact`` computes it in 64 bits from the definition.

    linear   z = x W^T + bias;  y = act(z) + residual                    x [rows, C], W [N, C]
    gated    [g, u] = x W^T + bias, N columns each;  y = act(g) * u      x [rows, C], W [2 N, C]

Gradients: dz = grad * act'(z) (gated: dg = grad * u * act'(g), du = grad * act(g)); grad_x = dz W, grad_weight = dz^T x,
grad_bias the column sums of dz.  The residual's gradient is grad itself.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token through a small projection: nothing but latency
        dict(name="linear_token_f32", op="linear", form="forward", dtype="f32", rows=1, C=128, N=64, act="none", bias=True,
             residual=True),
        # a decoding batch's projection back to the model's width: the weights' traffic
        dict(name="linear_tokens_bf16", op="linear", form="forward", dtype="bf16", rows=48, C=5632, N=2048, act="none",
             bias=False, residual=True),
        # the pixels of the 256 x 256 map, 128 hidden channels back to 64
        dict(name="linear_pixels_f32", op="linear", form="forward", dtype="f32", rows=65536, C=128, N=64, act="none", bias=True,
             residual=True),
        # an odd number of tokens through a layer whose sizes divide by nothing
        dict(name="linear_odd_bf16", op="linear", form="forward", dtype="bf16", rows=4093, C=1021, N=2303, act="gelu", bias=True,
             residual=False),
        # training the projection back to the model's width
        dict(name="linear_train_bf16", op="linear", form="train", dtype="bf16", rows=16384, C=5632, N=2048, act="none",
             bias=True, residual=True),
        # training a projection with an activation in float32
        dict(name="linear_train_f32", op="linear", form="train", dtype="f32", rows=2048, C=1024, N=2304, act="gelu", bias=True,
             residual=False),
        # one token through the gated projection of a wide model
        dict(name="gated_token_bf16", op="gated", form="forward", dtype="bf16", rows=1, C=2048, N=5632, act="silu", bias=False),
        # a decoding batch
        dict(name="gated_tokens_bf16", op="gated", form="forward", dtype="bf16", rows=24, C=2048, N=5632, act="silu", bias=False),
        # prompts
        dict(name="gated_prompt_bf16", op="gated", form="forward", dtype="bf16", rows=8192, C=2048, N=5632, act="silu",
             bias=False),
        # training a wide model
        dict(name="gated_train_bf16", op="gated", form="train", dtype="bf16", rows=16384, C=2048, N=5632, act="silu", bias=True),
        # training on the pixels of the 256 x 256 map of 64 channels
        dict(name="gated_train_pixels_f32", op="gated", form="train", dtype="f32", rows=65536, C=64, N=128, act="silu",
             bias=True),
        # training on an odd number of tokens with odd sizes
        dict(name="gated_train_odd_bf16", op="gated", form="train", dtype="bf16", rows=2045, C=321, N=867, act="gelu", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, form = rng.choice(["linear", "gated"]), rng.choice(["forward", "forward", "train"])
    dtype = rng.choice(["f32", "bf16"])
    few = form == "forward" and rng.random() < 0.4  # tokens of a decoding batch
    while True:
        rows = _log(rng, 1, 96) if few else _log(rng, 16, 65536)
        C, N = _log(rng, 16, 6000), _log(rng, 16, 6000)
        if rng.random() < 0.5:  # sizes as a model's configuration has them
            C, N = (-(-v // 64) * 64 for v in (C, N))
        products = (2 if op == "gated" else 1) * (3 if form == "train" else 1)
        if 2 * rows * C * N * products <= (1e11 if dtype == "f32" else 1e12) and rows * (C + 2 * N) <= 3e8:
            break
    case = dict(op=op, form=form, dtype=dtype, rows=rows, C=C, N=N, act=rng.choice(["none", "relu", "silu", "gelu"]),
                bias=rng.random() < 0.5)
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    return case


# ----------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = _DT[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dt)

    rows, C, N = case["rows"], case["C"], case["N"]
    out = 2 * N if case["op"] == "gated" else N
    s = {"op": case["op"], "form": case["form"], "act": case["act"]}
    s["x"] = normal(rows, C)
    s["weight"] = normal(out, C, scale=1 / math.sqrt(C))
    s["bias"] = normal(out, scale=0.1) if case["bias"] else None
    s["residual"] = normal(rows, N) if case.get("residual") else None
    s["grad"] = normal(rows, N) if case["form"] == "train" else None
    return s


# ------------------------------------------------------------------------------------ plain torch
def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _plain(s):
    dt, train = s["x"].dtype, s["form"] == "train"
    v = [s[k].float().requires_grad_(train) if s[k] is not None else None for k in ("x", "weight", "bias")]
    x, weight, bias = v
    with torch.set_grad_enabled(train):
        z = x @ weight.t()
        if bias is not None:
            z = z + bias
        if s["op"] == "gated":
            g, u = z.chunk(2, -1)
            y = _act(g, s["act"]) * u
        else:
            y = _act(z, s["act"])
            if s["residual"] is not None:
                y = y + s["residual"].float()
    out = {"y": y.detach().to(dt)}
    if train:
        names = [k for k, t in zip(("x", "weight", "bias"), v) if t is not None]
        grads = torch.autograd.grad(y, [t for t in v if t is not None], s["grad"].float())
        out.update({"grad_" + k: g.to(dt) for k, g in zip(names, grads)})
    return out


# ------------------------------------------------------------------------------- the package's own
def _own(s):
    from dynamic_dilated_depthwise_amd import feedforward as ff
    x, weight, act, train = s["x"], s["weight"], s["act"], s["form"] == "train"
    if s["op"] == "gated":
        y, saved = ff.gated_linear_fwd(x, weight, s["bias"], activation=act, save=train)
    else:
        y, saved = ff.linear_fwd(x, weight, s["bias"], s["residual"], activation=act, save=train)
    if not train:
        return {"y": y}
    bwd = ff.gated_linear_bwd if s["op"] == "gated" else ff.linear_bwd
    gx, gw, gb = bwd(s["grad"], x, weight, saved, activation=act)
    out = {"y": y, "grad_x": gx, "grad_weight": gw}
    if s["bias"] is not None:
        out["grad_bias"] = gb
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ least work
def work(case):
    e, rows, C, N = _BYTES[case["dtype"]], case["rows"], case["C"], case["N"]
    out = 2 * N if case["op"] == "gated" else N
    count = rows * C + out * C + rows * N
    count += out if case["bias"] else 0
    count += rows * N if case.get("residual") else 0
    flops = 2 * rows * C * out
    if case["form"] == "train":
        count += rows * N + rows * C + out * C + (out if case["bias"] else 0)
        flops *= 3
    return {"bytes": e * count, "flops": flops}


# ---------------------------------------------------------------------------------------- 64 bits
def _curve(z, act):
    """The activation and its derivative."""
    if act == "relu":
        on = (z > 0).double()
        return z * on, on
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    x, weight, bias, residual, grad = (s[k].double() if s[k] is not None else None
                                       for k in ("x", "weight", "bias", "residual", "grad"))
    N = case["N"]
    z = torch.nn.functional.linear(x, weight, bias)
    if case["op"] == "gated":
        a, da = _curve(z[:, :N], case["act"])
        y = a * z[:, N:]
    else:
        a, da = _curve(z, case["act"])
        y = a if residual is None else a + residual
    out = {"y": y}
    if grad is not None:
        dz = torch.cat([grad * z[:, N:] * da, grad * a], 1) if case["op"] == "gated" else grad * da
        out["grad_x"], out["grad_weight"] = torch.mm(dz, weight), torch.mm(dz.t().contiguous(), x)
        if bias is not None:
            out["grad_bias"] = dz.sum(0)
    return out
