"""The sequence operators' workloads: layer norm, the short causal convolution and the selective scan.

A case names an operator (``op``), a form (``prompt``: forward over whole sequences, ``train``: forward and backward,
``step``: one token of each sequence, the state updated in place) and its sizes.  ``run`` computes it in plain torch,
or through the package's own entry points where ``own`` is true; ``exact`` computes it in 64 bits from the definition,
token by token.

    layer norm       y = (x - mean) / sqrt(var + eps) * weight + bias over the last axis
    causal conv      u[t] = bias + sum_j weight[:, j] * x[t - (W - 1) + j];  y = silu(u)
    selective scan   dt = softplus(raw + dt_bias);  h[t] = exp(dt A) h[t-1] + dt x[t] (outer) B[t];
                     y[t] = h[t] C[t] + D x[t], one state [P, N] per head, B and C shared by the heads of a group

Sequences may be ragged (``lengths``): positions past a length give zero and leave the state alone.
"""
import math

import torch

own = False

EPS = 1e-5
CHUNK = 64  # tokens per chunk of the plain scan
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step's handful of rows: nothing but latency
        dict(name="norm_rows_bf16", op="norm", form="prompt", dtype="bf16", rows=7, C=1024),
        # training on the 256 x 256 map of 64 channels, a token a pixel
        dict(name="norm_train_pixels_f32", op="norm", form="train", dtype="f32", rows=65536, C=64),
        # training a wide model on an odd number of tokens
        dict(name="norm_train_wide_bf16", op="norm", form="train", dtype="bf16", rows=16381, C=2048),
        # a decoding batch in a larger cache of states
        dict(name="conv_step_bf16", op="conv", form="step", dtype="bf16", batch=64, D=2304, W=4),
        # a few prompts of different lengths that go on from cached states
        dict(name="conv_prompt_ragged_f32", op="conv", form="prompt", dtype="f32", batch=3, L=1021, D=640, W=4, ragged=True),
        # training on long sequences; the channels of 32 heads of 64 and their B and C
        dict(name="conv_train_bf16", op="conv", form="train", dtype="bf16", batch=2, L=8192, D=2304, W=4, ragged=False),
        # one sequence, two heads: the smallest step
        dict(name="scan_step_one_f32", op="scan", form="step", dtype="f32", batch=1, H=2, P=64, G=1, N=64),
        # a large decoding batch: the state's traffic
        dict(name="scan_step_batch_bf16", op="scan", form="step", dtype="bf16", batch=256, H=32, P=64, G=1, N=128),
        # the pixels of the 256 x 256 map as one sequence, 64 channels expanded to two heads
        dict(name="scan_prompt_pixels_f32", op="scan", form="prompt", dtype="f32", batch=1, L=65536, H=2, P=64, G=1, N=64,
             ragged=False),
        # prompts of different lengths, from cached states to cached states
        dict(name="scan_prompt_ragged_bf16", op="scan", form="prompt", dtype="bf16", batch=4, L=4096, H=32, P=64, G=1, N=128,
             ragged=True),
        # training on long sequences
        dict(name="scan_train_bf16", op="scan", form="train", dtype="bf16", batch=2, L=8192, H=32, P=64, G=1, N=64,
             ragged=False),
        # training with odd sizes and two groups, ragged
        dict(name="scan_train_odd_f32", op="scan", form="train", dtype="f32", batch=2, L=1021, H=6, P=48, G=2, N=24,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["f32", "bf16"])
    kind = rng.choice(["norm prompt", "norm train", "conv step", "conv prompt", "conv train", "scan step", "scan prompt",
                       "scan prompt", "scan train", "scan train"])
    op, form = kind.split()
    most = (33_000_000 if op == "norm" else 18_000_000 if form == "train" else 33_000_000)
    if op == "norm":
        C = _log(rng, 16, 6000)
        return dict(op=op, form=form, dtype=dtype, rows=_log(rng, 1, max(2, min(65536, most // C))), C=C)
    if op == "conv":
        D, W = _log(rng, 16, 4000), rng.choice([2, 3, 4])
        if form == "step":
            return dict(op=op, form=form, dtype=dtype, batch=_log(rng, 1, 512), D=D, W=W)
        batch = rng.choice([1, 1, 2, 3, 5, 8])
        L = _log(rng, 1, max(2, min(32768, most // (D * batch))))
        return dict(op=op, form=form, dtype=dtype, batch=batch, L=L, D=D, W=W, ragged=rng.random() < 0.5)
    P, N = rng.choice([16, 32, 40, 48, 64, 64, 96, 128]), rng.choice([16, 24, 32, 50, 64, 64, 100, 128])
    G = rng.choice([1, 1, 2, 4])
    H = G * rng.choice([1, 2, 3, 4, 8])
    if form == "step":
        return dict(op=op, form=form, dtype=dtype, batch=_log(rng, 1, max(2, min(512, 60_000_000 // (H * P * N)))), H=H, P=P,
                    G=G, N=N)
    most = (8_000_000 if dtype == "f32" else 16_000_000) if form == "train" else 8_000_000
    batch = rng.choice([1, 1, 2, 3, 5])
    L = _log(rng, 1, max(2, min(16384, most // (batch * H * P))))
    return dict(op=op, form=form, dtype=dtype, batch=batch, L=L, H=H, P=P, G=G, N=N, ragged=rng.random() < 0.5)


# ----------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = _DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    s = {"op": case["op"], "form": case["form"]}
    if case["op"] == "norm":
        R, C = case["rows"], case["C"]
        s["x"] = normal(R, C, scale=1.5) + normal(R, 1)
        s["weight"] = 1 + normal(C, scale=0.2)
        s["bias"] = normal(C, scale=0.2)
        if case["form"] == "train":
            s["grad"] = normal(R, C)
        return s
    Bt = case["batch"]
    if case["form"] == "step":
        # the states of a cache a quarter larger than the batch, at places in no order
        S = Bt + Bt // 4
        s["slots"] = torch.randperm(S, generator=gen, device="cuda")[:Bt].to(torch.int32)
    else:
        L = case["L"]
        s["lengths"] = None
        if case["ragged"]:
            n = torch.randint(L // 2, L + 1, (Bt,), generator=gen, device="cuda")
            n[0] = L
            s["lengths"] = n.to(torch.int32)
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        s["weight"] = uniform(D, W, lo=-1 / math.sqrt(W), hi=1 / math.sqrt(W)).to(dt)
        s["bias"] = normal(D, scale=0.1)
        if case["form"] == "step":
            s["x"] = normal(Bt, D)
            s["state"] = normal(S, W - 1, D)
            return s
        s["x"] = normal(Bt, L, D)
        s["initial"] = normal(Bt, W - 1, D) if case["form"] == "prompt" else None
        if case["form"] == "train":
            s["grad"] = normal(Bt, L, D)
        return s
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    s["A"] = -uniform(H, lo=1.0, hi=16.0)
    s["D"] = 1 + normal(H, scale=0.1, dtype=torch.float32)
    s["dt_bias"] = torch.log(torch.expm1(torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))))
    if case["form"] == "step":
        s["x"], s["dt"] = normal(Bt, H, P), normal(Bt, H, scale=0.5)
        s["B"], s["C"] = normal(Bt, G, N), normal(Bt, G, N)
        s["state"] = normal(S, H, P, N, dtype=torch.float32)
        return s
    s["x"], s["dt"] = normal(Bt, L, H, P), normal(Bt, L, H, scale=0.5)
    s["B"], s["C"] = normal(Bt, L, G, N), normal(Bt, L, G, N)
    s["initial"] = normal(Bt, H, P, N, dtype=torch.float32) if case["ragged"] and case["form"] == "prompt" else None
    if case["form"] == "train":
        s["grad"] = normal(Bt, L, H, P)
    return s


# ------------------------------------------------------------------------------------ plain torch
def _norm(x, weight, bias):
    xc = x - x.mean(-1, keepdim=True)
    return xc * torch.rsqrt((xc * xc).mean(-1, keepdim=True) + EPS) * weight + bias


def _silu(u):
    return u / (1 + torch.exp(-u))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _inside(L, lengths, device):
    """[B or 1, L] truth values: the positions before each sequence's length."""
    t = torch.arange(L, device=device)[None]
    return t < lengths[:, None] if lengths is not None else t >= 0


def _conv(x, weight, bias, initial, lengths):
    Bt, L, D = x.shape
    W = weight.shape[1]
    front = initial if initial is not None else x.new_zeros(Bt, W - 1, D)
    xp = torch.cat([front, x], 1)
    y = _silu(bias + sum(weight[:, j] * xp[:, j:j + L] for j in range(W)))
    y = torch.where(_inside(L, lengths, x.device)[..., None], y, 0)
    n = lengths.long() if lengths is not None else torch.full((Bt,), L, device=x.device)
    at = n[:, None] + torch.arange(W - 1, device=x.device)
    return y, xp.gather(1, at[..., None].expand(-1, -1, D))


def _scan(x, raw, A, B, C, D, dt_bias, initial, lengths):
    """The scan in chunks: products inside a chunk, and the chunks' states joined by one matrix of decays per head."""
    Bt, L, H, P = x.shape
    G, N = B.shape[2:]
    inside = _inside(L, lengths, x.device)[..., None]
    dt = torch.where(inside, _softplus(raw + dt_bias), 0)
    x = torch.where(inside[..., None], x, 0)
    pad = -L % CHUNK
    n = (L + pad) // CHUNK

    def chunks(t):  # [Bt, L, heads, ...] -> [Bt, heads, chunks, CHUNK, ...]
        t = torch.nn.functional.pad(t, [0, 0] * (t.dim() - 2) + [0, pad])
        return t.unflatten(1, (n, CHUNK)).movedim(3, 1)

    cx = chunks(x)
    cB, cC = (chunks(torch.where(inside[..., None], t, 0)) for t in (B, C))
    cB, cC = (t[:, :, None].expand(-1, -1, H // G, -1, -1, -1).flatten(1, 2) for t in (cB, cC))
    cdt = chunks(dt[..., None])[..., 0]
    s = torch.cumsum(cdt.double() * A.double()[:, None, None], -1)  # the decays' logarithms, from each chunk's start
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp((s[..., :, None] - s[..., None, :]).float().masked_fill(~low, -math.inf))
    y = ((cC @ cB.transpose(-1, -2)) * decay * cdt[..., None, :]) @ cx
    last = s[..., -1:]
    local = (cx * (torch.exp((last - s).float()) * cdt)[..., None]).transpose(-1, -2) @ cB  # [Bt, H, n, P, N]
    first = initial if initial is not None else x.new_zeros(Bt, H, P, N)
    local = torch.cat([first[:, :, None], local], 2)
    total = torch.cumsum(torch.nn.functional.pad(last[..., 0], (1, 0)), -1)
    lown = torch.ones(n + 1, n + 1, dtype=torch.bool, device=x.device).tril()
    across = torch.exp((total[..., :, None] - total[..., None, :]).float().masked_fill(~lown, -math.inf))
    states = (across @ local.flatten(-2)).unflatten(-1, (P, N))
    y = y + torch.exp(s.float())[..., None] * (cC @ states[:, :, :-1].transpose(-1, -2))
    y = y.movedim(1, 3).flatten(1, 2)[:, :L] + D[:, None] * x
    return torch.where(inside[..., None], y, 0), states[:, :, -1]


def _plain(s):
    dt = s["x"].dtype
    keys = {"norm": ("x", "weight", "bias"), "conv": ("x", "weight", "bias"),
            "scan": ("x", "dt", "A", "B", "C", "D", "dt_bias")}[s["op"]]
    v = [s[k].float() for k in keys]
    if s["form"] == "step":
        slots = s["slots"].long()
        old = s["state"][slots].float()
        if s["op"] == "conv":
            x, weight, bias = v
            new = torch.cat([old, x[:, None]], 1)
            y = _silu(bias + (new * weight.t()).sum(1))
            new = new[:, 1:]
        else:
            x, raw, A, B, C, D, dt_bias = v
            step = _softplus(raw + dt_bias)
            B, C = (t[:, :, None].expand(-1, -1, x.shape[1] // t.shape[1], -1).flatten(1, 2) for t in (B, C))
            new = torch.exp(step * A)[..., None, None] * old + (step[..., None] * x)[..., None] * B[:, :, None]
            y = (new * C[:, :, None]).sum(-1) + D[:, None] * x
        s["state"].index_copy_(0, slots, new.to(s["state"].dtype))
        return {"y": y.to(dt), "state": s["state"]}
    train = s["form"] == "train"
    v = [t.detach().requires_grad_(train) for t in v]
    initial = s["initial"].float() if s.get("initial") is not None else None
    with torch.set_grad_enabled(train):
        if s["op"] == "norm":
            y, last = _norm(*v), None
        elif s["op"] == "conv":
            y, last = _conv(*v, initial, s["lengths"])
            last = last.to(dt)
        else:
            y, last = _scan(*v, initial, s["lengths"])
    if train:
        grads = torch.autograd.grad(y, v, s["grad"].float())
        return {"y": y.detach().to(dt), **{"grad_" + k: g.to(s[k].dtype) for k, g in zip(keys, grads)}}
    return {"y": y.to(dt), "state": last} if last is not None else {"y": y.to(dt)}


# ------------------------------------------------------------------------------- the package's own
def _own(s):
    from dynamic_dilated_depthwise_amd import sequence as seq
    op, form = s["op"], s["form"]
    if op == "norm":
        x, w, b = s["x"], s["weight"], s["bias"]
        if form == "prompt":
            return {"y": seq.layer_norm_fwd(x, w, b, EPS)[0]}
        y, mean, rstd = seq.layer_norm_fwd(x, w, b, EPS, stats=True)
        gx, gw, gb = seq.layer_norm_bwd(s["grad"], x, w, mean, rstd)
        return {"y": y, "grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    if op == "conv":
        x, w, b = s["x"], s["weight"], s["bias"]
        if form == "step":
            return {"y": seq.causal_conv_step(x, w, b, s["state"], slots=s["slots"]), "state": s["state"]}
        if form == "prompt":
            y, last = seq.causal_conv_fwd(x, w, b, initial_state=s["initial"], lengths=s["lengths"], return_state=True)
            return {"y": y, "state": last}
        y, _ = seq.causal_conv_fwd(x, w, b, lengths=s["lengths"])
        gx, gw, gb, _ = seq.causal_conv_bwd(s["grad"], x, w, b, lengths=s["lengths"])
        return {"y": y, "grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    a = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dt_bias"])
    if form == "step":
        return {"y": seq.selective_scan_step(*a, s["state"], slots=s["slots"]), "state": s["state"]}
    if form == "prompt":
        y, last, _ = seq.selective_scan_fwd(*a, initial_state=s["initial"], lengths=s["lengths"], return_state=True)
        return {"y": y, "state": last}
    y, _, saved = seq.selective_scan_fwd(*a, lengths=s["lengths"], save=True)
    gx, gdt, gA, gB, gC, gD, gbias, _ = seq.selective_scan_bwd(s["grad"], *a, saved, lengths=s["lengths"])
    return {"y": y, "grad_x": gx, "grad_dt": gdt, "grad_A": gA, "grad_B": gB, "grad_C": gC, "grad_D": gD,
            "grad_dt_bias": gbias}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ least work
def work(case):
    e, form = _BYTES[case["dtype"]], case["form"]
    if case["op"] == "norm":
        n = case["rows"] * case["C"]
        return {"bytes": n * e * (2 if form == "prompt" else 4), "flops": n * (8 if form == "prompt" else 24)}
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        if form == "step":
            n = case["batch"] * D
            return {"bytes": n * e * (2 + 2 * (W - 1)) + D * e * (W + 1), "flops": n * (2 * W + 6)}
        n = case["batch"] * case["L"] * D
        return {"bytes": n * e * (2 if form == "prompt" else 4) + D * e * (W + 1),
                "flops": n * (2 * W + 6) * (1 if form == "prompt" else 4)}
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    if form == "step":
        Bt = case["batch"]
        return {"bytes": Bt * (8 * H * P * N + e * (2 * H * P + H + 2 * G * N)), "flops": Bt * H * P * N * 5}
    T = case["batch"] * case["L"]
    bytes_ = T * e * (2 * H * P + H + 2 * G * N)
    if form == "train":
        return {"bytes": 2 * bytes_, "flops": T * H * P * N * 15}
    state = 4 * case["batch"] * H * P * N
    return {"bytes": bytes_ + state * (2 if case["ragged"] else 1), "flops": T * H * P * N * 5}


# ---------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t) for k, t in s.items()}
    if case["op"] == "norm":
        return _exact_norm(d)
    if case["op"] == "conv":
        return _exact_conv_step(d) if case["form"] == "step" else _exact_conv(d)
    return _exact_scan_step(d) if case["form"] == "step" else _exact_scan(d)


def _exact_norm(d):
    x, w = d["x"], d["weight"]
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    std = (var + EPS).sqrt()
    xh = (x - mean) / std
    out = {"y": xh * w + d["bias"]}
    if "grad" in d:
        g = d["grad"]
        gw = g * w
        C = x.shape[1]
        out["grad_x"] = (gw * C - gw.sum(-1, keepdim=True) - xh * (gw * xh).sum(-1, keepdim=True)) / (C * std)
        out["grad_weight"], out["grad_bias"] = (g * xh).sum(0), g.sum(0)
    return out


def _exact_conv_step(d):
    slots = d["slots"].long()
    old = d["state"][slots]
    u = d["bias"] + d["x"] * d["weight"][:, -1]
    for j in range(old.shape[1]):
        u = u + old[:, j] * d["weight"][:, j]
    d["state"][slots] = torch.roll(torch.cat([d["x"][:, None], old[:, 1:]], 1), -1, 1)
    return {"y": u * torch.sigmoid(u), "state": d["state"]}


def _exact_conv(d):
    x, w = d["x"], d["weight"]
    Bt, L, D = x.shape
    W = w.shape[1]
    lengths = d["lengths"].tolist() if d["lengths"] is not None else [L] * Bt
    y, gx, last = torch.zeros_like(x), torch.zeros_like(x), x.new_zeros(Bt, W - 1, D)
    gw, gb = torch.zeros_like(w), torch.zeros_like(d["bias"])
    for b, n in enumerate(lengths):
        front = d["initial"][b] if d["initial"] is not None else x.new_zeros(W - 1, D)
        line = torch.cat([front, x[b, :n]])
        u = torch.nn.functional.conv1d(line.t()[None], w[:, None], d["bias"], groups=D)[0].t() if n else x.new_zeros(0, D)
        sig = torch.sigmoid(u)
        y[b, :n] = u * sig
        last[b] = line[n:]
        if "grad" in d:
            du = d["grad"][b, :n] * sig * (1 + u * (1 - sig))
            gline = torch.zeros_like(line)
            for j in range(W):
                gline[j:j + n] += w[:, j] * du
                gw[:, j] += (line[j:j + n] * du).sum(0)
            gx[b, :n] = gline[W - 1:]
            gb += du.sum(0)
    if "grad" in d:
        return {"y": y, "grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    return {"y": y, "state": last}


def _heads(t, H):
    return t[..., torch.arange(H, device=t.device) // (H // t.shape[-2]), :]


def _exact_scan_step(d):
    x, slots, H = d["x"], d["slots"].long(), d["x"].shape[1]
    step = torch.logaddexp(d["dt"] + d["dt_bias"], torch.zeros((), dtype=torch.float64, device=x.device))
    h = d["state"][slots] * torch.exp(step * d["A"])[:, :, None, None]
    h += torch.einsum("bhp,bhn->bhpn", x * step[..., None], _heads(d["B"], H))
    d["state"][slots] = h
    return {"y": torch.einsum("bhpn,bhn->bhp", h, _heads(d["C"], H)) + d["D"][:, None] * x, "state": d["state"]}


def _exact_scan(d):
    x, A, Dh = d["x"], d["A"], d["D"]
    Bt, L, H, P = x.shape
    G, N = d["B"].shape[2:]
    train = "grad" in d
    states = L * Bt * H * P * N * 8
    if states > 60e9 and train:
        return None
    n = d["lengths"] if d["lengths"] is not None else torch.full((Bt,), L, device=x.device)
    on = (torch.arange(L, device=x.device)[:, None] < n).double()  # [L, Bt]
    v = (d["dt"] + d["dt_bias"]).movedim(1, 0)
    step = torch.logaddexp(v, torch.zeros_like(v)) * on[..., None]  # [L, Bt, H]
    a = torch.exp(step * A)[..., None, None]
    xt, Bh, Ch = x.movedim(1, 0), _heads(d["B"], H).movedim(1, 0), _heads(d["C"], H).movedim(1, 0)
    sx = (step[..., None] * xt)[..., None]
    h = d["initial"].clone() if d["initial"] is not None else x.new_zeros(Bt, H, P, N)
    kept = x.new_empty(L, Bt, H, P, N) if train else None
    y = torch.empty_like(xt)
    for t in range(L):
        h = torch.addcmul(a[t] * h, sx[t], Bh[t][:, :, None])
        if train:
            kept[t] = h
        y[t] = (h @ Ch[t][..., None])[..., 0]
    y = (y + Dh[:, None] * xt) * on[:, :, None, None]
    if not train:
        return {"y": y.movedim(0, 1), "state": h}
    gy = d["grad"].movedim(1, 0) * on[:, :, None, None]
    g = torch.zeros_like(h)
    gx, gstep = torch.empty_like(xt), torch.empty_like(step)
    gBh, gCh, gA = torch.empty_like(Bh), torch.empty_like(Ch), torch.zeros_like(A)
    zero = torch.zeros_like(h)
    for t in range(L - 1, -1, -1):
        g = torch.addcmul(g, gy[t][..., None], Ch[t][:, :, None])
        gB = (g @ Bh[t][..., None])[..., 0]  # [Bt, H, P]
        gx[t] = step[t][..., None] * gB
        gBh[t] = (sx[t].transpose(-1, -2) @ g)[:, :, 0]
        gCh[t] = (gy[t][:, :, None] @ kept[t])[:, :, 0]
        e = a[t][..., 0, 0] * (g * (kept[t - 1] if t else zero)).sum((-1, -2))
        gstep[t] = (gB * xt[t]).sum(-1) + A * e
        gA += (step[t] * e).sum(0)
        g = g * a[t]
    del kept
    gx = (gx + Dh[:, None] * gy) * on[:, :, None, None]
    graw = gstep * torch.sigmoid(v) * on[..., None]
    per = H // G

    def grouped(t):  # [L, Bt, H, N] -> [Bt, L, G, N]
        return (t * on[:, :, None, None]).unflatten(2, (G, per)).sum(3).movedim(0, 1)

    return {"y": y.movedim(0, 1), "grad_x": gx.movedim(0, 1), "grad_dt": graw.movedim(0, 1), "grad_A": gA,
            "grad_B": grouped(gBh), "grad_C": grouped(gCh), "grad_D": (gy * xt).sum((0, 1, 3)),
            "grad_dt_bias": graw.sum((0, 1))}
