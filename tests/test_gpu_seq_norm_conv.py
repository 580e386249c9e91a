"""Layer norm and short causal convolution against their definitions in 64 bits, forward,
backward and by single tokens; refusals, streams, graphs.

Tolerances (seq_oracle.check): one rounding of the output plus 512 float32 roundings of the
sum's size; the longest sums here have under 512 terms but for the column sums of the tall
norm and the long convolution, which are joined pairwise in runs of fewer.
"""
import pytest
import torch

import seq_oracle as orc
from dynamic_dilated_depthwise_amd import sequence as seq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def announce(*a):
    print("[gpu case]", *a, flush=True)


def randn(gen, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=gen) * scale + shift).to(dtype).cuda()


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------- layer norm
# (rows, C): one element, one vector, tails of every length, each group width and vector
# count of both types, rows that only the workgroup or only the long kernel hold
NORM = [(1, 1), (3, 2), (5, 17), (33, 64), (2, 65), (7, 255), (4, 512), (3, 1023), (9, 1024), (2, 2047), (5, 4100), (3, 8192),
        (2, 8195), (2, 16390), (600, 24), (1100, 70)]


def norm_case(rows, C, dtype, seed=1):
    g = gen_of(seed)
    return (randn(g, rows, C, dtype=dtype, scale=1.5, shift=0.5), randn(g, C, dtype=dtype, scale=0.2, shift=1.0),
            randn(g, C, dtype=dtype, scale=0.2), randn(g, rows, C, dtype=dtype))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,C", NORM)
def test_layer_norm(rows, C, dt):
    announce("layer norm", rows, C, dt)
    x, w, b, grad = norm_case(rows, C, DT[dt])
    y, mean, rstd = seq.layer_norm_fwd(x, w, b, 1e-5, stats=True)
    got = (y, *seq.layer_norm_bwd(grad, x, w, mean, rstd))
    alone, none, none2 = seq.layer_norm_fwd(x, w, b, 1e-5)
    assert torch.equal(alone, y) and none is None and none2 is None
    want, size, _ = orc.norm(x, w, b, 1e-5, grad)
    for name, g, r, s in zip(("y", "grad_x", "grad_weight", "grad_bias"), got, want, size):
        orc.check(g, r, s, DT[dt], name)


@pytest.mark.parametrize("dt", DT)
def test_layer_norm_values(dt):
    """Constant rows (variance zero), rows far from zero, one infinite row beside finite ones."""
    announce("layer norm values", dt)
    dtype = DT[dt]
    x, w, b, grad = norm_case(6, 96, dtype)
    x[0] = 3.0
    x[1] = 0.0
    x[3, 5] = float("inf")
    y, mean, rstd = seq.layer_norm_fwd(x, w, b, stats=True)
    gx = seq.layer_norm_bwd(grad, x, w, mean, rstd)[0]
    assert torch.equal(y[0], b) and torch.equal(y[1], b)
    assert bool(y[3].isnan().any())
    keep = [0, 1, 2, 4, 5]
    assert bool(y[keep].isfinite().all()) and bool(gx[keep].isfinite().all())
    want, size, _ = orc.norm(x[keep], w, b, 1e-5, grad[keep])
    orc.check(gx[keep], want[1], size[1], dtype, "grad_x")


@pytest.mark.parametrize("dt", DT)
def test_layer_norm_strides_and_axes(dt):
    announce("layer norm strides", dt)
    dtype = DT[dt]
    x, w, b, grad = norm_case(10, 77, dtype)
    wide = torch.full((10, 100), float("nan"), device="cuda", dtype=dtype)
    wide[:, 3:80] = x
    gwide = torch.full((10, 91), float("nan"), device="cuda", dtype=dtype)
    gwide[:, 1:78] = grad
    y, m, r = seq.layer_norm_fwd(x, w, b, stats=True)
    y2, m2, r2 = seq.layer_norm_fwd(wide[:, 3:80], w, b, stats=True)
    assert torch.equal(y, y2) and torch.equal(m, m2) and torch.equal(r, r2)
    for p, q in zip(seq.layer_norm_bwd(grad, x, w, m, r), seq.layer_norm_bwd(gwide[:, 1:78], wide[:, 3:80], w, m, r)):
        assert torch.equal(p, q)
    y3, m3, _ = seq.layer_norm_fwd(x.view(2, 5, 77), w, b, stats=True)
    assert torch.equal(y3.view(10, 77), y) and m3.shape == (2, 5)
    # every row the same row
    y4 = seq.layer_norm_fwd(x[:1].expand(4, 77), w, b)[0]
    assert all(torch.equal(y4[k], y[0]) for k in range(4))


# --------------------------------------------------------------------------- convolution
# (batch, L, D, W): one token, shorter than the taps, longer than a walk, odd channel counts
CONV = [(1, 1, 1, 4), (2, 2, 5, 4), (1, 3, 16, 3), (3, 67, 40, 4), (2, 40, 33, 2), (2, 19, 64, 1), (1, 50, 23, 7),
        (2, 300, 136, 4), (1, 33, 1, 8), (5, 16, 259, 3)]


def conv_case(batch, L, D, W, dtype, seed=2):
    g = gen_of(seed)
    return (randn(g, batch, L, D, dtype=dtype), randn(g, D, W, dtype=dtype, scale=0.5), randn(g, D, dtype=dtype, scale=0.2),
            randn(g, batch, W - 1, D, dtype=dtype), randn(g, batch, L, D, dtype=dtype),
            randn(g, batch, W - 1, D, dtype=dtype))


def ragged(batch, L, seed=3):
    n = torch.randint(0, L + 1, (batch,), generator=gen_of(seed), dtype=torch.int32)
    n[0] = L
    if batch > 1:
        n[1] = 0
    if batch > 2:
        n[2] = 1
    return n.cuda()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("state", [False, True], ids=["fresh", "cached"])
@pytest.mark.parametrize("batch,L,D,W", CONV)
def test_causal_conv(batch, L, D, W, state, dt):
    announce("conv", batch, L, D, W, state, dt)
    x, w, b, init, grad, gs = conv_case(batch, L, D, W, DT[dt])
    lengths = ragged(batch, L) if state else None
    if not state or W == 1:
        init = gs = None
    if lengths is not None:  # what lies past a length must not matter
        off = torch.arange(L, device="cuda")[None] >= lengths[:, None]
        x[off] = float("nan")
        grad[off] = float("inf")
    y, last = seq.causal_conv_fwd(x, w, b, init, lengths, return_state=True)
    gx, gw, gb, gi = seq.causal_conv_bwd(grad, x, w, b, init, lengths, gs)
    xz, gz = (x, grad) if lengths is None else (x.masked_fill(off[..., None], 0), grad.masked_fill(off[..., None], 0))
    want, size = orc.conv(xz, w, b, init, lengths, gz, gs)
    got = {"y": y, "grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    if W > 1:
        assert torch.equal(last.double().cpu(), want["state"])
    if init is not None:
        got["grad_initial"] = gi
    else:
        assert gi is None
    for name, g in got.items():
        orc.check(g, want[name], size[name], DT[dt], name)
    y2, none = seq.causal_conv_fwd(x, w, b, init, lengths)
    assert none is None and torch.equal(y2, y)


@pytest.mark.parametrize("dt", DT)
def test_causal_conv_long_columns(dt):
    """The weight gradient's sums over many workgroups."""
    announce("conv long columns", dt)
    x, w, b, _, grad, _ = conv_case(2, 6000, 24, 4, DT[dt])
    y, _ = seq.causal_conv_fwd(x, w, b)
    gx, gw, gb, _ = seq.causal_conv_bwd(grad, x, w, b)
    want, size = orc.conv(x, w, b, grad=grad)
    for name, g in (("y", y), ("grad_x", gx), ("grad_weight", gw), ("grad_bias", gb)):
        orc.check(g, want[name], size[name], DT[dt], name)


@pytest.mark.parametrize("dt", DT)
def test_causal_conv_views(dt):
    """A slice of a projection, a broadcast batch, and a walk in two halves through the state."""
    announce("conv views", dt)
    dtype = DT[dt]
    x, w, b, init, grad, _ = conv_case(2, 41, 30, 4, dtype)
    y, last = seq.causal_conv_fwd(x, w, b, init, return_state=True)
    wide = torch.full((2, 41, 53), float("nan"), device="cuda", dtype=dtype)
    wide[..., 11:41] = x
    assert torch.equal(seq.causal_conv_fwd(wide[..., 11:41], w, b, init)[0], y)
    gwide = torch.full((41, 2, 37), float("nan"), device="cuda", dtype=dtype)
    gwide[..., 2:32] = grad.transpose(0, 1)
    for p, q in zip(seq.causal_conv_bwd(grad, x, w, b, init),
                    seq.causal_conv_bwd(gwide[..., 2:32].transpose(0, 1), wide[..., 11:41], w, b, init)):
        assert torch.equal(p, q)
    same = seq.causal_conv_fwd(x[:1].expand(3, 41, 30), w, b)[0]
    assert all(torch.equal(same[k], same[0]) for k in range(3))
    y1, mid = seq.causal_conv_fwd(x[:, :17], w, b, init, return_state=True)
    y2, end = seq.causal_conv_fwd(x[:, 17:], w, b, mid, return_state=True)
    assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(end, last)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("batch,D,W", [(1, 1, 4), (5, 40, 4), (3, 33, 2), (4, 259, 3), (2, 17, 8), (2, 16, 1)])
def test_causal_conv_step(batch, D, W, dt):
    announce("conv step", batch, D, W, dt)
    g = gen_of(5)
    dtype, S = DT[dt], batch + 2
    x, w, b, _, _, _ = conv_case(batch, 1, D, W, dtype)
    x = x[:, 0]
    state = randn(g, S, W - 1, D, dtype=dtype)
    slots = torch.randperm(S, generator=g)[:batch].to(torch.int32).cuda()
    if batch > 2:
        slots[1], slots[2] = -1, S  # places without a sequence
    before = state.clone()
    y = seq.causal_conv_step(x, w, b, state, slots)
    wy, sy, ws = orc.conv_step(x, w, b, before, slots)
    orc.check(y, wy, sy, dtype, "y")
    assert torch.equal(state.double().cpu(), ws)
    # without slots, and through the whole-sequence form
    st = before.clone()
    y2 = seq.causal_conv_step(x, w, b, st)
    y3, st3 = seq.causal_conv_fwd(x[:, None].contiguous(), w, b, before[:batch].contiguous() if W > 1 else None,
                                  return_state=True)
    orc.check(y2, y3[:, 0].double().cpu(), orc.conv_step(x, w, b, before, None)[1], dtype, "y")
    if W > 1:
        assert torch.equal(st[:batch], st3) and torch.equal(st[batch:], before[batch:])


# ------------------------------------------------------------------- gradients, refusals
def directional(f, args, grads, seed):
    """Central differences of sum(f * cotangent) in 64 bits along random directions against the
    kernels' gradients; returns (difference, gradient)."""
    g = gen_of(seed)
    d = [torch.randn(a.shape, generator=g, dtype=torch.float64) for a in args]
    a64 = [a.detach().double().cpu() for a in args]
    h = 1e-6
    up, down = (f(*[a + s * h * v for a, v in zip(a64, d)]) for s in (1, -1))
    return float((up - down) / (2 * h)), float(sum((v * q.double().cpu()).sum() for v, q in zip(d, grads)))


def test_gradients_against_differences():
    announce("differences")
    x, w, b, grad = norm_case(6, 50, torch.float32)
    y, m, r = seq.layer_norm_fwd(x, w, b, stats=True)
    g64 = grad.double().cpu()

    def norm(x, w, b):
        mu = x.mean(-1, keepdim=True)
        return (((x - mu) / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + 1e-5) * w + b) * g64).sum()

    diff, got = directional(norm, (x, w, b), seq.layer_norm_bwd(grad, x, w, m, r), 7)
    # gradients to 512 float32 roundings, differences to h^2 and 1e-16 / h
    assert abs(diff - got) <= 1e-4 * max(1, abs(diff))
    x, w, b, init, grad, gs = conv_case(2, 30, 12, 4, torch.float32)
    lengths = torch.tensor([30, 2], dtype=torch.int32, device="cuda")
    gx, gw, gb, gi = seq.causal_conv_bwd(grad, x, w, b, init, lengths, gs)

    def conv(x, w, b, i):
        y, last = orc._conv(x, w, b, i, lengths.cpu())
        return (y * grad.double().cpu()).sum() + (last * gs.double().cpu()).sum()

    diff, got = directional(conv, (x, w, b, init), (gx, gw, gb, gi), 8)
    assert abs(diff - got) <= 1e-4 * max(1, abs(diff))


def test_autograd():
    announce("autograd")
    x, w, b, grad = norm_case(12, 40, torch.float32)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    got = torch.autograd.grad((seq.layer_norm(*leaves) * grad).sum(), leaves)
    y, m, r = seq.layer_norm_fwd(x, w, b, stats=True)
    assert all(torch.equal(p, q) for p, q in zip(got, seq.layer_norm_bwd(grad, x, w, m, r)))
    x, w, b, init, grad, gs = conv_case(2, 25, 18, 4, torch.float32)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, init)]
    y, last = seq.causal_conv(*leaves)
    got = torch.autograd.grad((y * grad).sum() + (last * gs).sum(), leaves)
    assert all(torch.equal(p, q) for p, q in zip(got, seq.causal_conv_bwd(grad, x, w, b, init, None, gs)))
    got = torch.autograd.grad(seq.causal_conv(*leaves)[1].sum(), leaves)  # the state alone
    assert torch.equal(got[3], torch.zeros_like(init)) and float(got[0][:, -3:].sum()) == 2 * 3 * 18
    # a broadcast input: its gradient is the sum over where it went
    one = x[:1].clone().requires_grad_()
    g1, = torch.autograd.grad((seq.causal_conv(one.expand(2, 25, 18), w, b)[0] * grad).sum(), one)
    gx = seq.causal_conv_bwd(grad, x[:1].expand(2, 25, 18).contiguous(), w, b)[0]
    assert torch.equal(g1, gx.sum(0, keepdim=True))


def test_refusals():
    announce("refusals")
    x, w, b, _ = norm_case(4, 16, torch.float32)
    for call in (lambda: seq.layer_norm_fwd(x, w[:8], b), lambda: seq.layer_norm_fwd(x.half(), w.half(), b.half()),
                 lambda: seq.layer_norm_fwd(x, w.bfloat16(), b), lambda: seq.layer_norm_fwd(x.t(), w, b),
                 lambda: seq.layer_norm_fwd(x[:0], w, b), lambda: seq.layer_norm_fwd(x, w.cpu(), b),
                 lambda: seq.layer_norm_bwd(x[:3], x, w, x[:, 0], x[:, 0])):
        with pytest.raises(ValueError):
            call()
    x, w, b, init, grad, _ = conv_case(2, 6, 8, 4, torch.float32)
    n = torch.tensor([6, 6], device="cuda")
    for call in (lambda: seq.causal_conv_fwd(x[0], w, b), lambda: seq.causal_conv_fwd(x, w.t(), b),
                 lambda: seq.causal_conv_fwd(x, w, b, init[:, :2]), lambda: seq.causal_conv_fwd(x, w, b, lengths=n),
                 lambda: seq.causal_conv_fwd(x.transpose(1, 2), w, b), lambda: seq.causal_conv_fwd(x, w, b[:4]),
                 lambda: seq.causal_conv_fwd(x, w[:, :1].contiguous(), b, init[:, :0].contiguous()),
                 lambda: seq.causal_conv_bwd(grad[:, :3], x, w, b),
                 lambda: seq.causal_conv_step(x[:, 0], w, b, init.bfloat16()),
                 lambda: seq.causal_conv_step(x[:, 0], w, b, init, n)):
        with pytest.raises(ValueError):
            call()
    from dynamic_dilated_depthwise_amd import DDPMError
    with pytest.raises(DDPMError, match="UNSUPPORTED"):
        seq.causal_conv_fwd(x, torch.zeros(8, 9, device="cuda"), b)
    with pytest.raises(DDPMError, match="INVALID"):  # the token lies in the state that is updated
        seq.causal_conv_step(init[:, 0], w, b, init)


def test_streams_and_graph():
    """Every entry point on a stream of its own, and captured and replayed among eager work."""
    announce("streams and graph")
    xn, wn, bn, gn = norm_case(300, 200, torch.bfloat16)
    x, w, b, init, grad, gs = conv_case(2, 70, 48, 4, torch.bfloat16)
    state0 = init.clone()
    state = state0.clone()

    def step():
        y, m, r = seq.layer_norm_fwd(xn, wn, bn, stats=True)
        yc, last = seq.causal_conv_fwd(x, w, b, init, return_state=True)
        state.copy_(state0)
        ys = seq.causal_conv_step(x[:, 0], w, b, state)
        return (y, *seq.layer_norm_bwd(gn, xn, wn, m, r), yc, last, *seq.causal_conv_bwd(grad, x, w, b, init, None, gs), ys,
                state)

    eager = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, _, _ = seq.layer_norm_fwd(xn, wn, bn, stream=side)
    side.synchronize()
    assert torch.equal(y, eager[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    junk = torch.randn(256, 256, device="cuda")
    for _ in range(3):
        for t in outs[:-1]:
            t.fill_(float("nan"))
        junk = torch.tanh(junk @ junk / 256)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, eager))


def test_far_offsets():
    """Rows that start past 2^31 elements of one tensor."""
    announce("far offsets")
    far = (1 << 31) + 64
    flat = torch.empty(far + 5000, device="cuda", dtype=torch.bfloat16)
    x, w, b, init, grad, _ = conv_case(2, 9, 40, 4, torch.bfloat16)
    view = flat.as_strided((2, 9, 40), (far, 40, 1))
    view.copy_(x)
    assert torch.equal(seq.causal_conv_fwd(view, w, b, init)[0], seq.causal_conv_fwd(x, w, b, init)[0])
    for p, q in zip(seq.causal_conv_bwd(view, view, w, b, init), seq.causal_conv_bwd(x, x, w, b, init)):
        assert torch.equal(p, q)
    rows = flat.as_strided((2, 40), (far, 1))
    wn, bn = w[:, 0].contiguous(), b
    assert torch.equal(seq.layer_norm_fwd(rows, wn, bn)[0], seq.layer_norm_fwd(x[:, 0].contiguous(), wn, bn)[0])
