"""The selective scan against its recurrence in 64 bits: whole sequences forward and backward,
single tokens, states between calls; refusals, streams, graphs, far offsets.

Tolerances (seq_oracle.check): 512 float32 roundings of the sum's size (the longest sums have
a few hundred terms), one rounding of the output to its type, and, for the bfloat16 outputs
that are sums over decayed scores or states rounded to bfloat16 as matrix operands (y, grad_x,
grad_B, grad_C), one such rounding of the size.
"""
import pytest
import torch

import seq_oracle as orc
from dynamic_dilated_depthwise_amd import sequence as seq
from test_gpu_seq_norm_conv import DT, announce, directional, gen_of, ragged, randn

pytestmark = pytest.mark.gpu

NAMES = ("grad_x", "grad_dt", "grad_A", "grad_B", "grad_C", "grad_D", "grad_dt_bias", "grad_initial")
ROUNDED = ("y", "grad_x", "grad_B", "grad_C")


def case(batch, L, H, P, G, N, dtype, seed=11, fast=False):
    g = gen_of(seed)
    A = -(torch.rand(H, generator=g) * (60 if fast else 15) + 1).cuda()
    bias = (torch.rand(H, generator=g) * 4 - (1 if fast else 6)).cuda()
    return (randn(g, batch, L, H, P, dtype=dtype), randn(g, batch, L, H, dtype=dtype, scale=0.5), A,
            randn(g, batch, L, G, N, dtype=dtype), randn(g, batch, L, G, N, dtype=dtype), randn(g, H, shift=1.0), bias)


def compare(got, want, size, dtype):
    for name, g in got.items():
        t = torch.float32 if name in ("state", "grad_A", "grad_D", "grad_dt_bias", "grad_initial") else dtype
        orc.check(g, want[name], size[name], t, name, operand=dtype if name in ROUNDED and dtype != torch.float32 else None)


# (batch, L, H, P, G, N): one token, one chunk less or more a token, heads of one group over
# several workgroups, P beyond a slab, odd P and N, more chunks than the pass has parts
SIZES = [(1, 1, 1, 1, 1, 1), (2, 7, 2, 16, 1, 16), (1, 64, 2, 64, 2, 64), (1, 65, 2, 40, 1, 50), (2, 129, 4, 48, 2, 24),
         (1, 200, 3, 33, 1, 37), (1, 300, 2, 128, 1, 128), (3, 257, 2, 96, 1, 100), (1, 130, 6, 70, 3, 128),
         (1, 2300, 1, 20, 1, 12), (1, 150, 16, 8, 1, 16)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("state", [False, True], ids=["fresh", "cached"])
@pytest.mark.parametrize("batch,L,H,P,G,N", SIZES)
def test_scan(batch, L, H, P, G, N, state, dt):
    announce("scan", batch, L, H, P, G, N, state, dt)
    dtype = DT[dt]
    args = list(case(batch, L, H, P, G, N, dtype))
    g = gen_of(12)
    grad = randn(g, batch, L, H, P, dtype=dtype)
    init = randn(g, batch, H, P, N) if state else None
    gs = randn(g, batch, H, P, N) if state else None
    lengths = ragged(batch, L) if state else None
    clean = list(args) + [grad]
    if lengths is not None:  # what lies past a length must not matter
        off = torch.arange(L, device="cuda")[None] >= lengths[:, None]
        for k in (0, 1, 3, 4):
            args[k][off] = float("nan")
            clean[k] = args[k].masked_fill(off[(...,) + (None,) * (args[k].dim() - 2)], 0)
        grad[off] = float("inf")
        clean[7] = grad.masked_fill(off[..., None, None], 0)
    y, last, saved = seq.selective_scan_fwd(*args, init, lengths, return_state=True, save=True)
    got = dict(zip(NAMES, seq.selective_scan_bwd(grad, *args, saved, init, lengths, gs)))
    if init is None:
        assert got.pop("grad_initial") is None
    want, size = orc.scan(*clean[:7], init, lengths, clean[7], gs)
    compare({"y": y, "state": last, **got}, want, size, dtype)
    y2, none, none2 = seq.selective_scan_fwd(*args, init, lengths)
    assert none is None and none2 is None and torch.equal(y, y2)


@pytest.mark.parametrize("dt", DT)
def test_scan_fast_decay(dt):
    """Steps that forget everything at once beside steps of size zero, and dt far out."""
    announce("scan fast decay", dt)
    dtype = DT[dt]
    args = list(case(2, 200, 3, 24, 1, 20, dtype, fast=True))
    args[1][:, 50:60] = -200.0  # dt underflows to zero
    args[1][:, 100:103] = 1000.0  # a decay of exp(-1000 A)
    grad = randn(gen_of(3), 2, 200, 3, 24, dtype=dtype)
    y, last, saved = seq.selective_scan_fwd(*args, return_state=True, save=True)
    got = dict(zip(NAMES, seq.selective_scan_bwd(grad, *args, saved)))
    got.pop("grad_initial")
    assert all(bool(t.isfinite().all()) for t in (y, last, *got.values()))
    want, size = orc.scan(*args, grad=grad)
    compare({"y": y, "state": last, **got}, want, size, dtype)


@pytest.mark.parametrize("dt", DT)
def test_scan_views_and_halves(dt):
    """x, dt, B and C as slices of one projection; a sequence in two halves through its state."""
    announce("scan views", dt)
    dtype = DT[dt]
    B_, L, H, P, G, N = 2, 210, 4, 24, 2, 18
    x, draw, A, Bm, Cm, D, bias = case(B_, L, H, P, G, N, dtype)
    wide = torch.full((B_, L, H * P + 2 * G * N + H + 5), float("nan"), device="cuda", dtype=dtype)
    parts, at = [], 3
    for t in (x, Bm, Cm, draw):
        w = t[0, 0].numel()
        wide[..., at:at + w] = t.flatten(2)
        parts.append(wide[..., at:at + w].unflatten(2, t.shape[2:]))
        at += w
    grad = randn(gen_of(4), B_, L, H, P, dtype=dtype)
    gw = grad.transpose(0, 1).contiguous().transpose(0, 1)
    y, last, saved = seq.selective_scan_fwd(x, draw, A, Bm, Cm, D, bias, return_state=True, save=True)
    xs, bs, cs, ds = parts
    y2, last2, saved2 = seq.selective_scan_fwd(xs, ds, A, bs, cs, D, bias, return_state=True, save=True)
    assert torch.equal(y, y2) and torch.equal(last, last2)
    one = seq.selective_scan_bwd(grad, x, draw, A, Bm, Cm, D, bias, saved)
    two = seq.selective_scan_bwd(gw, xs, ds, A, bs, cs, D, bias, saved2)
    assert all(torch.equal(p, q) for p, q in zip(one[:7], two[:7]))
    cut = 77
    half = [t[:, :cut] for t in (x, draw, Bm, Cm)], [t[:, cut:] for t in (x, draw, Bm, Cm)]
    ya, mid, _ = seq.selective_scan_fwd(half[0][0], half[0][1], A, half[0][2], half[0][3], D, bias, return_state=True)
    yb, end, _ = seq.selective_scan_fwd(half[1][0], half[1][1], A, half[1][2], half[1][3], D, bias, mid, return_state=True)
    want, size = orc.scan(x, draw, A, Bm, Cm, D, bias)
    compare({"y": torch.cat([ya, yb], 1), "state": end}, want, size, dtype)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("batch,H,P,G,N", [(1, 1, 1, 1, 1), (1, 2, 64, 1, 64), (5, 4, 40, 2, 50), (3, 2, 33, 1, 37),
                                           (2, 3, 96, 1, 100), (40, 8, 64, 1, 128), (2, 2, 5, 2, 300), (2, 1, 300, 1, 24)])
def test_scan_step(batch, H, P, G, N, dt):
    announce("scan step", batch, H, P, G, N, dt)
    dtype, S = DT[dt], batch + 2
    x, draw, A, Bm, Cm, D, bias = case(batch, 1, H, P, G, N, dtype)
    x, draw, Bm, Cm = x[:, 0], draw[:, 0], Bm[:, 0], Cm[:, 0]
    g = gen_of(13)
    state = randn(g, S, H, P, N)
    slots = torch.randperm(S, generator=g)[:batch].to(torch.int32).cuda()
    if batch > 2:
        slots[1], slots[2] = -1, S  # places without a sequence
    before = state.clone()
    y = seq.selective_scan_step(x, draw, A, Bm, Cm, D, bias, state, slots)
    wy, sy, ws, ss = orc.scan_step(x, draw, A, Bm, Cm, D, bias, before, slots)
    orc.check(y, wy, sy, dtype, "y")
    orc.check(state, ws, ss, torch.float32, "state")
    untouched = [k for k in range(S) if k not in slots.tolist()]
    assert torch.equal(state[untouched], before[untouched])
    st = before.clone()
    y2 = seq.selective_scan_step(x, draw, A, Bm, Cm, D, bias, st)
    wy, sy, ws, ss = orc.scan_step(x, draw, A, Bm, Cm, D, bias, before, None)
    orc.check(y2, wy, sy, dtype, "y")
    orc.check(st, ws, ss, torch.float32, "state")


def test_scan_steps_equal_a_prompt():
    announce("scan steps")
    args = case(2, 30, 2, 32, 1, 16, torch.float32)
    x, draw, A, Bm, Cm, D, bias = args
    y, last, _ = seq.selective_scan_fwd(*args, return_state=True)
    state = torch.zeros(2, 2, 32, 16, device="cuda")
    steps = torch.stack([seq.selective_scan_step(x[:, t], draw[:, t], A, Bm[:, t], Cm[:, t], D, bias, state)
                         for t in range(30)], 1)
    want, size = orc.scan(*args)
    compare({"y": steps, "state": state}, want, size, torch.float32)
    compare({"y": y, "state": last}, want, size, torch.float32)


def test_gradients_against_differences():
    announce("scan differences")
    batch, L, H, P, G, N = 2, 70, 2, 6, 1, 5
    args = case(batch, L, H, P, G, N, torch.float32)
    g = gen_of(21)
    grad, init, gs = randn(g, batch, L, H, P), randn(g, batch, H, P, N), randn(g, batch, H, P, N)
    lengths = torch.tensor([70, 33], dtype=torch.int32, device="cuda")
    saved = seq.selective_scan_fwd(*args, init, lengths, save=True)[2]
    grads = seq.selective_scan_bwd(grad, *args, saved, init, lengths, gs)

    def f(x, draw, A, Bm, Cm, D, bias, init):
        on = torch.arange(L)[None] < lengths.cpu()[:, None]
        raw = draw + bias
        step = torch.logaddexp(raw, torch.zeros_like(raw))
        y, h = orc._scan(x, step, step, A, Bm, Cm, D, init, on)
        return (y * grad.double().cpu()).sum() + (h * gs.double().cpu()).sum()

    for only in range(8):  # one argument at a time
        a = [t.double().cpu() for t in (*args, init)]

        def one(v):
            return f(*a[:only], v, *a[only + 1:])

        diff, got = directional(one, ((*args, init)[only],), (grads[only],), 30 + only)
        # gradients to 512 float32 roundings of sums of a few thousand terms of size one
        assert abs(diff - got) <= 2e-3 * max(1, abs(diff)), (NAMES[only], diff, got)


def test_autograd():
    announce("scan autograd")
    args = case(2, 90, 4, 16, 2, 12, torch.float32)
    g = gen_of(5)
    init, grad, gs = randn(g, 2, 4, 16, 12), randn(g, 2, 90, 4, 16), randn(g, 2, 4, 16, 12)
    leaves = [t.clone().requires_grad_() for t in (*args, init)]
    y, last = seq.selective_scan(*leaves)
    got = torch.autograd.grad((y * grad).sum() + (last * gs).sum(), leaves)
    saved = seq.selective_scan_fwd(*args, init, save=True)[2]
    want = seq.selective_scan_bwd(grad, *args, saved, init, None, gs)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    y, last = seq.selective_scan(*leaves[:7])  # the state alone
    gx, = torch.autograd.grad((last * gs).sum(), leaves[0])
    w, s = orc.scan(*args, grad=torch.zeros_like(grad), grad_state=gs)
    orc.check(gx, w["grad_x"], s["grad_x"], torch.float32, "grad_x")
    # B shared by both groups: its gradient is the sum of theirs
    one = args[3][:, :, :1].clone().requires_grad_()
    full = list(args)
    full[3] = one.expand(2, 90, 2, 12)
    g1, = torch.autograd.grad((seq.selective_scan(*full)[0] * grad).sum(), one)
    full[3] = full[3].detach().contiguous()
    saved = seq.selective_scan_fwd(*full, save=True)[2]
    assert torch.equal(g1, seq.selective_scan_bwd(grad, *full, saved)[3].sum(2, keepdim=True))


def test_refusals():
    announce("scan refusals")
    x, draw, A, Bm, Cm, D, bias = a = case(2, 5, 4, 8, 2, 6, torch.float32)
    state = torch.zeros(2, 4, 8, 6, device="cuda")

    def swap(k, t):
        return a[:k] + (t,) + a[k + 1:]

    bad = [swap(0, x[:, :4]), swap(0, x.transpose(2, 3)), swap(0, x.half()), swap(1, draw[..., :3]), swap(2, A.double()),
           swap(2, A[:2]), swap(3, Bm[:, :, :1]), swap(3, Bm.bfloat16()), swap(4, Cm.transpose(0, 1)), swap(5, D.cpu()),
           swap(6, bias[None]), swap(0, x[:, :0]), swap(0, x[..., :3, :])]
    for args in bad:
        with pytest.raises(ValueError):
            seq.selective_scan_fwd(*args)
    for kw in (dict(initial_state=state.bfloat16()), dict(initial_state=state[:1]),
               dict(lengths=torch.tensor([5, 5], device="cuda")), dict(lengths=torch.tensor([5, 5], dtype=torch.int32))):
        with pytest.raises(ValueError):
            seq.selective_scan_fwd(*a, **kw)
    saved = seq.selective_scan_fwd(*a, save=True)[2]
    with pytest.raises(ValueError):
        seq.selective_scan_bwd(x, *a, saved[:-64])
    with pytest.raises(ValueError):
        seq.selective_scan_bwd(x.bfloat16(), *a, saved)
    with pytest.raises(TypeError):
        seq.selective_scan_bwd(x, *a, None)
    from dynamic_dilated_depthwise_amd import DDPMError
    with pytest.raises(DDPMError, match="UNSUPPORTED"):
        seq.selective_scan_fwd(*swap(4, torch.zeros(2, 5, 2, 129, device="cuda"))[:3],
                               *(torch.zeros(2, 5, 2, 129, device="cuda"),) * 2, D, bias)
    token = (x[:, 0], draw[:, 0], A, Bm[:, 0], Cm[:, 0], D, bias)
    for st in (state.bfloat16(), state[:, :2], state[0]):
        with pytest.raises(ValueError):
            seq.selective_scan_step(*token, st)
    with pytest.raises(ValueError):
        seq.selective_scan_step(*token, state, torch.tensor([0], dtype=torch.int32, device="cuda"))


def test_streams_and_graph():
    announce("scan streams and graph")
    args = case(2, 300, 4, 32, 1, 40, torch.bfloat16)
    g = gen_of(6)
    grad, init = randn(g, 2, 300, 4, 32, dtype=torch.bfloat16), randn(g, 2, 4, 32, 40)
    state = init.clone()
    x, draw, A, Bm, Cm, D, bias = args

    def step():
        y, last, saved = seq.selective_scan_fwd(*args, init, return_state=True, save=True)
        state.copy_(init)
        ys = seq.selective_scan_step(x[:, 0], draw[:, 0], A, Bm[:, 0], Cm[:, 0], D, bias, state)
        return (y, last, *seq.selective_scan_bwd(grad, *args, saved, init), ys, state)

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, last, saved = seq.selective_scan_fwd(*args, init, return_state=True, save=True, stream=side)
    back = seq.selective_scan_bwd(grad, *args, saved, init, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((y, last, *back), eager))
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


def test_far_slots():
    """A cache of states past 2^31 elements."""
    announce("scan far slots")
    H, P, N = 8, 64, 128
    S = (1 << 31) // (H * P * N) + 3
    state = torch.empty(S, H, P, N, device="cuda")
    x, draw, A, Bm, Cm, D, bias = case(2, 1, H, P, 1, N, torch.float32)
    near = randn(gen_of(9), 2, H, P, N)
    state[S - 1], state[0] = near[0], near[1]
    slots = torch.tensor([S - 1, 0], dtype=torch.int32, device="cuda")
    token = (x[:, 0], draw[:, 0], A, Bm[:, 0], Cm[:, 0], D, bias)
    y = seq.selective_scan_step(*token, state, slots)
    assert torch.equal(y, seq.selective_scan_step(*token, near))
    assert torch.equal(state[S - 1], near[0]) and torch.equal(state[0], near[1])
