"""The feed-forward operators against their definitions in 64 bits, forward and backward, at the sizes
where their forms change; views, refusals, streams, graphs, gradients against differences.

Tolerances (ff_oracle.check): one rounding of the output, one of the gradient that an activation's or a
gate's input takes to the type, and as many float32 roundings as the sums have terms, twice.
"""
import pytest
import torch

import ff_oracle as orc
from dynamic_dilated_depthwise_amd import feedforward as ff

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def announce(*a):
    print("[gpu case]", *a, flush=True)


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


def case(rows, C, N, dtype, gated=False, seed=1):
    """x, weight, bias, residual (gated: None), grad"""
    g = gen_of(seed)
    width = 2 * N if gated else N
    return (randn(g, rows, C, dtype=dtype), randn(g, width, C, dtype=dtype, scale=C ** -0.5),
            randn(g, width, dtype=dtype, scale=0.3), None if gated else randn(g, rows, N, dtype=dtype),
            randn(g, rows, N, dtype=dtype))


def forward(x, w, b, r, act, gated, **kw):
    return ff.gated_linear_fwd(x, w, b, act, **kw) if gated else ff.linear_fwd(x, w, b, r, act, **kw)


def backward(grad, x, w, saved, act, gated, **kw):
    return (ff.gated_linear_bwd if gated else ff.linear_bwd)(grad, x, w, saved, act, **kw)


def compare(x, w, b, r, grad, act, gated):
    dtype, rows, C, width = x.dtype, x.numel() // x.shape[-1], x.shape[-1], w.shape[0]
    y, saved = forward(x, w, b, r, act, gated, save=True)
    alone, none = forward(x, w, b, r, act, gated)
    assert none is None and torch.equal(alone, y)
    assert (saved is None) == (act == "none" and not gated)
    gx, gw, gb = backward(grad, x, w, saved, act, gated)
    want = orc.run(x, w, b, r, act, grad, gated)
    orc.check(y, want["y"], dtype, "y", 2 * C + 64)
    orc.check(gx, want["grad_x"], dtype, "grad_x", 2 * (C + width) + 64)
    orc.check(gw, want["grad_weight"], dtype, "grad_weight", 2 * (C + rows) + 64)
    orc.check(gb, want["grad_bias"], dtype, "grad_bias", 2 * (C + rows) + 64)


# (rows, C, N): one element; sizes below, at and above a step of the contraction, a fragment and a
# tile; whole chunks (straight to LDS) and others; a few tokens; long contractions with few tiles
# (split); many tiles
SIZES = [(1, 1, 1), (2, 3, 5), (1, 64, 16), (1, 129, 70), (3, 8, 8), (7, 72, 24), (16, 64, 64), (17, 65, 33), (33, 128, 96),
         (48, 200, 136), (65, 56, 130), (100, 257, 31), (130, 136, 264), (128, 128, 128), (129, 127, 129), (300, 64, 128),
         (5, 2048, 40), (64, 1024, 72), (2100, 40, 48), (1500, 33, 17)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("rows,C,N", SIZES)
def test_sizes(rows, C, N, gated, dt):
    announce("ff sizes", rows, C, N, gated, dt)
    compare(*case(rows, C, N, DT[dt], gated), "silu" if gated else "none", gated)


# A decoding batch's tokens, at each end of the forms' ranges of rows; contractions of a part of a step, of fewer
# steps than waves, and of many; results that end inside sixteen columns.
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("rows", [1, 8, 16, 17, 32, 33, 48, 49, 64])
def test_tokens(rows, gated, dt):
    announce("ff tokens", rows, gated, dt)
    for C, N in ((8, 24), (104, 40), (1024, 72), (2056, 130), (8200, 16), (8, 8200), (5633, 43), (1021, 2050)):
        x, w, b, r, _ = case(rows, C, N, DT[dt], gated)
        for act in ("none", "silu"):
            y = forward(x, w, b, r, act, gated)[0]
            orc.check(y, orc.run(x, w, b, r, act, gated=gated)["y"], DT[dt], f"y of {C} to {N}", 2 * C + 64)


# Many tiles, so that bfloat16 takes the large ones, for each product of the two passes: y, grad_x, grad_weight.
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("rows,C,N", [(3400, 88, 3304), (3333, 2944, 104), (104, 3368, 3400)])
def test_large_tiles(rows, C, N, gated):
    announce("ff large tiles", rows, C, N, gated)
    compare(*case(rows, C, N, torch.bfloat16, gated), "gelu", gated)


# Few columns of x and many of z: the backward makes z again, from whole chunks and from others.
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("rows,C,N", [(9001, 24, 1352), (8200, 37, 1501), (61, 40, 200040)])
def test_made_again(rows, C, N, gated, dt):
    announce("ff made again", rows, C, N, gated, dt)
    args = case(rows, C, N, DT[dt], gated)
    saved = forward(*args[:4], "silu", gated, save=True)[1]
    assert saved.numel() == args[1].shape[0] and torch.equal(saved, args[2].float())
    compare(*args, "silu", gated)
    assert not forward(args[0], args[1], None, None, "silu", gated, save=True)[1].any()


# Few channels, whose backward is one kernel: rows below, at and above a tile and a round of the chip.
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("rows,C,N", [(1, 1, 1), (63, 64, 128), (64, 8, 16), (65, 63, 127), (130, 33, 20), (1000, 17, 90), (33100, 64, 128),
                                      (40001, 50, 77)])
def test_few_channels(rows, C, N, gated, dt):
    announce("ff few channels", rows, C, N, gated, dt)
    args = case(rows, C, N if gated else 2 * N, DT[dt], gated)
    compare(*args, "gelu", gated)
    x, w, b, r, grad = args
    saved = forward(x, w, b, r, "gelu", gated, save=True)[1]
    gx, gw, gb = backward(grad, x, w, saved, "gelu", gated)
    assert torch.equal(backward(grad, x, w, saved, "gelu", gated, need_weight=False)[0], gx)
    for p, q in zip(backward(grad, x, w, saved, "gelu", gated, need_x=False)[1:], (gw, gb)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("act", ff.ACTIVATIONS)
def test_activations(act, gated, dt):
    announce("ff activations", act, gated, dt)
    x, w, b, r, grad = case(70, 40, 56, DT[dt], gated, seed=3)
    compare(x, w, b, r, grad, act, gated)
    compare(x, w, None, None, grad, act, gated)


@pytest.mark.parametrize("dt", DT)
def test_far_values(dt):
    """Activations far from zero: nothing overflows on the way, small results keep their size."""
    announce("ff far values", dt)
    dtype = DT[dt]
    z = torch.tensor([-1e4, -200., -100., -20., -9., -5., -1., -1e-3, -0., 0., 1e-3, 1., 9., 100., 1e4]).to(dtype)
    x, w = z[:, None].cuda(), torch.ones(1, 1, dtype=dtype).cuda()
    for act in ff.ACTIVATIONS:
        y, saved = ff.linear_fwd(x, w, activation=act, save=True)
        gx, _, _ = ff.linear_bwd(torch.ones_like(x), x, w, saved, act)
        a, da = orc.curve(x.double(), act)
        # the functions' own error: a few roundings of float32, of their argument times the logarithm's slope too
        tol = (orc.u(dtype) + 16 * orc.u(torch.float32) * (1 + x.double() ** 2))
        assert bool(((y.double() - a).abs() <= tol * a.abs() + 1e-37).all()), act
        assert bool(((gx.double() - da).abs() <= tol * da.abs() + 1e-37 + 2.0 ** -22 * da.abs().clamp(max=1)).all()), act


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_views_and_axes(gated, dt):
    """Rows of a wider tensor, more axes, one row for all; unaligned starts."""
    announce("ff views", gated, dt)
    dtype, act = DT[dt], "silu"
    x, w, b, r, grad = case(30, 72, 40, dtype, gated)
    y, saved = forward(x, w, b, r, act, gated, save=True)
    grads = backward(grad, x, w, saved, act, gated)

    def inside(t, left, right):
        wide = torch.full((t.shape[0], left + t.shape[1] + right), float("nan"), device="cuda", dtype=dtype)
        wide[:, left:left + t.shape[1]] = t
        return wide[:, left:left + t.shape[1]]

    xv, gv, rv = (inside(t, 8, 16) if t is not None else None for t in (x, grad, r))
    y2, saved2 = forward(xv, w, b, rv, act, gated, save=True)
    assert torch.equal(y2, y) and torch.equal(saved2, saved)
    for p, q in zip(backward(gv, xv, w, saved2, act, gated), grads):
        assert torch.equal(p, q)
    # starts of no whole chunk: another form, other orders of the sums
    compare(inside(x, 3, 2), w, b, inside(r, 1, 0) if r is not None else None, inside(grad, 1, 6), act, gated)
    x3, r3 = x.view(2, 3, 5, 72), r.view(2, 3, 5, 40) if r is not None else None
    y3, saved3 = forward(x3, w, b, r3, act, gated, save=True)
    assert y3.shape == (2, 3, 5, 40) and torch.equal(y3.view(30, 40), y)
    for p, q in zip(backward(grad.view(2, 3, 5, 40), x3, w, saved3, act, gated), grads):
        assert torch.equal(p.view(q.shape), q)
    y4, _ = forward(x[:1].expand(30, 72), w, b, r[:1].expand(30, 40) if r is not None else None, act, gated)
    assert all(torch.equal(y4[k], y[0]) for k in range(30))
    one = forward(x[0], w, b, r[0] if r is not None else None, act, gated)[0]
    assert one.shape == (40,)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("rows,C,N", [(9, 40, 24), (9, 77, 35), (140, 72, 24), (140, 1100, 24)])
def test_not_finite(rows, C, N, gated, dt):
    """Infinities and NaN stay in their rows; the gradients of other rows are what they are without them."""
    announce("ff not finite", rows, C, N, gated, dt)
    x, w, b, r, grad = case(rows, C, N, DT[dt], gated)
    y, saved = forward(x, w, b, r, "silu", gated, save=True)
    gx = backward(grad, x, w, saved, "silu", gated, need_weight=False)[0]
    bad, bgrad = x.clone(), grad.clone()
    bad[3, C - 1], bad[5, 0] = float("nan"), float("inf")
    bgrad[6, N - 1] = float("inf")
    y2, saved2 = forward(bad, w, b, r, "silu", gated, save=True)
    gx2, gw2, _ = backward(bgrad, bad, w, saved2, "silu", gated)
    keep = [k for k in range(rows) if k not in (3, 5, 6)]
    assert bool(y2[3].isnan().all()) and not bool(y2[5].isfinite().all())
    assert torch.equal(y2[keep], y[keep]) and torch.equal(gx2[keep], gx[keep])
    assert not bool(gx2[6].isfinite().all()) and not bool(gw2.isfinite().all())


def test_gradients_against_differences():
    announce("ff differences")
    for gated in (False, True):
        x, w, b, r, grad = case(9, 14, 11, torch.float32, gated)
        for act in ("none", "silu", "gelu"):
            saved = forward(x, w, b, r, act, gated, save=True)[1]
            grads = backward(grad, x, w, saved, act, gated)
            g = gen_of(5)
            d = [torch.randn(t.shape, generator=g, dtype=torch.float64).cuda() for t in (x, w, b)]
            h = 1e-6

            def value(s):
                args = [t.double() + s * h * v for t, v in zip((x, w, b), d)]
                return (orc.run(*args, r, act, gated=gated)["y"][0] * grad.double()).sum()

            diff = float((value(1) - value(-1)) / (2 * h))
            got = float(sum((v * q.double()).sum() for v, q in zip(d, grads)))
            # gradients to a few dozen float32 roundings, differences to h^2 and 1e-16 / h
            assert abs(diff - got) <= 1e-4 * max(1, abs(diff)), (gated, act)


@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_autograd(gated):
    announce("ff autograd", gated)
    x, w, b, r, grad = case(12, 40, 24, torch.float32, gated)
    act = "silu"
    saved = forward(x, w, b, r, act, gated, save=True)[1]
    want = list(backward(grad, x, w, saved, act, gated)) + ([] if gated else [grad])
    leaves = [t.clone().requires_grad_() for t in (x, w, b, r) if t is not None]
    call = (lambda *t: ff.gated_linear(*t, activation=act)) if gated else (lambda *t: ff.linear(*t, activation=act))
    y = call(*leaves)
    assert torch.equal(y, forward(x, w, b, r, act, gated)[0])
    got = torch.autograd.grad(y, leaves, grad)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    for k in range(len(leaves)):  # one of them alone
        some = [t.detach().requires_grad_(i == k) for i, t in enumerate(leaves)]
        g, = torch.autograd.grad(call(*some), some[k], grad)
        assert torch.equal(g, want[k]), k
    # without gradients, and gradients that are no contiguous rows
    with torch.no_grad():
        assert not call(*leaves).requires_grad
    got = torch.autograd.grad(call(*leaves).sum(), leaves)
    ones = backward(torch.ones_like(grad), x, w, saved, act, gated)
    assert all(torch.equal(p, q) for p, q in zip(got, ones))
    got = torch.autograd.grad(call(*leaves).t(), leaves, grad.t().contiguous())
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    # a broadcast row: its gradient is the sum over where it went
    one = x[:1].clone().requires_grad_()
    g1, = torch.autograd.grad(call(one.expand(12, 40), *leaves[1:]), one, grad)
    xs = x[:1].expand(12, 40)
    gx = backward(grad, xs, w, forward(xs, w, b, r, act, gated, save=True)[1], act, gated)[0]
    assert torch.equal(g1, gx.sum(0, keepdim=True))
    with pytest.raises(RuntimeError):  # once differentiable
        g, = torch.autograd.grad(call(*leaves), leaves[0], grad, create_graph=True)
        g.sum().backward()


def test_forward_mode_is_refused():
    announce("ff forward mode")
    import torch.autograd.forward_ad as fwAD
    x, w, b, r, _ = case(6, 10, 8, torch.float32)
    for mode in (torch.enable_grad, torch.no_grad):
        with mode(), fwAD.dual_level():
            for call in (lambda: ff.linear(fwAD.make_dual(x, x), w), lambda: ff.linear(x, w, b, fwAD.make_dual(r, r)),
                         lambda: ff.gated_linear(x, fwAD.make_dual(w, w))):
                with pytest.raises(RuntimeError, match="jvp|forward"):
                    call()


def test_refusals():
    announce("ff refusals")
    x, w, b, r, grad = case(6, 16, 8, torch.float32)
    w2 = torch.cat([w, w])
    for call in (lambda: ff.linear_fwd(x, w[:, :8]), lambda: ff.linear_fwd(x, w.t()), lambda: ff.linear_fwd(x, w, b[:4]),
                 lambda: ff.linear_fwd(x, w, b, r[:4]), lambda: ff.linear_fwd(x, w, b, r.bfloat16()),
                 lambda: ff.linear_fwd(x.bfloat16(), w), lambda: ff.linear_fwd(x.half(), w.half()),
                 lambda: ff.linear_fwd(x[:0], w), lambda: ff.linear_fwd(x.t().contiguous().t(), w),
                 lambda: ff.linear_fwd(x, w[:0]), lambda: ff.linear_fwd(x, w.cpu()), lambda: ff.linear_fwd(x, w, activation="tanh"),
                 lambda: ff.linear_bwd(grad[:3], x, w), lambda: ff.linear_bwd(grad, x, w, grad),
                 lambda: ff.linear_bwd(grad, x, w, grad.bfloat16(), "silu"), lambda: ff.gated_linear_fwd(x, w2[:15]),
                 lambda: ff.gated_linear_fwd(x, w2, b), lambda: ff.gated_linear_bwd(grad, x, w2, grad)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ff.linear_fwd(x, w, activation=1), lambda: ff.linear_bwd(grad, x, w, None, "silu"),
                 lambda: ff.gated_linear_bwd(grad, x, w2, None), lambda: ff.linear_fwd(x, [1.0])):
        with pytest.raises(TypeError):
            call()


def test_streams_and_graph():
    """Every entry point on a stream of its own, and captured and replayed among eager work."""
    announce("ff streams and graph")
    few, many = case(5, 2048, 264, torch.bfloat16), case(300, 72, 264, torch.bfloat16)
    gfew, gmany = case(5, 2048, 264, torch.bfloat16, True), case(300, 72, 264, torch.bfloat16, True)

    def step(stream=None):
        outs = []
        for args, gated in ((few, False), (many, False), (gfew, True), (gmany, True)):
            x, w, b, r, grad = args
            y, saved = forward(x, w, b, r, "gelu", gated, save=True, stream=stream)
            outs += [y, saved, *backward(grad, x, w, saved, "gelu", gated, stream=stream)]
        return outs

    eager = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = step(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    junk = torch.randn(256, 256, device="cuda")
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        junk = torch.tanh(junk @ junk / 256)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, eager))


# Long contractions with few tiles, for each product of the two passes: cut into pieces that a second kernel adds up.
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("rows,C,N", [(5000, 72, 40), (5001, 77, 41), (90, 72, 5000), (90, 5000, 72), (70, 4999, 71)])
def test_long_sums(rows, C, N, gated, dt):
    announce("ff long sums", rows, C, N, gated, dt)
    compare(*case(rows, C, N, DT[dt], gated), "silu", gated)


@pytest.mark.parametrize("dt", DT)
def test_copied_gradient(dt):
    """Without an activation the products take grad itself; of many rows that are no whole chunks, a copy."""
    announce("ff copied gradient", dt)
    x, w, b, r, grad = case(2051, 1030, 1203, DT[dt])
    compare(x, w, b, r, grad, "none", False)
    wide = torch.full((2051, 1210), float("nan"), device="cuda", dtype=DT[dt])
    wide[:, 3:1206] = grad
    want = ff.linear_bwd(grad, x, w)
    for p, q in zip(ff.linear_bwd(wide[:, 3:1206], x, w), want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("C,N", [(64, 32), (128, 32), (77, 32), (128, 70)])
def test_far_rows(C, N, gated):
    """Rows whose offsets pass 32 bits, in elements: what they are among near ones."""
    announce("ff far rows", C, N, gated)
    rows, ld, dtype = 300, 9000001 if C % 8 else 9000008, torch.bfloat16
    x, w, b, r, grad = case(rows, C, N, dtype, gated)
    base = torch.empty(rows * ld, device="cuda", dtype=dtype)

    def far(t, at):
        v = base.as_strided(t.shape, (ld, 1), at)
        return v.copy_(t)

    xf, gf, rf = far(x, 0), far(grad, 512), far(r, 1024) if r is not None else None
    xn, gn = (torch.cat([t, t[:, :1 if ld % 8 else 8]], 1)[:, :t.shape[1]] for t in (x, grad))
    y, saved = forward(xn, w, b, r, "silu", gated, save=True)
    yf, savedf = forward(xf, w, b, rf, "silu", gated, save=True)
    compare(xf, w, b, rf, gf, "silu", gated)
    assert not bool((xf != x).any()) and not bool((gf != grad).any())
    if C % 8:  # neither takes chunks: the same form, the same bits
        assert torch.equal(y, yf) and torch.equal(saved, savedf)


@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("rows,C,N", [(1 << 20, 64, 2304), (1 << 20, 72, 2304), ((1 << 20) + 1, 65, 2305)])
def test_far_results(rows, C, N, gated):
    """More than 2^31 elements of y, z and dz."""
    announce("ff far results", rows, C, N, gated)
    dtype, k = torch.bfloat16, 300
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(rows, C, generator=gen, device="cuda", dtype=dtype)
    w = torch.randn(N * (2 if gated else 1), C, generator=gen, device="cuda", dtype=dtype) * C ** -0.5
    grad = torch.randn(rows, N, generator=gen, device="cuda", dtype=dtype)
    grad[:-k] = 0  # so that the parameters' gradients are the last rows' too
    y, saved = forward(x, w, None, None, "gelu", gated, save=True)
    gx, gw, gb = backward(grad, x, w, saved, "gelu", gated)
    want = orc.run(x[-k:], w, None, None, "gelu", grad[-k:], gated)
    width = w.shape[0]
    orc.check(y[-k:], want["y"], dtype, "y", 2 * C + 64)
    orc.check(gx[-k:], want["grad_x"], dtype, "grad_x", 2 * (C + width) + 64)
    orc.check(gw, want["grad_weight"], dtype, "grad_weight", 2 * (C + k) + 64)
    orc.check(gb, want["grad_bias"], dtype, "grad_bias", 2 * (C + k) + 64)
    assert not gx[:-k].any()
    head = forward(x[:k], w, None, None, "gelu", gated)[0]
    orc.check(y[:k], orc.run(x[:k], w, None, None, "gelu", gated=gated)["y"], dtype, "y", 2 * C + 64)
    orc.check(head, orc.run(x[:k], w, None, None, "gelu", gated=gated)["y"], dtype, "y", 2 * C + 64)


def test_strides_of_single_elements():
    """The strides of axes of one element mean nothing."""
    announce("ff single elements")
    for gated in (False, True):
        x, w, b, r, grad = case(37, 1, 1, torch.float32, gated)
        odd = [t.as_strided((37, 1), (1, 9)) if t is not None else None for t in (x, r, grad)]
        saved = forward(x, w, b, r, "silu", gated, save=True)[1]
        assert torch.equal(forward(odd[0], w, b, odd[1], "silu", gated)[0], forward(x, w, b, r, "silu", gated)[0])
        for p, q in zip(backward(odd[2], odd[0], w, saved, "silu", gated), backward(grad, x, w, saved, "silu", gated)):
            assert torch.equal(p, q)
        x, w, b, r, grad = case(1, 40, 24, torch.float32, gated)
        odd = x.as_strided((1, 40), (7, 1))
        assert torch.equal(forward(odd, w, b, r, "silu", gated)[0], forward(x, w, b, r, "silu", gated)[0])


# every path of a call: few rows, pieces, copies of x and the weight, few channels, z made again, a copied grad
PATHS = [(5, 2048, 264, "gelu"), (300, 72, 264, "silu"), (2045, 321, 867, "gelu"), (3000, 64, 100, "silu"), (9001, 72, 1352, "silu"),
         (2051, 1030, 1203, "none")]


def step_of(args, act, gated, **kw):
    x, w, b, r, grad = args
    y, saved = forward(x, w, b, r, act, gated, save=True, **kw)
    return [t for t in (y, saved, *backward(grad, x, w, saved, act, gated, **kw)) if t is not None]


@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_two_streams_at_once(gated):
    announce("ff two streams", gated)
    work = [(case(rows, C, N, torch.bfloat16, gated), act) for rows, C, N, act in PATHS]
    want = [step_of(args, act, gated) for args, act in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [[step_of(args, act, gated, stream=s) for args, act in work] for s in streams]
        torch.cuda.synchronize()
        for one in got:
            for p, q in zip(one, want):
                assert len(p) == len(q) and all(torch.equal(a, b) for a, b in zip(p, q))


@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_two_graphs_of_one_pool(gated):
    """Their workspaces may be the same memory; each replay is whole by itself."""
    announce("ff two graphs", gated)
    work = [(case(rows, C, N, torch.bfloat16, gated), act) for rows, C, N, act in PATHS]
    halves = [work[::2], work[1::2]]
    want = [[t.clone() for args, act in half for t in step_of(args, act, gated)] for half in halves]
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for half in halves:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append([t for args, act in half for t in step_of(args, act, gated)])
        pool = g.pool()
        graphs.append(g)
    junk = torch.randn(256, 256, device="cuda")
    for k in (0, 1, 1, 0, 1, 0):
        for t in outs[k]:
            t.fill_(float("nan"))
        junk = torch.tanh(junk @ junk / 256)
        torch.cuda.synchronize()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs[k], want[k])), k


def test_arguments_let_go_of():
    """Tensors given up behind a call on another stream are not handed out before it has read them."""
    announce("ff let go")
    for gated in (False, True):
        args = case(2045, 321, 867, torch.bfloat16, gated)
        want = step_of(args, "gelu", gated)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        busy = torch.randn(4096, 4096, device="cuda")
        torch.cuda.synchronize()
        for _ in range(3):
            own = [t.clone() if t is not None else None for t in args]
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(4):
                    busy @ busy
            got = step_of(own, "gelu", gated, stream=side)
            sizes = [t.shape for t in own if t is not None]
            del own
            junk = [torch.full(s, float("nan"), device="cuda", dtype=torch.bfloat16) for s in sizes for _ in range(2)]
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want))
            del junk
