"""PixelMixer (layer norm, convolution and scan run together) against the same formulas in 64
bits: maps, prompts in parts, single tokens in a cache of states, gradients, a captured step.

Tolerances, relative to a tensor's largest value: in float32 the mixer adds to the operators'
512 roundings (2^-15) sums of up to 256 terms in its projections, whose errors the next
operators carry on with factors of a few: 2^-12.  In bfloat16 each of the nine tensors between
the operators is rounded once (2^-9 of its values, which the following sums average but the
normalisation and the gate can double): 2^-5.  Gradients of parameters are sums over all
tokens of terms of both signs and come out at a part of their terms' size: four times that.
"""
import pytest
import torch
import torch.nn.functional as F

import seq_oracle as orc
from dynamic_dilated_depthwise_amd.mixer import PixelMixer
from test_gpu_seq_norm_conv import DT, announce, gen_of, randn

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2.0 ** -12, torch.bfloat16: 2.0 ** -5}


def mixer(dtype, seed=7, **kw):
    torch.manual_seed(seed)
    return PixelMixer(**kw).cuda().to(dtype)


def plain(m, tokens, p, state=None, lengths=None):
    """PixelMixer.prompt from its formulas, on the CPU; p: the parameters by name, 64 bits."""
    batch, L, _ = tokens.shape
    mean = tokens.mean(-1, keepdim=True)
    rs = 1 / torch.sqrt(((tokens - mean) ** 2).mean(-1, keepdim=True) + m.eps)
    t = (tokens - mean) * rs * p["norm_weight"] + p["norm_bias"]
    z, u, raw = (t @ p["in_proj.weight"].t()).split([m.inner, m.channels, m.heads], -1)
    first, h = state if state is not None else (None, None)
    u, last = orc._conv(u, p["conv_weight"], p["conv_bias"], first, lengths)
    v, B, C = u.split([m.inner, m.shared, m.shared], -1)
    on = torch.ones(batch, L, dtype=torch.bool)
    if lengths is not None:
        on = torch.arange(L)[None] < lengths.cpu()[:, None]
    raw = raw + p["dt_bias"]
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    y, h = orc._scan(v.unflatten(-1, (m.heads, m.head_dim)), dt, dt, -torch.exp(p["A_log"]),
                     B.unflatten(-1, (m.groups, m.state_dim)), C.unflatten(-1, (m.groups, m.state_dim)), p["D"], h, on)
    return tokens + (y.flatten(-2) * F.silu(z)) @ p["out_proj.weight"].t(), (last, h)


def wide(m):
    return {k: t.detach().double().cpu().requires_grad_() for k, t in m.named_parameters()}


def near(got, want, dtype, name, times=1):
    err = float((got.detach().double().cpu() - want.detach()).abs().max() / want.detach().abs().max())
    assert err <= times * TOL[dtype], f"{name}: {err:.3g}"


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("kw,shape", [(dict(), (1, 64, 12, 17)), (dict(dim=24, heads=4, head_dim=20, state_dim=18, groups=2, width=3),
                                                                   (2, 24, 5, 7))])
def test_map_and_gradients(kw, shape, dt):
    announce("mixer map", kw, shape, dt)
    dtype = DT[dt]
    m = mixer(dtype, **kw)
    g = gen_of(31)
    x, grad = randn(g, *shape, dtype=dtype), randn(g, *shape, dtype=dtype)
    with torch.no_grad():
        quiet = m(x)
    x.requires_grad_()
    out = m(x)
    out.backward(grad)
    near(out, quiet.double().cpu(), dtype, "with and without gradients")
    p = wide(m)
    xd = x.detach().double().cpu().requires_grad_()
    want, _ = plain(m, xd.flatten(2).transpose(1, 2), p)
    want = want.transpose(1, 2).unflatten(2, shape[2:])
    want.backward(grad.double().cpu())
    near(out, want, dtype, "out")
    near(x.grad, xd.grad, dtype, "grad x")
    for k, t in m.named_parameters():
        near(t.grad, p[k].grad, dtype, "grad " + k, 4)


@pytest.mark.parametrize("dt", DT)
def test_prompt_then_tokens(dt):
    """A ragged prompt, its states put into a larger cache, three tokens a sequence from there."""
    announce("mixer prompt", dt)
    dtype = DT[dt]
    m = mixer(dtype, dim=40, heads=3, head_dim=16, state_dim=24)
    batch, L, more = 3, 37, 3
    tokens = randn(gen_of(32), batch, L + more, 40, dtype=dtype)
    lengths = torch.tensor([37, 20, 2], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        out, (line, h) = m.prompt(tokens[:, :L].contiguous(), lengths=lengths)
    slots = torch.tensor([4, 0, 3], dtype=torch.int32, device="cuda")
    cache = m.new_state(5)
    for c, t in zip(cache, (line, h)):
        c[slots.long()] = t
    steps = [m.step(tokens[:, L + k], cache, slots) for k in range(more)]
    p = {k: t.detach() for k, t in wide(m).items()}
    for b in range(batch):
        n = int(lengths[b])
        own = torch.cat([tokens[b, :n], tokens[b, L:]])[None].double().cpu()
        want, (wline, wh) = plain(m, own, p)
        near(out[b, :n], want[0, :n], dtype, "prompt")
        assert torch.equal(out[b, n:], tokens[b, n:L])
        near(torch.stack([s[b] for s in steps]), want[0, n:], dtype, "steps")
        near(cache[0][slots[b]], wline[0], dtype, "convolution's state")
        near(cache[1][slots[b]], wh[0], dtype, "scan's state")
    # in two parts through the state
    one, _ = m.prompt(tokens)
    a, state = m.prompt(tokens[:, :11].contiguous())
    b_, _ = m.prompt(tokens[:, 11:].contiguous(), state)
    near(torch.cat([a, b_], 1), one.detach().double().cpu(), dtype, "two parts")


def test_captured_training_step():
    """Gradients in a graph, replayed beside eager work; no eager graph of the leaves is left at the capture."""
    announce("mixer graph")
    m = mixer(torch.float32, dim=32, heads=2, head_dim=32, state_dim=16)
    g = gen_of(33)
    x, grad = randn(g, 1, 32, 9, 9), randn(g, 1, 32, 9, 9)
    params = list(m.parameters())

    def step():
        return torch.autograd.grad(m(x), params, grad)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    junk = torch.randn(256, 256, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        junk = torch.tanh(junk @ junk / 256)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, e in zip(got, eager):
            near(t, e.double().cpu(), torch.float32, "replayed gradient")


def test_refusals():
    announce("mixer refusals")
    m = mixer(torch.float32)
    for bad in (torch.zeros(1, 63, 4, 4, device="cuda"), torch.zeros(64, 4, 4, device="cuda")):
        with pytest.raises(ValueError):
            m(bad)
    with pytest.raises(ValueError):
        m.prompt(torch.zeros(1, 64, device="cuda"))
    with pytest.raises(ValueError):
        m.step(torch.zeros(1, 63, device="cuda"), m.new_state(1))
    with pytest.raises(ValueError):
        m(torch.zeros(1, 64, 4, 4, device="cuda", dtype=torch.float16))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_autocast(kind):
    """A float32 mixer under autocast: the projections in autocast's type, the operators and states in
    float32.  Tolerances as for the bfloat16 mixer, whose roundings are a part of these or coarser."""
    announce("mixer autocast", kind)
    m = mixer(torch.float32, dim=24, heads=4, head_dim=20, state_dim=18, groups=2, width=3)
    g = gen_of(35)
    x, grad = randn(g, 2, 24, 5, 7), randn(g, 2, 24, 5, 7)
    x.requires_grad_()
    with torch.autocast("cuda", dtype=kind):
        out = m(x)
    out.backward(grad)
    p = wide(m)
    xd = x.detach().double().cpu().requires_grad_()
    want, _ = plain(m, xd.flatten(2).transpose(1, 2), p)
    want = want.transpose(1, 2).unflatten(2, (5, 7))
    want.backward(grad.double().cpu())
    near(out, want, torch.bfloat16, "out")
    near(x.grad, xd.grad, torch.bfloat16, "grad x")
    for k, t in m.named_parameters():
        assert t.grad.dtype == torch.float32
        near(t.grad, p[k].grad, torch.bfloat16, "grad " + k, 4)
    # a prompt in autocast's own type, its states, and tokens from there
    tokens = randn(g, 2, 6, 24).to(kind)
    with torch.no_grad(), torch.autocast("cuda", dtype=kind):
        start, state = m.prompt(tokens[:, :4].contiguous())
        rest = [m.step(tokens[:, t].contiguous(), state) for t in (4, 5)]
    assert all(t.dtype == torch.float32 for t in state)
    want, _ = plain(m, tokens.double().cpu(), {k: t.detach() for k, t in p.items()})
    near(torch.cat([start, torch.stack(rest, 1)], 1), want, torch.bfloat16, "prompt and tokens")


@pytest.mark.parametrize("dt", DT)
def test_past_a_length(dt):
    """Tokens past a length come out as they are and take part in no gradient, whatever they and the
    gradients there hold."""
    announce("mixer past a length", dt)
    dtype = DT[dt]
    m = mixer(dtype, dim=24, heads=2, head_dim=16, state_dim=12)
    g = gen_of(36)
    tokens, grad = randn(g, 2, 9, 24, dtype=dtype), randn(g, 2, 9, 24, dtype=dtype)
    lengths = torch.tensor([9, 4], dtype=torch.int32, device="cuda")
    params = list(m.parameters())

    def run(fill, gfill):
        t, gr = tokens.clone(), grad.clone()
        t[1, 4:], gr[1, 4:] = fill, gfill
        t.requires_grad_()
        out, _ = m.prompt(t, lengths=lengths)
        return out.detach(), torch.autograd.grad(out, [t, *params], gr)

    out, (gt, *gp) = run(0.0, 0.0)
    for bad in (float("nan"), float("inf")):
        out2, (gt2, *gp2) = run(bad, bad)
        same = torch.full_like(out2[1, 4:], bad)
        assert torch.equal(out2[0], out[0]) and torch.equal(out2[1, :4], out[1, :4])
        assert torch.equal(out2[1, 4:], same) or bool(out2[1, 4:].isnan().all() and same.isnan().all())
        assert torch.equal(gt2[0], gt[0]) and torch.equal(gt2[1, :4], gt[1, :4])
        assert all(torch.equal(p, q) for p, q in zip(gp, gp2))
