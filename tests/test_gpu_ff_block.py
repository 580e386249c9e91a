"""PixelFeedForward (layer norm, gated projection and projection back run together) and PixelBlock
against the same formulas in 64 bits: maps, ragged prompts, single tokens, gradients, a captured step.

Tolerances, relative to a tensor's largest value: in float32 three operators of up to a few hundred
roundings each, carried on with factors of a few: 2^-12.  In bfloat16 the norm's output, the gated
product and the gradients between the operators are rounded once each (2^-9 of their values, which the
following sums average but the normalisation and the gate can double): 2^-6; with the mixer before it
2^-5 (its own) more.  Gradients of parameters are sums over all tokens of terms of both signs and come
out at a part of their terms' size: four times that.
"""
import pytest
import torch

import ff_oracle as orc
from dynamic_dilated_depthwise_amd.mixer import PixelBlock, PixelFeedForward, PixelMixer
from test_gpu_ff import DT, announce, gen_of, randn

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2.0 ** -12, torch.bfloat16: 2.0 ** -6}
WITH_MIXER = {torch.float32: 2.0 ** -11, torch.bfloat16: 2.0 ** -5 + 2.0 ** -6}


def make(kind, dtype, seed=7, **kw):
    torch.manual_seed(seed)
    m = kind(**kw)
    with torch.no_grad():
        for k, p in m.named_parameters():
            if k.endswith("up_bias") or k.endswith("down_bias") or k.endswith("norm_bias"):
                p.copy_(torch.randn_like(p) * 0.2)
    return m.cuda().to(dtype)


def plain(m, tokens, p):
    """PixelFeedForward.tokens from its formulas; p: the parameters by name, 64 bits."""
    mean = tokens.mean(-1, keepdim=True)
    rs = 1 / torch.sqrt(((tokens - mean) ** 2).mean(-1, keepdim=True) + m.eps)
    z = ((tokens - mean) * rs * p["norm_weight"] + p["norm_bias"]) @ p["up_weight"].t()
    z = z + p["up_bias"] if m.up_bias is not None else z
    g, u = z.split(m.hidden, -1)
    y = (orc.curve(g, m.activation)[0] * u) @ p["down_weight"].t()
    return tokens + (y + p["down_bias"] if m.down_bias is not None else y)


def wide(m):
    return {k: t.detach().double().requires_grad_() for k, t in m.named_parameters()}


def near(got, want, tol, name):
    err = float((got.detach().double() - want.detach()).abs().max() / want.detach().abs().max())
    assert err <= tol, f"{name}: {err:.3g}"


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("kw,shape", [(dict(), (1, 64, 12, 17)), (dict(dim=24, hidden=37, activation="gelu"), (2, 24, 5, 7)),
                                      (dict(dim=33, hidden=80, bias=False, activation="relu"), (1, 33, 3, 1))])
def test_map_and_gradients(kw, shape, dt):
    announce("ff block map", kw, shape, dt)
    dtype = DT[dt]
    m = make(PixelFeedForward, dtype, **kw)
    g = gen_of(31)
    x, grad = randn(g, *shape, dtype=dtype), randn(g, *shape, dtype=dtype)
    with torch.no_grad():
        quiet = m(x)
    x.requires_grad_()
    out = m(x)
    out.backward(grad)
    assert torch.equal(out, quiet)
    p = wide(m)
    xd = x.detach().double().requires_grad_()
    want = plain(m, xd.flatten(2).transpose(1, 2), p).transpose(1, 2).unflatten(2, shape[2:])
    want.backward(grad.double())
    near(out, want, TOL[dtype], "out")
    near(x.grad, xd.grad, TOL[dtype], "grad x")
    for k, t in m.named_parameters():
        near(t.grad, p[k].grad, 4 * TOL[dtype], "grad " + k)


@pytest.mark.parametrize("dt", DT)
def test_block_prompt_then_tokens(dt):
    """A ragged prompt with garbage past its lengths, then tokens from its states: the block is the mixer
    and the feed-forward of each token."""
    announce("ff block prompt", dt)
    dtype = DT[dt]
    m = make(PixelBlock, dtype, dim=40, hidden=72, heads=3, head_dim=16, state_dim=24)
    assert isinstance(m.mixer, PixelMixer)
    batch, L = 3, 21
    tokens = randn(gen_of(32), batch, L + 1, 40, dtype=dtype)
    lengths = torch.tensor([21, 9, 0], dtype=torch.int32, device="cuda")
    past = torch.arange(L, device="cuda")[None] >= lengths[:, None]
    prompt = tokens[:, :L].masked_fill(past[..., None], float("nan"))
    out, state = m.prompt(prompt, lengths=lengths)
    mixed, mstate = m.mixer.prompt(prompt, lengths=lengths)
    assert all(torch.equal(a, b) for a, b in zip(state, mstate))
    p = wide(m.feed_forward)
    near(out[~past], plain(m.feed_forward, mixed[~past].double(), p), TOL[dtype], "prompt")
    assert bool(out[past].isnan().all())
    out.masked_fill(past[..., None], 0).float().square().sum().backward()
    assert all(bool(t.grad.isfinite().all()) for t in m.parameters())
    with torch.no_grad():
        state2 = [t.detach().clone() for t in state]
        one = m.step(tokens[:, L], state2)
        line = [t.detach().clone() for t in state]
        near(one, plain(m.feed_forward, m.mixer.step(tokens[:, L], line).double(), p), TOL[dtype], "step")
        assert all(torch.equal(a, b) for a, b in zip(state2, line))


@pytest.mark.parametrize("dt", DT)
def test_block_gradients(dt):
    """A map through the block: gradients through the feed-forward into the mixer's."""
    announce("ff block gradients", dt)
    dtype = DT[dt]
    m = make(PixelBlock, dtype, dim=24, hidden=40, heads=2, head_dim=16, state_dim=12)
    g = gen_of(33)
    x, grad = randn(g, 1, 24, 6, 5, dtype=dtype).requires_grad_(), randn(g, 1, 24, 6, 5, dtype=dtype)
    m(x).backward(grad)
    # the mixer's output as a leaf: the feed-forward's gradients against the formulas, and what it hands on
    xm = x.detach().requires_grad_()
    mixed = m.mixer(xm)
    leaf = mixed.detach().double().flatten(2).transpose(1, 2).requires_grad_()
    p = wide(m.feed_forward)
    want = plain(m.feed_forward, leaf, p)
    want.backward(grad.double().flatten(2).transpose(1, 2))
    for k, t in m.feed_forward.named_parameters():
        near(t.grad, p[k].grad, 4 * TOL[dtype], "grad " + k)
    mixed.backward(leaf.grad.to(dtype).transpose(1, 2).unflatten(2, (6, 5)))
    near(x.grad, xm.grad.double(), WITH_MIXER[dtype], "grad x")


def test_autocast():
    """Under autocast the module's type stays, also for tokens of another one."""
    announce("ff block autocast")
    m = make(PixelFeedForward, torch.float32, dim=24, hidden=40)
    x = randn(gen_of(34), 5, 24)
    with torch.no_grad():
        want = m.tokens(x)
        with torch.autocast("cuda", torch.bfloat16):
            assert torch.equal(m.tokens(x), want)
            low = m.tokens(x.bfloat16())
        assert low.dtype == torch.float32 and torch.equal(low, m.tokens(x.bfloat16().float()))


def test_captured_training_step():
    """Gradients in a graph, replayed beside eager work; no eager graph of the leaves is left at the capture."""
    announce("ff block graph")
    m = make(PixelFeedForward, torch.bfloat16, dim=64, hidden=128)
    x, grad = randn(gen_of(35), 1, 64, 16, 16, dtype=torch.bfloat16), randn(gen_of(36), 1, 64, 16, 16, dtype=torch.bfloat16)
    leaves = list(m.parameters())

    def step():
        out = m(x)
        return (out.detach(), *torch.autograd.grad(out, leaves, grad))

    eager = [t.clone() for t in step()]
    torch.cuda.synchronize()
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
