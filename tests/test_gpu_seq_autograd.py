"""The sequence operators beside torch's autograd: states written in place, forward-mode tangents."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

from dynamic_dilated_depthwise_amd import sequence as seq
from dynamic_dilated_depthwise_amd.mixer import PixelMixer
from test_gpu_seq_norm_conv import announce, conv_case, gen_of, norm_case, randn
from test_gpu_seq_scan import case

pytestmark = pytest.mark.gpu


def test_step_after_a_prompt():
    """A step moves states that a differentiable prompt has kept: its backward must refuse, not use them."""
    announce("step after a prompt")
    torch.manual_seed(3)
    m = PixelMixer(dim=24, heads=2, head_dim=16, state_dim=12).cuda()
    tokens = randn(gen_of(4), 2, 9, 24)
    state = m.new_state(2)
    versions = [t._version for t in state]
    out, _ = m.prompt(tokens, state)
    m.step(tokens[:, 0].contiguous(), state)
    assert all(t._version > v for t, v in zip(state, versions))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def _steps():
    x, w, b, line, _, _ = conv_case(3, 1, 16, 4, torch.float32)
    sx, draw, A, Bm, Cm, D, bias = case(3, 1, 2, 8, 1, 6, torch.float32)
    h = randn(gen_of(5), 3, 2, 8, 6)
    return ((lambda s: seq.causal_conv_step(x[:, 0], w, b, s), line),
            (lambda s: seq.selective_scan_step(sx[:, 0], draw[:, 0], A, Bm[:, 0], Cm[:, 0], D, bias, s), h))


def test_states_that_require_grad():
    """In grad mode a state that requires gradients is not overwritten."""
    announce("states that require grad")
    for step, state in _steps():
        leaf = state.clone().requires_grad_()
        with pytest.raises(ValueError, match="requires grad"):
            step(leaf)
        assert torch.equal(leaf, state)
        version = leaf._version
        with torch.no_grad():
            step(leaf)
        assert leaf._version > version and not torch.equal(leaf, state)
        plain = state.clone()
        step(plain)
        assert torch.equal(plain, leaf.detach())


def test_forward_mode_is_refused():
    """A tangent is never dropped: the differentiable forms raise for dual inputs."""
    announce("forward mode")
    x, w, b, grad = norm_case(6, 40, torch.float32)
    cx, cw, cb, init, _, _ = conv_case(2, 9, 12, 4, torch.float32)
    args = case(2, 9, 2, 8, 1, 6, torch.float32)
    m = PixelMixer(dim=12, heads=2, head_dim=8, state_dim=6).cuda()
    tokens = randn(gen_of(6), 1, 5, 12)
    for mode in (torch.enable_grad, torch.no_grad):
        with mode(), fwAD.dual_level():
            for call in (lambda: seq.layer_norm(fwAD.make_dual(x, grad), w, b),
                         lambda: seq.layer_norm(x, fwAD.make_dual(w, b), b),
                         lambda: seq.causal_conv(cx, cw, cb, fwAD.make_dual(init, init)),
                         lambda: seq.selective_scan(*args[:6], fwAD.make_dual(args[6], args[6])),
                         lambda: m.prompt(fwAD.make_dual(tokens, tokens))):
                with pytest.raises(RuntimeError, match="jvp|forward"):
                    call()
            assert seq.layer_norm(x, w, b).shape == x.shape  # no tangent, no refusal
