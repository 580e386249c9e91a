"""PixelMixer's host logic: constructor refusals, states, no CPU fallback."""
import pytest
import torch

from dynamic_dilated_depthwise_amd.mixer import PixelMixer


@pytest.mark.parametrize("kw", [dict(heads=3, groups=2), dict(width=1), dict(width=9), dict(state_dim=0), dict(state_dim=129)])
def test_constructor_refusals(kw):
    with pytest.raises(ValueError):
        PixelMixer(**kw)


def test_states_and_sizes():
    m = PixelMixer(dim=24, heads=4, head_dim=20, state_dim=18, groups=2, width=3).bfloat16()
    line, h = m.new_state(5)
    assert line.shape == (5, 2, 4 * 20 + 2 * 2 * 18) and line.dtype == torch.bfloat16
    assert h.shape == (5, 4, 20, 18) and h.dtype == torch.float32
    assert all(t.dtype == torch.float32 for t in m._scan_parameters())
    assert m.in_proj.weight.shape == (4 * 20 + m.channels + 4, 24)


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="device tensor"):
        PixelMixer()(torch.zeros(1, 64, 4, 4))


def test_tangents_are_seen():
    """Forward-mode tangents have no requires_grad; the choice of the autograd form sees them."""
    import torch.autograd.forward_ad as fwAD
    from dynamic_dilated_depthwise_amd import sequence as seq
    t = torch.ones(3)
    assert not seq._differentiated(t, None) and seq._differentiated(t, torch.ones(3, requires_grad=True))
    with torch.no_grad():
        assert not seq._differentiated(torch.ones(3, requires_grad=True))
        with fwAD.dual_level():
            assert seq._differentiated(None, t, fwAD.make_dual(t, t)) and not seq._differentiated(t)


@pytest.mark.parametrize("lengths", [torch.zeros(2, dtype=torch.int32), torch.zeros(1), torch.zeros(1, 1, dtype=torch.int32),
                                     torch.zeros(1, dtype=torch.int32, device="meta")])
def test_lengths_are_checked(lengths):
    with pytest.raises(ValueError, match="lengths must be"):
        PixelMixer().prompt(torch.zeros(1, 4, 64), lengths=lengths)
