"""What the differentiable feed-forward operators keep for their backward."""
import pytest
import torch

from dynamic_dilated_depthwise_amd import feedforward as ff
from test_gpu_ff import announce, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "silu"])
def test_residual_alone_keeps_nothing(act):
    """Its gradient is grad: neither z nor the operands are kept, and they may change before the backward."""
    announce("ff residual alone", act)
    x, w, b, r, grad = case(300, 72, 264, torch.bfloat16)
    want = ff.linear_fwd(x, w, b, r, act)[0]
    y = ff.linear(x, w, b, r.requires_grad_(), act)
    assert torch.equal(y, want) and not y.grad_fn.saved_tensors
    x.zero_()
    y.backward(grad)
    assert torch.equal(r.grad, grad)
    y = ff.linear(x, w, b.requires_grad_(), r, act)
    assert len(y.grad_fn.saved_tensors) == 3 and (y.grad_fn.saved_tensors[2] is None) == (act == "none")
