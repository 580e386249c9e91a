"""Batches whose rows pass 2^31."""
import pytest
import torch

from dynamic_dilated_depthwise_amd import sequence as seq
from test_gpu_seq_norm_conv import announce

pytestmark = pytest.mark.gpu


def test_conv_state_of_many_sequences():
    """batch * (width - 1) passes 2^31: the returned state of every sequence is its own last inputs."""
    announce("conv state of many sequences")
    W, batch = 8, (1 << 31) // 7 + 100
    x = torch.empty(batch, 1, 1, device="cuda", dtype=torch.bfloat16)
    x.view(-1).copy_(torch.arange(batch, device="cuda", dtype=torch.int32) % 251)
    x += 1
    w, b = torch.zeros(1, W, device="cuda", dtype=torch.bfloat16), torch.zeros(1, device="cuda", dtype=torch.bfloat16)
    _, last = seq.causal_conv_fwd(x, w, b, return_state=True)
    assert bool((last[:, :W - 2] == 0).all())
    assert torch.equal(last[:, W - 2], x[:, 0])
