"""Infinities and NaN in scans: what the recurrence makes of them, and no more."""
import pytest
import torch

import seq_oracle as orc
from dynamic_dilated_depthwise_amd import sequence as seq
from test_gpu_seq_norm_conv import DT, announce
from test_gpu_seq_scan import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("save", [False, True], ids=["alone", "saved"])
def test_nan_decay_rate(save, dt):
    """A head whose A is NaN has no finite output; the others do not notice."""
    announce("scan NaN in A", save, dt)
    args = list(case(2, 150, 3, 16, 1, 20, DT[dt]))
    y, last, _ = seq.selective_scan_fwd(*args, return_state=True, save=save)
    args[2] = args[2].clone()
    args[2][1] = float("nan")
    y2, last2, _ = seq.selective_scan_fwd(*args, return_state=True, save=save)
    assert bool(y2[:, :, 1].isnan().all()) and bool(last2[:, 1].isnan().all())
    for h in (0, 2):
        assert torch.equal(y2[:, :, h], y[:, :, h]) and torch.equal(last2[:, h], last[:, h])
