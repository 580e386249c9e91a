"""Infinities and NaN in scans: what the recurrence makes of them, and no more."""
import pytest
import torch

import seq_oracle as orc
from dynamic_dilated_depthwise_amd import sequence as seq
from test_gpu_seq_norm_conv import DT, announce, gen_of, randn
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


BAD = {"nan": float("nan"), "inf": float("inf")}


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("where", ["x", "dt", "B", "C"])
@pytest.mark.parametrize("at", [0, 15, 16, 31, 40, 63, 64, 90, 127, 128, 140])
def test_tokens_before(at, where, bad, dt):
    """A value that is not finite reaches its token and those behind it, and no earlier one: not in its
    tile of tokens either."""
    announce("scan not finite", at, where, bad, dt)
    P, N = 20, 12
    args = list(case(2, 150, 4, P, 2, N, DT[dt]))
    want, size = orc.scan(*args)
    k = {"x": 0, "dt": 1, "B": 3, "C": 4}[where]
    args[k] = args[k].clone()
    args[k][(1, at, 1, 3)[:args[k].dim()]] = BAD[bad]  # of sequence 1: head 1 (x, dt) or group 1 (B, C)
    y, last, _ = seq.selective_scan_fwd(*args, return_state=True)
    heads = [1] if where in ("x", "dt") else [2, 3]
    touched = torch.zeros(2, 150, 4, P, dtype=torch.bool)
    for h in heads:
        if where == "C":
            touched[1, at, h] = True
        elif where == "x":
            touched[1, at:, h, 3] = True
        else:
            touched[1, at:, h] = True
    y = y.cpu()
    assert not bool(y[touched].isfinite().any())
    assert bool(y[~touched].isfinite().all())
    clean = want["y"].masked_fill(touched, 0)
    orc.check(y.masked_fill(touched, 0), clean, size["y"], DT[dt], "y", operand=None)
    tstate = torch.zeros(2, 4, P, N, dtype=torch.bool)
    if where == "x":
        tstate[1, 1, 3] = True
    elif where == "B":
        tstate[1, 2:, :, 3] = True
    elif where == "dt":
        tstate[1, 1] = True
    last = last.cpu()
    assert not bool(last[tstate].isfinite().any())
    orc.check(last.masked_fill(tstate, 0), want["state"].masked_fill(tstate, 0), size["state"], torch.float32, "state")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("at", [0, 70, 130, 299])
def test_tokens_before_in_segments(at, dt):
    """The same where the call takes segments of chunks, with states that enter them and a length."""
    announce("scan not finite, segments", at, dt)
    H, P, G, N = 512, 8, 256, 12
    args = list(case(1, 310, H, P, G, N, DT[dt]))
    init = randn(gen_of(12), 1, H, P, N)
    lengths = torch.tensor([300], dtype=torch.int32, device="cuda")
    want, size = orc.scan(*args, init, lengths)
    args[0][0, at, 100, 5] = float("nan")
    args[0][0, 300:, 7] = float("nan")
    y, last, _ = seq.selective_scan_fwd(*args, init, lengths, return_state=True)
    touched = torch.zeros(1, 310, H, P, dtype=torch.bool)
    touched[0, at:300, 100, 5] = True
    y, last = y.cpu(), last.cpu()
    assert bool(y[touched].isnan().all()) and bool(last[0, 100, 5].isnan().all())
    orc.check(y.masked_fill(touched, 0), want["y"].masked_fill(touched, 0), size["y"], DT[dt], "y")
    last[0, 100, 5] = want["state"][0, 100, 5].float()
    orc.check(last, want["state"], size["state"], torch.float32, "state")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("where", ["x", "grad"])
def test_gradients_elsewhere(where, dt):
    """What a NaN may reach in the backward: its chunk, what flows on from there in the recurrence and its
    adjoint, and sums over the tokens; not another sequence, nor another head's x and dt."""
    announce("scan gradients not finite", where, dt)
    L, at = 600, 300  # in the third chunk of 128, the fifth of 64: tokens 256 to 383 and 256 to 319
    args = list(case(2, L, 4, 20, 2, 12, DT[dt]))
    grad = randn(gen_of(12), 2, L, 4, 20, dtype=DT[dt])
    saved = seq.selective_scan_fwd(*args, save=True)[2]
    clean = seq.selective_scan_bwd(grad, *args, saved)
    t = args[0] if where == "x" else grad
    t[1, at, 1, 3] = float("nan")
    saved = seq.selective_scan_fwd(*args, save=True)[2]
    got = seq.selective_scan_bwd(grad, *args, saved)
    gx, gdt, gA, gB, gC, gD, gbias, _ = range(8)
    away = slice(0, 256) if where == "x" else slice(384, L)  # x flows on to later states, grad to earlier adjoints
    for k in (gx, gdt, gB, gC):
        assert torch.equal(got[k][0], clean[k][0])
        assert torch.equal(got[k][1, away], clean[k][1, away])
    for k in (gx, gdt):
        assert torch.equal(got[k][:, :, [0, 2, 3]], clean[k][:, :, [0, 2, 3]])
    for k in (gB, gC):
        assert torch.equal(got[k][:, :, 1], clean[k][:, :, 1])
    for k in (gA, gD, gbias):
        assert torch.equal(got[k][[0, 2, 3]], clean[k][[0, 2, 3]])
    assert bool(got[gA][1].isnan()) and bool(got[gD][1].isnan()) and bool(got[gbias][1].isnan())
