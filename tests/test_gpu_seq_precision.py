"""bfloat16 scans whose error is that of their own outputs: no operand made on the way is rounded
to bfloat16 alone.

Tolerances (seq_oracle.check): one rounding of the output to its type and 512 float32 roundings
(2^-15) of the sum's size.  An operand of two bfloat16 terms is off by at most 2^-18 of itself, one
of a single term by 2^-9, which sums of a few dozen terms do not average below 2^-13.
"""
import pytest
import torch

import seq_oracle as orc
from dynamic_dilated_depthwise_amd import sequence as seq
from test_gpu_seq_norm_conv import DT, announce, gen_of, ragged, randn
from test_gpu_seq_scan import NAMES, case

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def close(got, want, size):
    for name, g in got.items():
        orc.check(g, want[name], size[name], g.dtype, name)


# both term counts of P and N that matter: whole vectors and not, one slab and two, one chunk and more
SIZES = [(2, 100, 2, 64, 1, 64), (1, 300, 2, 64, 1, 128), (2, 260, 4, 24, 2, 20), (1, 200, 2, 96, 1, 50), (1, 150, 1, 33, 1, 37)]


@pytest.mark.parametrize("state", [False, True], ids=["fresh", "cached"])
@pytest.mark.parametrize("batch,L,H,P,G,N", SIZES)
def test_outputs(batch, L, H, P, G, N, state):
    announce("scan precision", batch, L, H, P, G, N, state)
    args = case(batch, L, H, P, G, N, BF16)
    init = randn(gen_of(12), batch, H, P, N) if state else None
    y, last, _ = seq.selective_scan_fwd(*args, init, return_state=True, save=True)
    close({"y": y, "state": last}, *orc.scan(*args, init))


# calls that keep nothing and take segments of chunks (512 workgroups of them)
@pytest.mark.parametrize("state", [False, True], ids=["fresh", "cached"])
@pytest.mark.parametrize("batch,L,H,P,G,N", [(1, 300, 512, 8, 256, 24), (1, 1100, 512, 8, 256, 16), (2, 260, 256, 9, 128, 64),
                                             (1, 300, 256, 72, 256, 37)])
def test_segments(batch, L, H, P, G, N, state):
    announce("segments precision", batch, L, H, P, G, N, state)
    args = case(batch, L, H, P, G, N, BF16)
    init = randn(gen_of(12), batch, H, P, N) if state else None
    lengths = ragged(batch, L) if batch > 1 else None
    y, last, _ = seq.selective_scan_fwd(*args, init, lengths, return_state=True)
    close({"y": y, "state": last}, *orc.scan(*args, init, lengths))


@pytest.mark.parametrize("batch,L,H,P,G,N", SIZES)
def test_gradients(batch, L, H, P, G, N):
    announce("scan gradients' precision", batch, L, H, P, G, N)
    args = case(batch, L, H, P, G, N, BF16)
    g = gen_of(12)
    grad, init, gs = randn(g, batch, L, H, P, dtype=BF16), randn(g, batch, H, P, N), randn(g, batch, H, P, N)
    saved = seq.selective_scan_fwd(*args, init, save=True)[2]
    got = dict(zip(NAMES, seq.selective_scan_bwd(grad, *args, saved, init, None, gs)))
    close(got, *orc.scan(*args, init, grad=grad, grad_state=gs))


@pytest.mark.parametrize("dt", DT)
def test_slow_after_fast(dt):
    """Small steps that follow many strong ones in a chunk: their decays are differences of large sums."""
    announce("scan slow after fast", dt)
    args = list(case(1, 250, 2, 16, 1, 12, DT[dt], fast=True))
    args[1][:, :60] = 1000.0
    args[1][:, 60:] = -4.0 - args[6].to(DT[dt])  # dt about 0.02 whatever the bias
    y, last, _ = seq.selective_scan_fwd(*args, return_state=True)
    close({"y": y, "state": last}, *orc.scan(*args))
