"""The sequence operators where calls take other paths: scans long enough for segments of chunks,
infinities next to a length, arguments let go of while their stream still works."""
import pytest
import torch

import seq_oracle as orc
from dynamic_dilated_depthwise_amd import sequence as seq
from test_gpu_seq_norm_conv import DT, announce, conv_case, gen_of, norm_case, ragged, randn
from test_gpu_seq_scan import case, compare

pytestmark = pytest.mark.gpu


# A call that keeps nothing takes segments where 512 workgroups (batch * segments * groups * pairs
# of heads or slabs) are left: two heads at once; one head, odd P and N; two slabs at once.
# Tolerances as for the scan's other calls: what a segment adds to the entering state is rounded
# relative to its own size, which is part of the sum's.
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("state", [False, True], ids=["fresh", "cached"])
@pytest.mark.parametrize("batch,L,H,P,G,N", [(1, 1300, 512, 4, 256, 6), (2, 700, 128, 9, 128, 37), (3, 260, 96, 70, 96, 100)])
def test_scan_segments(batch, L, H, P, G, N, state, dt):
    announce("scan segments", batch, L, H, P, G, N, state, dt)
    dtype = DT[dt]
    args = list(case(batch, L, H, P, G, N, dtype))
    init = randn(gen_of(12), batch, H, P, N) if state else None
    lengths = ragged(batch, L) if state else None
    clean = list(args)
    if lengths is not None:
        off = torch.arange(L, device="cuda")[None] >= lengths[:, None]
        for k in (0, 1, 3, 4):
            args[k][off] = float("nan")
            clean[k] = args[k].masked_fill(off[(...,) + (None,) * (args[k].dim() - 2)], 0)
    y, last, _ = seq.selective_scan_fwd(*args, init, lengths, return_state=True)
    want, size = orc.scan(*clean, init, lengths)
    compare({"y": y, "state": last}, want, size, dtype)
    kept, end, _ = seq.selective_scan_fwd(*args, init, lengths, return_state=True, save=True)
    compare({"y": kept, "state": end}, want, size, dtype)


@pytest.mark.parametrize("dt", DT)
def test_conv_infinity_before_a_length(dt):
    """What the taps reach from past a length changes nothing there."""
    announce("conv infinity", dt)
    x, w, b, _, grad, _ = conv_case(2, 40, 24, 4, DT[dt])
    lengths = torch.tensor([17, 40], dtype=torch.int32, device="cuda")
    x[0, 16] = float("inf")
    y, last = seq.causal_conv_fwd(x, w, b, lengths=lengths, return_state=True)
    gx = seq.causal_conv_bwd(grad, x, w, b, lengths=lengths)[0]
    assert bool((y[0, 17:] == 0).all()) and bool((gx[0, 17:] == 0).all())
    assert bool(torch.isinf(last[0, -1]).all())
    clean = x.clone()
    clean[0, 16] = 0
    assert torch.equal(gx[1], seq.causal_conv_bwd(grad, clean, w, b, lengths=lengths)[0][1])


def test_arguments_let_go_of():
    """A call on a stream of its own keeps its arguments' memory until it is done."""
    announce("arguments let go of")
    x, w, b, _ = norm_case(4096, 512, torch.float32)
    want = seq.layer_norm_fwd(x, w, b)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    y = seq.layer_norm_fwd(x, w, b, stream=side)[0]
    shape = x.shape
    del x
    torch.full(shape, float("nan"), device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_without_gradients():
    """The differentiable forms give the same values where no gradient is asked for."""
    announce("without gradients")
    x, w, b, grad = norm_case(12, 40, torch.float32)
    leaf = x.clone().requires_grad_()
    y = seq.layer_norm(leaf, w, b)
    assert y.requires_grad and not seq.layer_norm(x, w, b).requires_grad
    with torch.no_grad():
        assert torch.equal(seq.layer_norm(leaf, w, b), y)
    with pytest.raises(RuntimeError):  # once differentiable
        g, = torch.autograd.grad(y, leaf, grad, create_graph=True)
        g.sum().backward()


def test_steps_without_slots():
    """Fewer states than sequences are refused: the rest would have had no output and no state."""
    announce("steps without slots")
    x, w, b, line, _, _ = conv_case(3, 1, 16, 4, torch.float32)
    with pytest.raises(ValueError, match="places"):
        seq.causal_conv_step(x[:, 0], w, b, line[:2].contiguous())
    sx, draw, A, Bm, Cm, D, bias = case(3, 1, 2, 8, 1, 6, torch.float32)
    with pytest.raises(ValueError, match="places"):
        seq.selective_scan_step(sx[:, 0], draw[:, 0], A, Bm[:, 0], Cm[:, 0], D, bias, torch.zeros(2, 2, 8, 6, device="cuda"))
    seq.selective_scan_step(sx[:, 0], draw[:, 0], A, Bm[:, 0], Cm[:, 0], D, bias, torch.zeros(2, 2, 8, 6, device="cuda"),
                            torch.tensor([1, 0, -1], dtype=torch.int32, device="cuda"))
