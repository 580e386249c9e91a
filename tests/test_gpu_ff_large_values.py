"""float32 operands up to the type's largest numbers, in each place of each product: what is a number in 64
bits and float32 is one here, and the right one.

Tolerances are ff_oracle.check's.  The operands beside the large ones are small, so that no term and no sum
leaves float32's range.
"""
import pytest
import torch

import ff_oracle as orc
from dynamic_dilated_depthwise_amd import feedforward as ff
from test_gpu_ff import announce, case

pytestmark = pytest.mark.gpu

MOST = torch.finfo(torch.float32).max
LARGE = [-MOST, MOST, 3.3895313892515355e38, -3.3961775292304e38, 3.3961778e38, -3.2e38]  # bfloat16's largest, half a step above, ...


def spread(t):
    """t, small, with a large value in each of its first rows, no two in one column."""
    t = t.mul(0.02).clamp(-0.08, 0.08)
    for k in range(min(len(LARGE), *t.shape)):
        t[k, k] = LARGE[k]
    return t


def product(a, b):
    """a b^T in 64 bits, the same of the terms' absolute values, and no operand that is rounded."""
    a, b = a.double(), b.double()
    want = a @ b.t()
    return want, a.abs() @ b.abs().t(), torch.zeros_like(want)


def places(x, w, grad):
    """The three operands, small but for one of them at a time."""
    small = [t.mul(0.02).clamp(-0.08, 0.08) for t in (x, w, grad)]
    for k in range(3):
        yield (k, *(spread(t) if k == i else s for i, (t, s) in enumerate(zip((x, w, grad), small))))


def gradients(dz, x, w):
    return {"grad_x": product(dz, w.t()), "grad_weight": product(dz.t(), x.t()),
            "grad_bias": product(dz.t(), torch.ones(1, len(dz), device="cuda"))}


def compare(got, want, place, count):
    for name, t in zip(want, got):
        assert float(want[name][1].max()) <= MOST, "the case leaves float32's range"
        value, size, none = (v.reshape(t.shape) for v in want[name])
        orc.check(t, (value, size, none), torch.float32, f"{name}, place {place}", count)


# few rows (whole chunks and not), tiles (whole chunks and not, pieces, several tiles)
SIZES = [(1, 64, 40), (6, 65, 40), (40, 200, 24), (300, 72, 264), (300, 65, 130), (130, 4096, 72), (90, 72, 5000), (2600, 264, 2312)]


@pytest.mark.parametrize("rows,C,N", SIZES)
def test_products(rows, C, N):
    announce("ff large values", rows, C, N)
    x, w, _, _, grad = case(rows, C, N, torch.float32)
    for place, x, w, grad in places(x, w, grad):
        compare([ff.linear_fwd(x, w)[0]], {"y": product(x, w)}, place, 2 * C + 64)
        compare(ff.linear_bwd(grad, x, w), gradients(grad, x, w), place, 2 * (C + N + rows) + 64)


@pytest.mark.parametrize("rows,C,N", [(70, 64, 100), (33, 40, 60)])
def test_few_channels(rows, C, N):
    """The backward in one kernel, behind relu: dz is grad or zero, and a bias of one leaves no z near zero."""
    announce("ff large values, few channels", rows, C, N)
    x, w, b, _, grad = case(rows, C, N, torch.float32)
    b.fill_(1)
    for place, x, w, grad in places(x, w, grad):
        y, saved = ff.linear_fwd(x, w, b, activation="relu", save=True)
        z = product(x, w)
        compare([y], {"y": ((z[0] + 1).clamp(min=0), z[1] + 1, z[2])}, place, 2 * C + 64)
        assert bool((((z[0] + 1).abs() > 1e-4 * z[1]) | ((z[0] + 1).abs() > 0.1)).all())  # whose sign is sure
        compare(ff.linear_bwd(grad, x, w, saved, "relu"), gradients(grad * (z[0] > -1), x, w), place, 2 * (C + N + rows) + 64)
