"""Feed-forward operators whose error is that of their own outputs: nothing made on the way is rounded to
bfloat16 alone.

Tolerances.  Each element (ff_oracle.check): one rounding of the output, float32 roundings of the sums, and
u(bfloat16)^2 of the gradient of the activation's or gate's input, which is what two bfloat16 terms leave
of it.  All elements together: the error's norm is at most 1.1 times that of the result's own rounding.
What the float32 sums and the second term's rounding add to it is below 2^-7 of that; a gradient in one
term adds a second rounding of the same size (1.41 times), and over the thousand and more elements of an
output (a hundred of grad_bias, whose roundings are the same ones on both sides but for few) neither
moves by a tenth.
"""
import pytest
import torch

import ff_oracle as orc
from test_gpu_ff import announce, backward, case, forward

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def close(got, want, name, count):
    value, size, operand = want
    orc.check(got, (value, size, operand * orc.u(BF16)), BF16, name, count)
    one = (value.to(BF16).double() - value).norm()
    err = (got.double() - value).norm()
    assert float(err) <= 1.1 * float(one), f"{name}: {float(err / one):.3f} times its rounding's error"


# z kept and dz by a kernel of its own (whole chunks, copies, one step, pieces, a few rows, large tiles), z made
# again (whole chunks and copies), few channels in one kernel
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,C,N", [(300, 72, 264), (2045, 321, 867), (129, 130, 135), (5000, 96, 200), (9, 2048, 264),
                                      (2048, 2048, 2304), (9001, 72, 1352), (8200, 37, 1501), (3000, 64, 100), (40001, 50, 77)])
def test_gradients(rows, C, N, act, gated):
    announce("ff gradients' precision", rows, C, N, act, gated)
    x, w, b, r, grad = case(rows, C, N, BF16, gated)
    saved = forward(x, w, b, r, act, gated, save=True)[1]
    gx, gw, gb = backward(grad, x, w, saved, act, gated)
    want = orc.run(x, w, b, r, act, grad, gated)
    width = w.shape[0]
    close(gx, want["grad_x"], "grad_x", 2 * (C + width) + 64)
    close(gw, want["grad_weight"], "grad_weight", 2 * (C + rows) + 64)
    close(gb, want["grad_bias"], "grad_bias", 2 * (C + rows) + 64)


@pytest.mark.parametrize("rows,C,N", [(70, 8, 16), (300, 72, 264), (70, 77, 35), (9001, 72, 1352)])
def test_gradient_beyond_the_type(rows, C, N):
    """A gate's gradient between bfloat16's largest number and float32's: the products of it that are numbers."""
    announce("ff gradient beyond bfloat16", rows, C, N)
    x, w, b, _, grad = (torch.zeros_like(t) if t is not None else None for t in case(rows, C, N, BF16, True))
    b[N], grad[3, 0], w[0, :] = 1 + 2.0 ** -7, 1.984375 * 2.0 ** 127, 0.5  # u of column 0, and what weighs dg
    saved = forward(x, w, b, None, "none", True, save=True)[1]
    gx, gw, gb = backward(grad, x, w, saved, "none", True)
    dg = (1 + 2.0 ** -7) * 1.984375 * 2.0 ** 127
    assert torch.finfo(BF16).max < dg < torch.finfo(torch.float32).max
    want = torch.zeros_like(gx)
    want[3] = dg / 2
    assert torch.equal(gx, want)
    assert not gw.any() and not gb[1:].any()
