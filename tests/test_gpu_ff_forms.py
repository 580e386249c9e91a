"""Every kernel of the feed-forward operators (ff_cases.py) against 64 bits.

Tolerances: ff_oracle.check's of each element, and in bfloat16 of all of them together that the error's norm is
at most 1.1 times that of the result's own rounding (test_gpu_ff_precision.py).
"""
import pytest
import torch

import ff_oracle as orc
from ff_cases import CASES
from test_gpu_ff import DT, announce, backward, case, forward

pytestmark = pytest.mark.gpu

IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("dt,op,act,rows,C,N", CASES, ids=IDS)
def test_forms(dt, op, act, rows, C, N):
    announce("ff forms", dt, op, act, rows, C, N)
    dtype, gated = DT[dt], op == "gated"
    x, w, b, r, grad = case(rows, C, N, dtype, gated)
    y, saved = forward(x, w, b, r, act, gated, save=True)
    gx, gw, gb = backward(grad, x, w, saved, act, gated)
    want, width = orc.run(x, w, b, r, act, grad, gated), w.shape[0]
    for name, t, count in (("y", y, C), ("grad_x", gx, C + width), ("grad_weight", gw, C + rows), ("grad_bias", gb, C + rows)):
        value, size, operand = want[name]
        orc.check(t, (value, size, operand * orc.u(dtype)), dtype, name, 2 * count + 64)
        if dtype == torch.bfloat16 and t.numel() >= 100:
            one = float((value.to(dtype).double() - value).norm())
            err = float((t.double() - value).norm())
            assert err <= 1.1 * one, f"{name}: {err / one:.3f} times its rounding's error"
