"""float32 products that consist of one term each, in every kernel (ff_cases.py): what is lost of an operand or of
a product of two shows, as it does not among the roundings of a long sum.

Tolerances, in roundings of float32 (u = 2^-24).  An operand is three bfloat16 terms, exactly, the second at
most 2^-8 of it and the third 2^-16; the three of nine products that are left out are at most 2.1 u of the
whole, the last addition's rounding is one u (two, if the matrix unit cuts it off) and those before it are
2^-7 of that: 5 u.  Without the third term, or without the product of two second ones, 2^-16 is missing.
A gate's gradient that is itself such a product, 1 u for each multiplication more.
"""
import pytest
import torch

import ff_oracle as orc
from dynamic_dilated_depthwise_amd import feedforward as ff
from ff_cases import CASES
from test_gpu_ff import announce, gen_of

pytestmark = pytest.mark.gpu

U = orc.u(torch.float32)
F32 = [c for c in CASES if c[0] == "f32"]


def values(gen, *shape):
    """Numbers of 24 bits between one and two, of either sign."""
    t = 1 + torch.rand(*shape, generator=gen, dtype=torch.float64)
    return (t * (torch.randint(0, 2, shape, generator=gen) * 2 - 1)).float().cuda()


def sparse(gen, rows, cols):
    """At most one number in a row and in a column, all over the matrix."""
    n = min(rows, cols)
    t = torch.zeros(rows, cols, device="cuda")
    r, c = (torch.arange(n) * rows // n).cuda(), (torch.arange(n) * cols // n)[torch.randperm(n, generator=gen)].cuda()
    t[r, c] = values(gen, n)
    return t


def near(got, want, roundings, name):
    over = (got.double() - want).abs() - roundings * U * want.abs()
    assert bool((over <= 0).all()), f"{name}: over the bound by {float((over / want.abs().clamp(min=1e-30)).max() / U):.3g} u"


def product(a, b):
    return a.double() @ b.double()


@pytest.mark.parametrize("op,act,rows,C,N", [c[1:] for c in F32 if c[1] == "linear"])
def test_linear(op, act, rows, C, N):
    announce("ff terms", op, act, rows, C, N)
    g = gen_of(rows + C + N)
    x, w, grad, one = values(g, rows, C), sparse(g, N, C), values(g, rows, N), sparse(g, rows, N)
    near(ff.linear_fwd(x, w)[0], product(x, w.t()), 5, "y")
    saved = None
    if act != "none":  # relu of what is positive: its slope is one
        act = "relu"
        saved = ff.linear_fwd(x, w, torch.full((N,), 64., device="cuda"), activation=act, save=True)[1]
    near(ff.linear_bwd(grad, x, w, saved, act, need_weight=False)[0], product(grad, w), 5, "grad_x")
    _, gw, gb = ff.linear_bwd(one, x, w, saved, act, need_x=False)
    near(gw, product(one.t(), x), 5, "grad_weight")
    assert torch.equal(gb, one.sum(0))


@pytest.mark.parametrize("half", [0, 1], ids=["gate", "other"])
@pytest.mark.parametrize("op,act,rows,C,N", [c[1:] for c in F32 if c[1] == "gated"])
def test_gated(op, act, rows, C, N, half):
    """One of the halves is one everywhere, so that y is the other one."""
    announce("ff terms", op, act, rows, C, N, half)
    g = gen_of(rows + C + N)
    x, w, grad, one = values(g, rows, C), sparse(g, N, C), values(g, rows, N), sparse(g, rows, N)
    z = product(x, w.t())
    both, bias = torch.zeros(2 * N, C, device="cuda"), torch.zeros(2 * N, device="cuda")
    this, that = slice(half * N, half * N + N), slice(N - half * N, 2 * N - half * N)
    both[this], bias[that] = w, 1
    y, saved = ff.gated_linear_fwd(x, both, bias, "none", save=True)
    near(y, z, 5, "y")
    near(ff.gated_linear_bwd(grad, x, both, saved, "none", need_weight=False)[0], product(grad, w), 5, "grad_x")
    _, gw, gb = ff.gated_linear_bwd(one, x, both, saved, "none", need_x=False)
    near(gw[this], product(one.t(), x), 5, "grad_weight")
    assert torch.equal(gb[this], one.sum(0))
    dz = one.double() * z  # of the half that is one: a product of two roundings and a term
    near(gw[that], dz.t() @ x.double(), 5 + 5 + 2 + 0.1, "grad_weight of the other half")
    near(gb[that], dz.sum(0), 5 + 2 + 0.1, "grad_bias of the other half")
