"""Sizes that the sequence kernels would walk past an int, and a wrong eps, are refused (no GPU)."""
import pytest

import test_seq_abi_cpu as abi
from test_seq_abi_cpu import INVALID, lib  # noqa: F401 (a fixture)

NEAR = (1 << 31) - 65535  # one above the most


def test_rows_near_2_31(lib):  # noqa: F811
    assert abi._norm(lib, C=NEAR) == INVALID and abi._norm_bwd(lib, C=NEAR) == INVALID
    assert lib.ddpm_layer_norm_bwd_workspace(1, NEAR, abi.F32) == 0
    assert lib.ddpm_layer_norm_bwd_workspace(1, NEAR - 1, abi.F32) > 0
    for kw in (dict(L=NEAR), dict(D=NEAR)):
        assert abi._conv(lib, **kw) == INVALID and abi._conv_bwd(lib, **kw) == INVALID, kw
    assert abi._conv_step(lib, D=NEAR) == INVALID


def test_scan_near_2_31(lib):  # noqa: F811
    # the padded rows of a state count four elements for N = 1
    for kw in (dict(P=1 << 29, N=1), dict(heads=1 << 16, P=1 << 15, N=1), dict(heads=1 << 24, groups=1 << 24, P=1, N=128)):
        for call in (abi._scan, abi._scan_bwd, abi._scan_step):
            assert call(lib, **kw) == INVALID, (call.__name__, kw)


@pytest.mark.parametrize("eps", [-1e-5, float("nan"), -float("inf")])
def test_eps(lib, eps):  # noqa: F811
    A = abi.A
    assert lib.ddpm_layer_norm_fwd(A[0], A[1], A[2], A[3], None, None, 4, 8, 8, eps, abi.F32, None) == INVALID


def test_steps_without_slots(lib):  # noqa: F811
    """Without slots sequence b's state is the b-th: there must be as many (the struct's and the call's batch is 2)."""
    for call in (abi._conv_step, abi._scan_step):
        name = "n" if call is abi._conv_step else "slots"
        assert call(lib, S=1, **{name: None}) == INVALID, call.__name__


@pytest.mark.parametrize("dtype,Q", [(abi.F32, 64), (abi.BF16, 128)])
def test_workspace_with_segments(lib, dtype, Q):  # noqa: F811
    """Long calls hold one float32 state a chunk and head whether they keep it or not, and two numbers a chunk and head."""
    batch, L, H, P, N = 4, 4096, 32, 64, 128
    nc = L // Q
    kept = batch * H * nc * (3 * Q + 1 + P * N)
    got = lib.ddpm_selective_scan_fwd_workspace(abi._struct(batch=batch, L=L, heads=H, P=P, groups=1, N=N, dtype=dtype)) // 4
    assert kept <= got <= kept + 2 * batch * H * nc + 6 * 64
