"""C-ABI checks of the feed-forward operators that need no GPU: exports, refusals, workspace sizes;
the modules' host logic.

Every refused call fails validation, so nothing reaches the HIP runtime.
"""
import ctypes
import os
import re

import pytest
import torch

import dynamic_dilated_depthwise_amd as ddpm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = -1, -2
F32, BF16 = 0, 1
NONE, RELU, SILU, GELU = range(4)
# well-aligned addresses far apart, never dereferenced
A = [(k + 1) << 40 for k in range(24)]

_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
SIGNATURES = {
    "ddpm_linear_fwd": [_P] * 7 + [_I64] * 5 + [_I, _I, _P],
    "ddpm_linear_bwd": [_P] * 8 + [_I64] * 5 + [_I, _I, _P],
    "ddpm_gated_linear_fwd": [_P] * 6 + [_I64] * 4 + [_I, _I, _P],
    "ddpm_gated_linear_bwd": [_P] * 8 + [_I64] * 5 + [_I, _I, _P],
    "ddpm_linear_saved": [_I64] * 3 + [_I, _I],
    "ddpm_gated_linear_saved": [_I64] * 3 + [_I],
    "ddpm_linear_fwd_workspace": [_I64] * 3 + [_I],
    "ddpm_linear_bwd_workspace": [_I64] * 3 + [_I, _I],
    "ddpm_gated_linear_fwd_workspace": [_I64] * 3 + [_I],
    "ddpm_gated_linear_bwd_workspace": [_I64] * 3 + [_I],
}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ddpm.library_path()):
        from dynamic_dilated_depthwise_amd import build
        build.build(verbose=False)
    lib = ctypes.CDLL(ddpm.library_path())  # its own handle: declarations of this file only
    for name, args in SIGNATURES.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = _I64 if name.endswith(("_workspace", "_saved")) else _I
    return lib


def test_exports_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ddpm_ff.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ddpm_[a-z_]+)\s*\(", text)))
    assert names == sorted(SIGNATURES)


# sizes whose calls need a workspace (a long contraction, few tiles)
SIZE = dict(rows=200, C=8192, N=64)


def _linear(lib, x=A[0], w=A[1], b=A[2], r=A[3], y=A[4], s=A[5], ws=A[6], rows=200, C=8192, N=64, xr=8192, rr=64, act=SILU, dt=F32):
    return lib.ddpm_linear_fwd(x, w, b, r, y, s, ws, rows, C, N, xr, rr, act, dt, None)


def _linear_bwd(lib, g=A[0], x=A[1], w=A[2], s=A[3], gx=A[4], gw=A[5], gb=A[6], ws=A[7], rows=200, C=8192, N=64, xr=8192, gr=64,
                act=SILU, dt=F32):
    return lib.ddpm_linear_bwd(g, x, w, s, gx, gw, gb, ws, rows, C, N, xr, gr, act, dt, None)


def _gated(lib, x=A[0], w=A[1], b=A[2], y=A[4], s=A[5], ws=A[6], rows=200, C=8192, N=64, xr=8192, act=SILU, dt=F32):
    return lib.ddpm_gated_linear_fwd(x, w, b, y, s, ws, rows, C, N, xr, act, dt, None)


def _gated_bwd(lib, g=A[0], x=A[1], w=A[2], s=A[3], gx=A[4], gw=A[5], gb=A[6], ws=A[7], rows=200, C=8192, N=64, xr=8192, gr=64,
               act=SILU, dt=F32):
    return lib.ddpm_gated_linear_bwd(g, x, w, s, gx, gw, gb, ws, rows, C, N, xr, gr, act, dt, None)


CALLS = (_linear, _linear_bwd, _gated, _gated_bwd)


@pytest.mark.parametrize("call,required,optional", [
    (_linear, "x w y ws", "b r s"), (_linear_bwd, "g x w s ws", "gx gw gb"), (_gated, "x w y ws", "b s"),
    (_gated_bwd, "g x w s ws", "gx gw gb")])
def test_null_and_misaligned_pointers(lib, call, required, optional):
    for name in required.split():
        assert call(lib, **{name: 0}) == INVALID, name
    for name in (required + " " + optional).split():
        assert call(lib, **{name: (9 << 50) + 2}) == INVALID, name  # float32 needs 4 bytes, workspaces 16
    if "gw" in optional:  # both or neither
        assert call(lib, gw=0) == INVALID and call(lib, gb=0) == INVALID


def test_sizes(lib):
    for call in CALLS:
        for kw in (dict(rows=0), dict(C=0), dict(N=0), dict(rows=-1), dict(rows=1 << 31), dict(C=1 << 31), dict(N=1 << 31),
                   dict(rows=1 << 30, C=1 << 30), dict(C=1 << 30, N=1 << 30), dict(xr=-1), dict(act=4), dict(act=-1), dict(dt=2),
                   dict(dt=-1)):
            assert call(lib, **kw) == INVALID, (call.__name__, kw)
    assert _linear(lib, rr=-1) == INVALID and _linear_bwd(lib, gr=-1) == INVALID and _gated_bwd(lib, gr=-1) == INVALID


def test_overlapping_outputs(lib):
    assert _linear(lib, y=A[0] + 16) == INVALID and _linear(lib, y=A[3]) == INVALID and _linear(lib, s=A[4]) == INVALID
    assert _linear(lib, ws=A[4]) == INVALID and _gated(lib, y=A[1]) == INVALID and _gated(lib, s=A[4] + 4) == INVALID
    for call in (_linear_bwd, _gated_bwd):
        assert call(lib, gx=A[1]) == INVALID and call(lib, gw=A[2]) == INVALID and call(lib, gb=A[5] + 4) == INVALID
        assert call(lib, ws=A[3]) == INVALID and call(lib, ws=A[4]) == INVALID


def test_workspace_sizes(lib):
    for dt, size in ((F32, 4), (BF16, 2)):
        # few tiles and a long contraction: float32 sums of several splits
        assert lib.ddpm_linear_fwd_workspace(200, 8192, 64, dt) >= 2 * 4 * 200 * 64
        assert lib.ddpm_gated_linear_fwd_workspace(200, 8192, 64, dt) >= 2 * 4 * 200 * 128
        # the gradient of the activation's input, where it is not grad
        assert lib.ddpm_linear_bwd_workspace(5, 8, 16, SILU, dt) >= 5 * 16 * size
        assert lib.ddpm_linear_bwd_workspace(5, 8, 16, NONE, dt) == 0
        assert lib.ddpm_gated_linear_bwd_workspace(5, 8, 16, dt) >= 5 * 32 * size
        assert lib.ddpm_linear_fwd_workspace(5, 8, 16, dt) == 0
    assert lib.ddpm_linear_fwd_workspace(0, 8, 16, F32) == 0 and lib.ddpm_linear_fwd_workspace(5, 8, 16, 7) == 0
    assert lib.ddpm_linear_bwd_workspace(5, 8, 16, 9, F32) == 0 and lib.ddpm_gated_linear_bwd_workspace(5, -8, 16, F32) == 0


def test_saved_sizes(lib):
    for dt, again in ((F32, 64), (BF16, 256)):
        # few columns of x and many rows: the bias, otherwise z
        rows = 1 << 20
        assert lib.ddpm_linear_saved(rows, again, 40, GELU, dt) == 40 and lib.ddpm_gated_linear_saved(rows, again, 40, dt) == 80
        assert lib.ddpm_linear_saved(3, 64, 256, GELU, dt) == 256 and lib.ddpm_gated_linear_saved(3, 64, 128, dt) == 256
        for r, C, N in ((100, again, 400), (rows, 4096, 40)):
            assert lib.ddpm_linear_saved(r, C, N, GELU, dt) == N * r and lib.ddpm_gated_linear_saved(r, C, N, dt) == 2 * N * r
        assert lib.ddpm_linear_saved(rows, again, 40, NONE, dt) == 0 and lib.ddpm_linear_saved(100, 4096, 40, NONE, dt) == 0
    assert lib.ddpm_linear_saved(0, 8, 8, SILU, F32) == 0 and lib.ddpm_gated_linear_saved(8, 8, 8, 5) == 0


def test_binding_rejects_host_tensors(lib):
    from dynamic_dilated_depthwise_amd import feedforward as ff
    x, w = torch.zeros(2, 8), torch.zeros(4, 8)
    for call in (lambda: ff.linear_fwd(x, w), lambda: ff.linear(x, w), lambda: ff.gated_linear(x, w),
                 lambda: ff.linear_bwd(x[:, :4], x, w), lambda: ff.gated_linear_bwd(x[:, :2], x, w, x[:, :4])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ff.linear_fwd([1.0], w)


# ------------------------------------------------------------------------------- modules
def test_module_refusals():
    from dynamic_dilated_depthwise_amd.mixer import PixelBlock, PixelFeedForward
    for kw in (dict(activation="tanh"), dict(dim=0), dict(hidden=0)):
        with pytest.raises(ValueError):
            PixelFeedForward(**kw)
    with pytest.raises(ValueError):
        PixelBlock(dim=24, hidden=40, heads=3, groups=2)
    m = PixelFeedForward(dim=24, hidden=40, bias=False)
    assert m.up_weight.shape == (80, 24) and m.down_weight.shape == (24, 40) and m.up_bias is None and m.down_bias is None
    for call in (lambda: m(torch.zeros(1, 23, 4, 4)), lambda: m.tokens(torch.zeros(5, 23)), lambda: m.tokens(torch.zeros(5, 24)),
                 lambda: m.tokens(torch.zeros(5, 24), torch.zeros(5, dtype=torch.int32)),
                 lambda: m.tokens(torch.zeros(2, 5, 24), torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
    line, h = PixelBlock(dim=24, hidden=40, heads=4, head_dim=20, state_dim=18).new_state(5)
    assert line.shape[0] == 5 and h.shape == (5, 4, 20, 18)
