"""C-ABI checks of the sequence operators that need no GPU: exports, refusals, workspace sizes.

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
# well-aligned addresses far apart, never dereferenced
A = [(k + 1) << 40 for k in range(24)]


_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


class Scan(ctypes.Structure):
    """ddpm_scan of the C header."""
    _fields_ = ([(n, _P) for n in ("x", "dt", "B", "C", "A", "D", "dt_bias", "initial_state", "lengths")] +
                [(n, _I64) for n in ("batch", "length", "x_batch", "x_token", "dt_batch", "dt_token", "B_batch", "B_token",
                                     "C_batch", "C_token")] +
                [(n, ctypes.c_int32) for n in ("heads", "P", "groups", "N", "dtype")])


_SCAN = ctypes.POINTER(Scan)
SIGNATURES = {
    "ddpm_layer_norm_fwd": [_P] * 6 + [_I64] * 3 + [ctypes.c_float, _I, _P],
    "ddpm_layer_norm_bwd": [_P] * 9 + [_I64] * 4 + [_I, _P],
    "ddpm_causal_conv_fwd": [_P] * 7 + [_I64] * 3 + [_I] + [_I64] * 2 + [_I, _P],
    "ddpm_causal_conv_bwd": [_P] * 12 + [_I64] * 3 + [_I] + [_I64] * 4 + [_I, _P],
    "ddpm_causal_conv_step": [_P] * 6 + [_I64] * 3 + [_I, _I64, _I, _P],
    "ddpm_selective_scan_fwd": [_SCAN, _P, _P, _I, _P, _P],
    "ddpm_selective_scan_bwd": [_SCAN, _P, _P, _I64, _I64] + [_P] * 11,
    "ddpm_selective_scan_step": [_SCAN, _P, _P, _I64, _P, _P],
    "ddpm_layer_norm_bwd_workspace": [_I64, _I64, _I],
    "ddpm_causal_conv_bwd_workspace": [_I64, _I64, _I64, _I, _I],
    "ddpm_selective_scan_fwd_workspace": [_SCAN],
    "ddpm_selective_scan_bwd_workspace": [_SCAN],
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
        f.restype = _I64 if name.endswith("_workspace") else _I
    return lib


def test_exports_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ddpm_seq.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ddpm_[a-z_]+)\s*\(", text)))
    assert names == sorted(SIGNATURES)
    for name in names:
        assert hasattr(lib, name), name


def _norm(lib, x=A[0], w=A[1], b=A[2], y=A[3], m=A[4], r=A[5], rows=4, C=8, row=8, dt=F32):
    return lib.ddpm_layer_norm_fwd(x, w, b, y, m, r, rows, C, row, 1e-5, dt, None)


def _norm_bwd(lib, g=A[0], x=A[1], w=A[2], m=A[3], r=A[4], gx=A[5], gw=A[6], gb=A[7], ws=A[8], rows=4, C=8, row=8, grow=8,
              dt=F32):
    return lib.ddpm_layer_norm_bwd(g, x, w, m, r, gx, gw, gb, ws, rows, C, row, grow, dt, None)


def _conv(lib, x=A[0], w=A[1], b=A[2], i=A[3], n=A[4], y=A[5], f=A[6], B=2, L=8, D=16, W=4, sb=128, st=16, dt=F32):
    return lib.ddpm_causal_conv_fwd(x, w, b, i, n, y, f, B, L, D, W, sb, st, dt, None)


def _conv_bwd(lib, g=A[0], x=A[1], w=A[2], b=A[3], i=A[4], n=A[5], gs=A[6], gx=A[7], gw=A[8], gb=A[9], gi=A[10], ws=A[11],
              B=2, L=8, D=16, W=4, sb=128, st=16, gsb=128, gst=16, dt=F32):
    return lib.ddpm_causal_conv_bwd(g, x, w, b, i, n, gs, gx, gw, gb, gi, ws, B, L, D, W, sb, st, gsb, gst, dt, None)


def _conv_step(lib, x=A[0], w=A[1], b=A[2], s=A[3], n=A[4], y=A[5], B=2, S=3, D=16, W=4, sb=16, dt=F32):
    return lib.ddpm_causal_conv_step(x, w, b, s, n, y, B, S, D, W, sb, dt, None)


def _struct(L=8, **kw):
    v = dict(x=A[0], dt=A[1], B=A[2], C=A[3], A=A[4], D=A[5], dt_bias=A[6], initial_state=A[7], lengths=A[8], batch=2,
             length=L, x_batch=8 * 8, x_token=8, dt_batch=16, dt_token=2, B_batch=64, B_token=8, C_batch=64, C_token=8,
             heads=2, P=4, groups=1, N=8, dtype=F32)
    v.update(kw)
    return Scan(**v)


def _scan(lib, y=A[10], f=A[11], ws=A[12], **kw):
    return lib.ddpm_selective_scan_fwd(_struct(**kw), y, f, 1, ws, None)


def _scan_bwd(lib, sv=A[10], g=A[11], gb=64, gt=8, gs=A[12], gx=A[13], gdt=A[14], gA=A[15], gB=A[16], gC=A[17], gD=A[18],
              gbias=A[19], gi=A[20], ws=A[21], **kw):
    return lib.ddpm_selective_scan_bwd(_struct(**kw), sv, g, gb, gt, gs, gx, gdt, gA, gB, gC, gD, gbias, gi, ws, None)


def _scan_step(lib, state=A[10], slots=A[11], S=3, y=A[12], L=1, **kw):
    return lib.ddpm_selective_scan_step(_struct(L=L, **kw), state, slots, S, y, None)


@pytest.mark.parametrize("call,names", [
    (_norm, "x w b y"), (_norm_bwd, "g x w m r gx gw gb ws"), (_conv, "x w b y"), (_conv_bwd, "g x w b gx gw gb ws"),
    (_conv_step, "x w b s y"), (_scan, "x dt B C A D dt_bias y ws"),
    (_scan_bwd, "x dt B C A D dt_bias sv g gx gdt gA gB gC gD gbias ws"), (_scan_step, "x dt B C A D dt_bias state y")])
def test_null_and_misaligned_pointers(lib, call, names):
    for name in names.split():
        assert call(lib, **{name: 0}) == INVALID, name
        assert call(lib, **{name: (9 << 50) + 2}) == INVALID, name  # float32 needs 4 bytes, workspaces 16


def test_sizes(lib):
    for kw in (dict(rows=0), dict(C=0), dict(C=1 << 31), dict(rows=-1), dict(row=-1), dict(dt=2), dict(dt=-1)):
        assert _norm(lib, **kw) == INVALID and _norm_bwd(lib, **kw) == INVALID, kw
    assert _norm(lib, m=0) == INVALID and _norm(lib, r=0) == INVALID  # both or neither
    assert _norm_bwd(lib, grow=-1) == INVALID
    for kw in (dict(B=0), dict(L=0), dict(D=0), dict(W=0), dict(L=1 << 31), dict(sb=-1), dict(st=-1), dict(dt=7)):
        assert _conv(lib, **kw) == INVALID and _conv_bwd(lib, **kw) == INVALID, kw
    assert _conv(lib, W=9) == UNSUPPORTED and _conv_bwd(lib, W=9) == UNSUPPORTED and _conv_step(lib, W=9) == UNSUPPORTED
    assert _conv(lib, W=1) == INVALID and _conv_bwd(lib, W=1) == INVALID and _conv_step(lib, W=1) == INVALID  # no state
    for kw in (dict(B=0), dict(S=0), dict(D=0), dict(sb=-1)):
        assert _conv_step(lib, **kw) == INVALID, kw
    for kw in (dict(batch=0), dict(heads=0), dict(P=0), dict(N=0), dict(groups=0), dict(heads=3, groups=2),
               dict(dtype=2), dict(x_token=-1), dict(B_batch=-1), dict(dt_token=-5), dict(C_batch=-1),
               dict(P=1 << 20, N=1 << 12), dict(heads=1 << 20, P=1 << 12),
               dict(batch=1 << 30, heads=1 << 10, P=1 << 10, N=128)):
        for call in (_scan, _scan_bwd, _scan_step):
            assert call(lib, **kw) == INVALID, (call.__name__, kw)
    for call in (_scan, _scan_bwd):
        assert call(lib, L=0) == INVALID and call(lib, L=(1 << 31) - 1) == INVALID
        assert call(lib, N=129) == UNSUPPORTED
    assert _scan_step(lib, S=0) == INVALID and _scan_step(lib, L=2) == INVALID
    assert _scan_bwd(lib, gb=-1) == INVALID and _scan_bwd(lib, gt=-1) == INVALID


def test_overlapping_outputs(lib):
    assert _norm(lib, y=A[0]) == INVALID and _norm(lib, m=A[3]) == INVALID
    assert _norm_bwd(lib, gx=A[1] + 4) == INVALID and _norm_bwd(lib, gb=A[6]) == INVALID
    assert _conv(lib, y=A[0] + 16) == INVALID and _conv(lib, f=A[3]) == INVALID
    assert _conv_bwd(lib, gx=A[0]) == INVALID and _conv_bwd(lib, gi=A[4]) == INVALID and _conv_bwd(lib, ws=A[7]) == INVALID
    assert _conv_step(lib, y=A[3]) == INVALID and _conv_step(lib, s=A[0]) == INVALID
    assert _scan(lib, y=A[0]) == INVALID and _scan(lib, f=A[7]) == INVALID and _scan(lib, ws=A[10]) == INVALID
    assert _scan_bwd(lib, ws=A[10]) == INVALID and _scan_bwd(lib, gB=A[2]) == INVALID and _scan_bwd(lib, gi=A[12]) == INVALID
    assert _scan_step(lib, y=A[0]) == INVALID and _scan_step(lib, state=A[2]) == INVALID


def test_workspace_sizes(lib):
    # bfloat16 chunks have 128 tokens, float32 chunks 64: three times and one state a chunk and head
    for dt, Q in ((F32, 64), (BF16, 128)):
        for L in (1, Q, Q + 1, 1000):
            nc = -(-L // Q)
            need = 4 * 2 * 2 * nc * (3 * Q + 4 * 8)
            got = lib.ddpm_selective_scan_fwd_workspace(_struct(L=L, dtype=dt))
            assert need <= got <= need + 4 * 4 * 64
            assert lib.ddpm_selective_scan_bwd_workspace(_struct(L=L, dtype=dt)) >= 4 * 2 * 2 * nc * 4 * 8
    assert lib.ddpm_selective_scan_fwd_workspace(_struct(batch=0)) == 0
    assert lib.ddpm_layer_norm_bwd_workspace(3, 70, F32) > 0 and lib.ddpm_layer_norm_bwd_workspace(0, 70, F32) == 0
    assert lib.ddpm_causal_conv_bwd_workspace(1, 1, 1, 4, BF16) > 0
    assert lib.ddpm_causal_conv_bwd_workspace(1, 1, 1, 9, BF16) == 0


def test_binding_rejects_host_tensors(lib):
    from dynamic_dilated_depthwise_amd import sequence as seq
    x = torch.zeros(2, 8, 16)
    with pytest.raises(ValueError):
        seq.layer_norm_fwd(x, torch.ones(16), torch.zeros(16))
    with pytest.raises(ValueError):
        seq.causal_conv_fwd(x, torch.zeros(16, 4), torch.zeros(16))
    with pytest.raises(ValueError):
        seq.causal_conv_step(x[0], torch.zeros(16, 4), torch.zeros(16), torch.zeros(8, 3, 16))
    v = torch.zeros(2)
    with pytest.raises(ValueError):
        seq.selective_scan_fwd(x.view(2, 8, 2, 8), x[..., :2], v, x[:, :, None], x[:, :, None], v, v)
    with pytest.raises(TypeError):
        seq.layer_norm_fwd([1.0], torch.ones(1), torch.zeros(1))


def test_struct_matches_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ddpm_seq.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{(.*?)\} ddpm_scan;", text, re.S).group(1)
    names = [re.sub(r"\W", "", v.split()[-1]) for line in body.split(";") if line.strip()
             for v in line.replace("*", " ").split(",")]
    assert names == [n for n, _ in Scan._fields_]
    assert ctypes.sizeof(Scan) == 9 * 8 + 10 * 8 + 5 * 4 + 4
