"""The forms that larger calls of the sequence operators take, each checked at a size that takes it:
several heads of a group in a workgroup, long passes over the chunks, whole-vector segments, long
walks and runs of the convolution, several rows of the norm in a group.  What a call takes shows in
its workspace, which every test here compares with the form that it means to check.

Tolerances: seq_oracle.check, as for the operators' smaller calls; no chain of sums here is longer
than 512 terms.
"""
import ctypes

import pytest
import torch

import seq_oracle as orc
from dynamic_dilated_depthwise_amd import sequence as seq
from test_gpu_seq_norm_conv import DT, announce, conv_case, gen_of, norm_case, randn
from test_gpu_seq_scan import NAMES, case
from test_seq_abi_cpu import _struct, lib  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def pad64(n):
    return -(-n // 64) * 64


def scan_struct(batch, L, H, P, G, N, dt):
    return _struct(batch=batch, L=L, heads=H, P=P, groups=G, N=N, dtype=int(dt == "bf16"))


def bwd_splits(lib, batch, L, H, P, G, N, dt):  # noqa: F811
    """Workgroups that share a chunk and a group in the scan's backward."""
    Q = 128 if dt == "bf16" else 64
    nc = -(-L // Q)
    tokens = batch * H * nc * Q
    base = (pad64(batch * H * nc * P * (-(-N // 4) * 4)) + pad64(6 * H * batch * nc) + 3 * pad64(2 * tokens) +
            pad64(4 * batch * H * nc * (Q // 16)))
    part = lib.ddpm_selective_scan_bwd_workspace(ctypes.byref(scan_struct(batch, L, H, P, G, N, dt))) // 4 - base
    if part == 0:
        return 1
    splits = part // (2 * batch * L * G * N)
    assert part == pad64(2 * splits * batch * L * G * N)
    return splits


def segments(lib, batch, L, H, P, G, N, dt):  # noqa: F811
    """Segments of a sequence in a call that keeps nothing, 0 without."""
    Q = 128 if dt == "bf16" else 64
    nc = -(-L // Q)
    kept = 3 * pad64(batch * H * nc * Q) + pad64(batch * H * nc) + pad64(batch * H * nc * P * (-(-N // 4) * 4))
    more = lib.ddpm_selective_scan_fwd_workspace(ctypes.byref(scan_struct(batch, L, H, P, G, N, dt))) // 4 - kept
    if more == 0:
        return 0
    for n in range(1, nc):
        if more == pad64(batch * H * nc) + pad64(batch * H * n):
            return n
    raise AssertionError("the workspace's layout is not the one that is meant")


def close(got, want, size):
    for name, g in got.items():
        orc.check(g, want[name], size[name], g.dtype, name)


def some_lengths(batch, L, seed=3):
    n = torch.randint(0, L + 1, (batch,), generator=gen_of(seed), dtype=torch.int32)
    n[0], n[-1] = L, 0
    return n.cuda()


# (batch, L, H, P, G, N) and the workgroups a group takes in each type: fewer than its heads
HEADS = [((64, 130, 8, 8, 2, 8), {"bf16": 1, "f32": 2}), ((32, 130, 8, 16, 1, 40), {"bf16": 4, "f32": 2}),
         ((64, 130, 8, 9, 2, 12), {"bf16": 1, "f32": 2}), ((128, 20, 8, 8, 2, 100), {"bf16": 1, "f32": 1}),
         ((128, 10, 4, 72, 2, 20), {"bf16": 1, "f32": 1}), ((128, 10, 4, 70, 2, 90), {"bf16": 1, "f32": 1}),
         ((20, 40, 24, 8, 2, 50), {"bf16": 6, "f32": 6})]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("sizes,splits", HEADS)
def test_heads_of_a_workgroup(lib, sizes, splits, dt):  # noqa: F811
    announce("scan heads", sizes, dt)
    batch, L, H, P, G, N = sizes
    assert bwd_splits(lib, *sizes, dt) == splits[dt] < H // G
    dtype = DT[dt]
    args = list(case(*sizes, dtype))
    g = gen_of(12)
    grad, init, gs = randn(g, batch, L, H, P, dtype=dtype), randn(g, batch, H, P, N), randn(g, batch, H, P, N)
    lengths = some_lengths(batch, L)
    off = torch.arange(L, device="cuda")[None] >= lengths[:, None]
    clean = [t.masked_fill(off[(...,) + (None,) * (t.dim() - 2)], 0) if k in (0, 1, 3, 4) else t for k, t in enumerate(args)]
    for k in (0, 1, 3, 4):
        args[k][off] = float("nan")
    y, last, saved = seq.selective_scan_fwd(*args, init, lengths, return_state=True, save=True)
    got = dict(zip(NAMES, seq.selective_scan_bwd(grad, *args, saved, init, lengths, gs)))
    want, size = orc.scan(*clean, init, lengths, grad.masked_fill(off[..., None, None], 0), gs)
    close({"y": y, "state": last, **got}, want, size)
    y2, last2, _ = seq.selective_scan_fwd(*args, init, lengths, return_state=True)
    close({"y": y2, "state": last2}, want, size)


# The pass over the chunks, whose states are float32 whatever the inputs' type: 16 runs with more
# states than a run keeps, and 64 with more and, in a shorter sequence, with fewer.
@pytest.mark.parametrize("chunks,lengths", [(70, [70 * 64 - 17, 33 * 64]), (260, [260 * 64 - 17, 100 * 64 + 1])])
def test_many_chunks(chunks, lengths):
    announce("scan chunks", chunks)
    L = lengths[0]
    args = case(2, L, 1, 3, 1, 5, torch.float32)
    g = gen_of(12)
    grad, init, gs = randn(g, 2, L, 1, 3), randn(g, 2, 1, 3, 5), randn(g, 2, 1, 3, 5)
    lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, last, saved = seq.selective_scan_fwd(*args, init, lengths, return_state=True, save=True)
    got = dict(zip(NAMES, seq.selective_scan_bwd(grad, *args, saved, init, lengths, gs)))
    close({"y": y, "state": last, **got}, *orc.scan(*args, init, lengths, grad, gs))


# Segments of chunks whose P and N are in whole vectors of both types, for each width of the state;
# eight chunks a segment and fewer, two heads and one at once.
SEGMENTS = [((2, 300, 256, 8, 128, 24), {"bf16": 2, "f32": 2}), ((2, 300, 256, 8, 128, 64), {"bf16": 2, "f32": 2}),
            ((2, 300, 256, 8, 128, 128), {"bf16": 2, "f32": 2}), ((1, 1100, 512, 8, 256, 16), {"bf16": 2, "f32": 3}),
            ((2, 300, 128, 16, 128, 48), {"bf16": 2, "f32": 2})]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("state", [False, True], ids=["fresh", "cached"])
@pytest.mark.parametrize("sizes,count", SEGMENTS)
def test_whole_vector_segments(lib, sizes, count, state, dt):  # noqa: F811
    announce("scan segments", sizes, state, dt)
    batch, L, H, P, G, N = sizes
    assert segments(lib, *sizes, dt) == count[dt]
    args = list(case(*sizes, DT[dt]))
    init = randn(gen_of(12), batch, H, P, N) if state else None
    lengths = torch.tensor([L, 150][:batch], dtype=torch.int32, device="cuda") if state else None
    y, last, _ = seq.selective_scan_fwd(*args, init, lengths, return_state=True)
    close({"y": y, "state": last}, *orc.scan(*args, init, lengths))


# --------------------------------------------------------------------------- convolution
def conv_oracle(x, weight, bias, initial, lengths, grad, grad_state):
    """seq_oracle.conv with its 64-bit sums on the GPU, which these sizes need."""
    leaves = [t.double().requires_grad_() for t in (x, weight, bias, initial)]
    ab = [t.detach().abs().requires_grad_() for t in leaves]
    with torch.device("cuda"):
        y, last = orc._conv(*leaves, lengths)
        us, ls = orc._conv(*ab, lengths, positive=True)
    g, gs = grad.double(), grad_state.double()
    names = ("grad_x", "grad_weight", "grad_bias", "grad_initial")
    out = dict(zip(names, torch.autograd.grad((y * g).sum() + (last * gs).sum(), leaves)))
    size = dict(zip(names, torch.autograd.grad((us * g.abs() * (1 + us.detach())).sum() + (ls * gs.abs()).sum(), ab)))
    out |= {"y": y.detach(), "state": last.detach()}
    size |= {"y": us.detach(), "state": ls.detach()}
    return {k: t.cpu() for k, t in out.items()}, {k: t.cpu() for k, t in size.items()}


def conv_splits(batch, L, D, W, run):
    nvec = -(-D // 4)
    cl = next(c for c in (8, 16, 32, 64) if c == 64 or c >= nvec)
    return -(-batch * -(-L // run) // (256 // cl))


# (batch, L, D, W), tokens of a backward walk, the types in which the forward takes eight tokens a
# thread (from 2^20 vectors of 16 bytes on)
BOTH = ("f32", "bf16")
CONV = [((3, 12001, 264, 4), 29, BOTH), ((3, 11003, 259, 4), 29, BOTH), ((2, 16300, 265, 3), 30, BOTH), ((2, 16300, 264, 2), 31, BOTH),
        ((2, 16300, 264, 7), 26, BOTH), ((2, 16300, 263, 1), 32, BOTH), ((2, 9000, 256, 4), 13, ("f32",)),
        ((2, 9001, 255, 3), 14, ("f32",)), ((2, 9000, 258, 8), 9, ("f32",)), ((1, 9000, 7, 4), 5, ())]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("sizes,run,eight", CONV)
def test_conv_walks(lib, sizes, run, eight, dt):  # noqa: F811
    announce("conv walks", sizes, dt)
    batch, L, D, W = sizes
    assert lib.ddpm_causal_conv_bwd_workspace(*sizes, int(dt == "bf16")) == conv_splits(*sizes, run) * D * (W + 1) * 4
    assert (batch * L * -(-D // (8 if dt == "bf16" else 4)) >= 1 << 20) == (dt in eight)
    x, w, b, init, grad, gs = conv_case(*sizes, DT[dt])
    lengths = torch.tensor([L, L - 7, 13][:batch], dtype=torch.int32, device="cuda")
    off = torch.arange(L, device="cuda")[None] >= lengths[:, None]
    xz, gz = x.masked_fill(off[..., None], 0), grad.masked_fill(off[..., None], 0)
    x[off], grad[off] = float("nan"), float("inf")
    i, s = (init, gs) if W > 1 else (None, None)
    y, last = seq.causal_conv_fwd(x, w, b, i, lengths, return_state=True)
    got = dict(zip(("grad_x", "grad_weight", "grad_bias", "grad_initial"), seq.causal_conv_bwd(grad, x, w, b, i, lengths, s)))
    want, size = conv_oracle(xz, w, b, init, lengths, gz, gs)
    if W == 1:
        del got["grad_initial"]
    close({"y": y, "state": last, **got}, want, size)


# ---------------------------------------------------------------------------- layer norm
# Groups of 16 lanes, a wave and a workgroup with one to eight vectors a lane in both types, and
# rows that only the long kernels hold; each with more rows than the backward has groups, the last
# turn in part.
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,C", [(16389, 40), (16390, 7), (4099, 200), (4099, 300), (4099, 1000), (2051, 2000), (1030, 3999),
                                    (1027, 8000), (1026, 16000), (130, 20001)])
def test_norm_rows_of_a_group(lib, rows, C, dt):  # noqa: F811
    announce("norm rows", rows, C, dt)
    dtype = DT[dt]
    n = -(-C // (8 if dt == "bf16" else 4))
    long = n > 2048
    per = 1 if n > 256 else 4 if n > 16 else 16
    parts = 64 if long else 512
    assert lib.ddpm_layer_norm_bwd_workspace(rows, C, int(dt == "bf16")) == min(parts, -(-rows // per)) * 2 * C * 4
    assert rows > parts * per and rows % (parts * per)
    x, w, b, grad = norm_case(rows, C, dtype)
    y, mean, rstd = seq.layer_norm_fwd(x, w, b, 1e-5, stats=True)
    got = (y, *seq.layer_norm_bwd(grad, x, w, mean, rstd))
    want, size, _ = orc.norm(x, w, b, 1e-5, grad)
    for name, g, r, s in zip(("y", "grad_x", "grad_weight", "grad_bias"), got, want, size):
        orc.check(g, r, s, dtype, name)
