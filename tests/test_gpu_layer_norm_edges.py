"""Layer norm on the GPU where its arithmetic is under strain: rows of extreme spread, constant rows,
large means, strided rows, and gradients summed over many rows.

Tolerances, in units of 2^-24 on the magnitude sum M of a value's terms.  A sum over a row passes
d = 28 + D / 1024 additions at most (16 elements of a thread, or D / 1024 of the widest form, then the
lanes and the warps).  In first order
    mean   d + 4
    rstd   (d + 4) / 2 + 4: the variance's sum, halved by the root, and the root
    n      mean and rstd together: 2 d + 8
    y      n, and two roundings: 2 d + 12
    dx     rstd, n twice, a sum and a few products: 6 d + 32
    dw     n, and the depth of the sum over the rows: R / 64 of a thread, 16 rows of a
           block, 156 blocks of a column: 2 d + 12 + min(R, R / 64 + 172)
    db     that depth
and half a step of the output's type.  An error that is common to a whole column would pass the bounds of dw and
db at many rows, so they are held to 1e-5 in the norm as well: independent roundings add like a random walk.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn
from oracle import layer_ops as ops
from test_gpu_layer_ops import TYPES, close, make

pytestmark = pytest.mark.gpu


def depth(D):
    return 28 + D // 1024


def rows_of(form, t, R, D):
    """An uninitialised [R, D] whose rows are dense, or one element off within wider ones."""
    if form == "dense":
        return torch.empty(R, D, dtype=t, device="cuda")
    return torch.empty(R, D + 9, dtype=t, device="cuda")[:, 1:1 + D]


def fill(view, values):
    view.copy_(values)
    return view, view.double().cpu().numpy()


def check(x, x64, w, w64, dy, dy64, eps, b=None, b64=None):
    R, D = x64.shape
    d = depth(D)
    y, mean, rstd = gdn.gdn_layer_norm_forward(x, w, bias=b, eps=eps)
    wy, wm, wr = ops.layer_norm(x64, w64, b64, eps)
    My, Mx, Mw, Mb = ops.layer_norm_bounds(x64, w64, dy64, eps)
    close("mean", mean, wm, np.abs(x64).mean(1), d + 4)
    close("rstd", rstd, wr, wr, (d + 4) / 2 + 4)
    close("y", y, wy, My + (0 if b64 is None else np.abs(b64)), 2 * d + 12)
    dx, dw, db = gdn.gdn_layer_norm_backward(x, w, dy, mean, rstd)
    wx, ww, wb = ops.layer_norm_backward(x64, w64, dy64, eps)
    K = min(R, R // 64 + 172)
    close("dx", dx, wx, Mx, 6 * d + 32)
    close("dw", dw, ww, Mw, 2 * d + 12 + K)
    close("db", db, wb, Mb, K)
    for name, got, want in (("dw", dw, ww), ("db", db, wb)):
        err = np.linalg.norm(got.double().cpu().numpy() - want)
        assert err <= 1e-5 * np.linalg.norm(want), (name, err / np.linalg.norm(want))


# columns and rows of the forms: vectors, shifted vectors, single elements, wider than the registers
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form,D", [("dense", 64), ("dense", 1024), ("dense", 1003), ("off", 1003), ("off", 64),
                                    ("dense", 20001)])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_rows_of_extreme_spread(dtype, form, D, eps):
    """Rows scaled from 1e-16 to 1e16 (with eps = 1e-5, from 1): rstd is as small and as large, its cube out of range."""
    t = TYPES[dtype]
    rng = np.random.default_rng([5, D])
    scales = [1.0, 1e15, 1e16, 1e12] + ([1e-14, 1e-16, 1e-12] if eps == 0 else [])
    x = make(rng, t, len(scales), D)[0].float() * torch.tensor(scales, device="cuda")[:, None]
    x, x64 = fill(rows_of(form, t, len(scales), D), x)
    dy, dy64 = fill(rows_of(form, t, len(scales), D), make(rng, t, len(scales), D)[0])
    check(x, x64, *make(rng, t, D), dy, dy64, eps)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form,R,D", [("dense", 50000, 35), ("off", 50000, 33), ("dense", 30000, 64), ("dense", 9000, 128),
                                      ("dense", 3000, 1003), ("off", 1500, 1000), ("dense", 2000, 4098),
                                      ("dense", 1000, 2560), ("dense", 7, 16), ("off", 5, 3), ("dense", 150, 1),
                                      ("dense", 300, 12001), ("dense", 90, 20001)])
@pytest.mark.parametrize("bias", [True, False])
def test_many_rows(dtype, form, R, D, bias):
    """Blocks that walk several groups of rows, and join them: every row counts in dw and db."""
    t = TYPES[dtype]
    rng = np.random.default_rng([6, R, D])
    x, x64 = fill(rows_of(form, t, R, D), make(rng, t, R, D)[0])
    dy, dy64 = fill(rows_of(form, t, R, D), make(rng, t, R, D)[0])
    check(x, x64, *make(rng, t, D), dy, dy64, 1e-5, *(make(rng, t, D) if bias else (None, None)))


@pytest.mark.parametrize("form,R,D", [("dense", 60, 64), ("dense", 60, 1003), ("off", 60, 130), ("dense", 60, 9001)])
def test_rows_of_large_mean(form, R, D):
    """Mean 1000 and spread 1: the values and the gradients, not their shapes alone."""
    rng = np.random.default_rng([7, D])
    x, x64 = fill(rows_of(form, torch.float32, R, D), make(rng, torch.float32, R, D)[0] + 1000)
    dy, dy64 = fill(rows_of(form, torch.float32, R, D), make(rng, torch.float32, R, D)[0])
    w, w64 = make(rng, torch.float32, D)
    d, eps = depth(D), 1e-5
    y, mean, rstd = gdn.gdn_layer_norm_forward(x, w, eps=eps)
    wy, wm, _ = ops.layer_norm(x64, w64, None, eps)
    My, Mx, Mw, Mb = ops.layer_norm_bounds(x64, w64, dy64, eps)
    close("mean", mean, wm, np.abs(x64).mean(1), d + 4)
    close("y", y, wy, My, 2 * d + 12)
    got = gdn.gdn_layer_norm_backward(x, w, dy, mean, rstd)
    K = (6 * d + 32, 2 * d + 12 + R, R)
    for name, g, want, m, k in zip(("dx", "dw", "db"), got, ops.layer_norm_backward(x64, w64, dy64, eps), (Mx, Mw, Mb), K):
        close(name, g, want, m, k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form,D", [("dense", 64), ("dense", 1003), ("off", 77), ("dense", 20001)])
def test_constant_rows(dtype, form, D):
    """With eps a constant row gives y = bias; with eps = 0 it is not a number, and its neighbours are."""
    t = TYPES[dtype]
    rng = np.random.default_rng([8, D])
    x = make(rng, t, 5, D)[0]
    x[1], x[3] = 0.0, 1.5
    x, x64 = fill(rows_of(form, t, 5, D), x)
    dy, dy64 = fill(rows_of(form, t, 5, D), make(rng, t, 5, D)[0])
    (w, w64), (b, b64) = make(rng, t, D), make(rng, t, D)
    check(x, x64, w, w64, dy, dy64, 1e-5, b, b64)
    y, mean, rstd = gdn.gdn_layer_norm_forward(x, w, bias=b, eps=0.0)
    assert torch.equal(y[[1, 3]].isnan(), torch.ones_like(y[[1, 3]], dtype=torch.bool)) and torch.isinf(rstd[[1, 3]]).all()
    dx = gdn.gdn_layer_norm_backward(x, w, dy, mean, rstd)[0]
    keep = [0, 2, 4]
    wy = ops.layer_norm(x64[keep], w64, b64, 0.0)[0]
    My, Mx, _, _ = ops.layer_norm_bounds(x64[keep], w64, dy64[keep], 0.0)
    close("y", y[keep], wy, My + np.abs(b64), 2 * depth(D) + 12)
    close("dx", dx[keep], ops.layer_norm_backward(x64[keep], w64, dy64[keep], 0.0)[0], Mx, 6 * depth(D) + 32)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_gradients_per_head(dtype):
    """[tokens, heads, d]: the values of dx, and dw and db summed over tokens and heads."""
    t = TYPES[dtype]
    rng = np.random.default_rng(9)
    (x, x64), (dy, dy64), (w, w64) = make(rng, t, 50, 6, 32), make(rng, t, 50, 6, 32), make(rng, t, 32)
    _, mean, rstd = gdn.gdn_layer_norm_forward(x, w)
    got = gdn.gdn_layer_norm_backward(x, w, dy, mean, rstd)
    assert got[0].shape == x.shape
    a = (x64.reshape(300, 32), w64, dy64.reshape(300, 32))
    for name, g, want, m in zip(("dx", "dw", "db"), got, ops.layer_norm_backward(*a), ops.layer_norm_bounds(*a)[1:]):
        close(name, g.view(want.shape), want, m, 6 * 28 + 32 + (176 if name != "dx" else 0))
