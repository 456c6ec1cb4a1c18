"""The layer operators on the GPU against their 64-bit definitions.

Tolerances.  An output in type t is off by at most half a step of t relative to its
value, plus the rounding of the fp32 evaluation: at most K units of 2^-24 on
the magnitude sum M of the value's terms, where K counts the roundings that a
term passes through.  2^x in one instruction is off by 2.5 units (measured
1.5e-7), a sigmoid by that, a division (2 units) and its argument's rounding.
    convolution  W + 1 products and sums, silu: K = W + 2 + 24 on M and on the value (a
                 sigmoid's argument |v| <= 20 is off by |v| 2^-24 relative to e^-v)
    scan         a term passes at most L decays, each 2.5 + 2 units and off by the
                 error of its exponent (counted on M with halved rates: the bound
                 covers r exp(-r) <= exp(-r/2)), then the sums over S states and
                 the channels of a group and the rows: K = 8 (L + 8) + S + Dg + 60
    layer norm   sums over D and rows: K = 2 D + R + 40
"""
import numpy as np
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn
from oracle import layer_ops as ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # eps / 2: half a step


def make(rng, dtype, *shape, scale=1.0):
    """A device tensor and the same values in 64 bits."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def close(name, got, want, M, K):
    got_t = got.dtype
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if not got.size:
        return
    tol = HALF[got_t] * np.abs(want) * (1 + 2.0 ** -7) + K * U * M + 1e-37
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (name, int(bad.sum()), np.unravel_index(np.argmax(err - tol), err.shape),
                           float((err - tol).max()), float(err.max()))


def offsets(lengths):
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return torch.from_numpy(cu).cuda(), cu


LENGTHS = {"one": [1], "short": [0, 1, 2, 0, 3, 4, 1], "ragged": [70, 0, 1, 129, 2, 33, 16],
           "long": [301]}


# ------------------------------------------------------------------ convolution
def conv_case(dtype, D, W, lengths, bias, state, seed=0, wtype=None):
    rng = np.random.default_rng([seed, D, W, len(lengths)])
    cu, cu_h = offsets(lengths)
    T, N = int(cu_h[-1]), len(lengths)
    d = dict(x=make(rng, dtype, T, D), w=make(rng, wtype or dtype, D, W, scale=W ** -0.5), dy=make(rng, dtype, T, D))
    d["b"] = make(rng, wtype or dtype, D, scale=0.3) if bias else (None, None)
    d["s"] = make(rng, dtype, N, W - 1, D) if state else (None, None)
    d["do"] = make(rng, torch.float32, N, W - 1, D) if state else (None, None)
    return d, cu, cu_h


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,W,bias,state,act", [(64, 4, True, True, True), (36, 4, True, True, True), (22, 3, True, True, True), (33, 3, False, True, True),
                                                (1, 2, True, False, False), (2056, 4, False, False, True),
                                                (130, 2, True, True, True)])
def test_conv(dtype, D, W, bias, state, act, lengths):
    t = TYPES[dtype]
    d, cu, cu_h = conv_case(t, D, W, LENGTHS[lengths], bias, state)
    y, so = gdn.gdn_conv_forward(d["x"][0], d["w"][0], cu, bias=d["b"][0], state_in=d["s"][0], silu=act)
    a = (d["x"][1], d["w"][1], cu_h, d["b"][1], d["s"][1], act)
    wy, ws, _ = ops.conv(*a)
    M = ops.conv(*a, bound=True)[2]
    K = W + 26
    close("y", y, wy, 1.1 * M + np.abs(wy), K)
    assert torch.equal(so.double().cpu(), torch.from_numpy(ws))
    g = gdn.gdn_conv_backward(d["x"][0], d["w"][0], d["dy"][0], cu, bias=d["b"][0], state_in=d["s"][0], silu=act,
                              dstate_out=d["do"][0])
    a = (d["x"][1], d["w"][1], d["dy"][1], cu_h, d["b"][1], d["s"][1], act, d["do"][1])
    want, M = ops.conv_backward(*a), ops.conv_backward(*a, bound=True)
    K = 2 * W + 60 + len(wy)
    for name, got, w, m in zip(("dx", "dw", "db", "dstate"), g, want, M):
        if got is not None:
            close(name, got, w, m, K)
    assert (g[2] is None) == (not bias)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,D,W,bias,act", [(1, 1, 2, False, True), (3, 64, 4, True, True), (65, 33, 3, True, False),
                                            (5, 2056, 4, False, True)])
def test_conv_step(dtype, N, D, W, bias, act):
    t = TYPES[dtype]
    rng = np.random.default_rng([N, D])
    x, x64 = make(rng, t, N, D)
    w, w64 = make(rng, t, D, W)
    s, s64 = make(rng, t, N, W - 1, D)
    b, b64 = make(rng, t, D) if bias else (None, None)
    apart = torch.empty_like(s)
    y2 = gdn.gdn_conv_step(x, w, s, bias=b, silu=act, state_out=apart)
    y = gdn.gdn_conv_step(x, w, s, bias=b, silu=act)
    cu = np.arange(N + 1)
    wy, ws, _ = ops.conv(x64, w64, cu, b64, s64, act)
    close("y", y, wy, 1.1 * ops.conv(x64, w64, cu, b64, s64, act, True)[2] + np.abs(wy), W + 26)
    assert torch.equal(s.double().cpu(), torch.from_numpy(ws)) and torch.equal(apart, s) and torch.equal(y, y2)


def test_conv_weight_types_mix():
    d, cu, cu_h = conv_case(torch.bfloat16, 40, 4, [9, 20], True, True, wtype=torch.float32)
    y, _ = gdn.gdn_conv_forward(d["x"][0], d["w"][0], cu, bias=d["b"][0], state_in=d["s"][0])
    a = (d["x"][1], d["w"][1], cu_h, d["b"][1], d["s"][1], True)
    close("y", y, ops.conv(*a)[0], 1.1 * ops.conv(*a, bound=True)[2] + np.abs(ops.conv(*a)[0]), 30)


# ------------------------------------------------------------------------- scan
def ssm_case(dtype, D, G, S, lengths, z=True, skip=True, bias=True, state=True, soft=True, seed=0):
    rng = np.random.default_rng([seed, D, G, S, len(lengths)])
    cu, cu_h = offsets(lengths)
    T, N, f32 = int(cu_h[-1]), len(lengths), torch.float32
    c = dict(x=make(rng, dtype, T, D), dt=make(rng, dtype, T, D, scale=0.5), B=make(rng, dtype, T, G, S),
             C=make(rng, dtype, T, G, S))
    A = -(np.arange(1, S + 1) * np.exp(0.1 * rng.standard_normal((D, S)))).astype(np.float32)
    c["A"] = (torch.from_numpy(A).cuda(), A.astype(np.float64))
    c["z"] = make(rng, dtype, T, D) if z else (None, None)
    c["D"] = make(rng, f32, D) if skip else (None, None)
    c["dt_bias"] = (None, None)
    if not soft:
        c["dt"] = (c["dt"][0].abs() * 0.1, None)
        c["dt"] = (c["dt"][0], c["dt"][0].double().cpu().numpy())
    if bias:
        width = np.exp(rng.uniform(np.log(1e-3), np.log(0.3), D))
        b = (width + np.log(-np.expm1(-width))).astype(np.float32) if soft else width.astype(np.float32)
        c["dt_bias"] = (torch.from_numpy(b).cuda(), b.astype(np.float64))
    c["state_in"] = make(rng, f32, N, D, S) if state else (None, None)
    g = {k: v[0] for k, v in c.items()}
    h = {k: v[1] for k, v in c.items()}
    h["dt_softplus"] = soft
    return g, h, make(rng, dtype, T, D), make(rng, f32, N, D, S) if state else (None, None), cu, cu_h


def ssm_run(g, cu, soft=True, **kw):
    opt = {k: g[k] for k in ("D", "z", "dt_bias", "state_in")}
    return gdn.gdn_ssm_forward(g["x"], g["dt"], g["A"], g["B"], g["C"], cu, dt_softplus=soft, **opt, **kw)


def ssm_grads(g, dy, states, cu, do, soft=True, **kw):
    opt = {k: g[k] for k in ("D", "z", "dt_bias")}
    return gdn.gdn_ssm_backward(g["x"], g["dt"], g["A"], g["B"], g["C"], dy, states, cu, dt_softplus=soft,
                                dstate_out=do, **opt, **kw)


SSM_GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate_in")


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,G,S,full,soft", [(128, 1, 16, True, True), (70, 2, 16, True, True), (1, 1, 16, False, True),
                                             (96, 3, 32, True, False), (40, 1, 32, False, True),
                                             (48, 2, 64, True, True), (33, 1, 64, True, True)])
def test_ssm(dtype, D, G, S, full, soft, lengths):
    g, h, dy, do, cu, cu_h = ssm_case(TYPES[dtype], D, G, S, LENGTHS[lengths], z=full, skip=full, bias=full,
                                      state=full, soft=soft)
    y, last, states = ssm_run(g, cu, soft, save_states=True)
    wy, wl, _ = ops.ssm(h, cu_h)
    My, Ml, _ = ops.ssm(h, cu_h, bound=True)
    K = 8 * (max(LENGTHS[lengths]) + 8) + S + D // G + 60
    close("y", y, wy, My, K)
    close("state_out", last, wl, Ml, K)
    got = ssm_grads(g, dy[0], states, cu, do[0], soft)
    want, M = ops.ssm_backward(h, dy[1], cu_h, do[1]), ops.ssm_backward(h, dy[1], cu_h, do[1], bound=True)
    K += len(wy)
    for name, t in zip(SSM_GRADS, got):
        if t is not None:
            close(name, t, want[name], M[name], K)
    assert (got[5] is None) == (not full) and (got[6] is None) == (not full) and (got[7] is None) == (not full)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,D,G,S,full", [(1, 1, 1, 16, True), (5, 70, 2, 16, False), (3, 96, 3, 32, True),
                                          (33, 40, 1, 64, True)])
def test_ssm_step(dtype, N, D, G, S, full):
    g, h, _, _, _, _ = ssm_case(TYPES[dtype], D, G, S, [1] * N, z=full, skip=full, bias=full)
    wy, wl, _ = ops.ssm(h, np.arange(N + 1))
    My, Ml, _ = ops.ssm(h, np.arange(N + 1), bound=True)
    opt = {k: g[k] for k in ("D", "z", "dt_bias")}
    apart = torch.empty_like(g["state_in"])
    y2 = gdn.gdn_ssm_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["state_in"], state_out=apart, **opt)
    y = gdn.gdn_ssm_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["state_in"], **opt)
    close("y", y, wy, My, 72 + S)
    close("state", g["state_in"], wl, Ml, 72 + S)
    assert torch.equal(apart, g["state_in"]) and torch.equal(y, y2)


def test_ssm_long_sequences_are_cut_into_chunks():
    # 64 channels over 3000 tokens: many chunks; slow and fast decays, a state in and out
    g, h, dy, do, cu, cu_h = ssm_case(torch.float32, 64, 1, 16, [2500, 0, 517])
    y, last, states = ssm_run(g, cu, save_states=True)
    wy, wl, _ = ops.ssm(h, cu_h)
    My, Ml, _ = ops.ssm(h, cu_h, bound=True)
    K = 8 * 2508 + 140
    close("y", y, wy, My, K)
    close("state_out", last, wl, Ml, K)
    # and much closer than that bound on the whole: independent roundings add like a random walk
    assert np.linalg.norm(y.double().cpu().numpy() - wy) <= 1e-5 * np.linalg.norm(wy)
    got = ssm_grads(g, dy[0], states, cu, do[0])
    want, M = ops.ssm_backward(h, dy[1], cu_h, do[1]), ops.ssm_backward(h, dy[1], cu_h, do[1], bound=True)
    for name, t in zip(SSM_GRADS, got):
        close(name, t, want[name], M[name], K + len(wy))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,S", [(2400, 16), (2401, 16), (2400, 32), (2400, 64)])
def test_ssm_many_channels(dtype, D, S):
    # enough channels for the short tiles of the forward
    lengths = [40, 0, 1, 65, 130, 2, 70]
    g, h, _, _, cu, cu_h = ssm_case(TYPES[dtype], D, 1, S, lengths)
    y, last, _ = ssm_run(g, cu)
    wy, wl, _ = ops.ssm(h, cu_h)
    My, Ml, _ = ops.ssm(h, cu_h, bound=True)
    K = 8 * 138 + S + D + 60
    close("y", y, wy, My, K)
    close("state_out", last, wl, Ml, K)


def test_ssm_zero_and_extreme_steps():
    # steps of exactly 0 (softplus of a very negative input) keep the state; very long ones forget it
    g, h, dy, do, cu, cu_h = ssm_case(torch.float32, 32, 1, 16, [40, 40], bias=False)
    dt = h["dt"].copy()
    dt[:, ::2] = -200.0
    dt[5, 1::2] = 90.0
    g["dt"] = torch.from_numpy(dt.astype(np.float32)).cuda()
    h["dt"] = dt.astype(np.float32).astype(np.float64)
    y, last, states = ssm_run(g, cu, save_states=True)
    wy, wl, _ = ops.ssm(h, cu_h)
    My, Ml, _ = ops.ssm(h, cu_h, bound=True)
    close("y", y, wy, My, 8 * 48 + 110)
    close("state_out", last, wl, Ml, 8 * 48 + 110)
    assert torch.equal(last[:, ::2], g["state_in"][:, ::2])
    for t in ssm_grads(g, dy[0], states, cu, do[0]):
        assert t is None or torch.isfinite(t).all()


# ------------------------------------------------------------------- layer norm
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,D", [(1, 1), (7, 16), (300, 33), (64, 128), (9, 1000), (5, 1003), (3, 4096), (2, 16384),
                                 (2, 20001), (1025, 64), (700, 2048), (4, 6000), (3, 8200), (2, 3001), (2, 9001),
                                 (50000, 35), (3000, 1003), (2000, 4098)])
@pytest.mark.parametrize("bias", [True, False])
def test_layer_norm(dtype, R, D, bias):
    t = TYPES[dtype]
    rng = np.random.default_rng([R, D])
    x, x64 = make(rng, t, R, D)
    w, w64 = make(rng, t, D)
    b, b64 = make(rng, t, D) if bias else (None, None)
    dy, dy64 = make(rng, t, R, D)
    y, mean, rstd = gdn.gdn_layer_norm_forward(x, w, bias=b)
    wy, wm, wr = ops.layer_norm(x64, w64, b64)
    K = 2 * D + R + 40
    My, Mx, Mw, Mb = ops.layer_norm_bounds(x64, w64, dy64)
    close("y", y, wy, My + (np.abs(b64) if bias else 0), K)
    close("mean", mean, wm, np.abs(x64).mean(1), K)
    close("rstd", rstd, wr, wr, K)
    got = gdn.gdn_layer_norm_backward(x, w, dy, mean, rstd)
    for name, g, want, m in zip(("dx", "dw", "db"), got, ops.layer_norm_backward(x64, w64, dy64), (Mx, Mw, Mb)):
        close(name, g, want, m, K)


def test_layer_norm_of_heads_and_of_a_shifted_row():
    rng = np.random.default_rng(3)
    x, x64 = make(rng, torch.float32, 5, 6, 64)
    x, x64 = x + 1000, x64 + 0.0
    x64 = x.double().cpu().numpy()
    w, w64 = make(rng, torch.float32, 64)
    y, mean, rstd = gdn.gdn_layer_norm_forward(x, w)
    assert y.shape == x.shape and mean.shape == (5, 6)
    flat = x64.reshape(30, 64)
    wy, _, _ = ops.layer_norm(flat, w64)
    close("y", y.view(30, 64), wy, ops.layer_norm_bounds(flat, w64), 2 * 64 + 70)
    dx, dw, db = gdn.gdn_layer_norm_backward(x, w, torch.ones_like(x), mean, rstd)
    assert dx.shape == x.shape and dw.shape == db.shape == (64,)


# ------------------------------------------------------- what a program does with them
def test_strided_rows_and_unaligned_slices_give_the_same():
    """Slices of one wide projection: whole vectors apart, and one element off."""
    rng = np.random.default_rng(11)
    T, D, S = 50, 64, 16
    for off in (0, 1):
        wide, _ = make(rng, torch.bfloat16, T, off + 3 * D + 2 * S + 8)
        x, dt, z = (wide[:, off + i * D:off + (i + 1) * D] for i in range(3))
        B = wide[:, off + 3 * D:off + 3 * D + S].unflatten(1, (1, S))
        C = wide[:, off + 3 * D + S:off + 3 * D + 2 * S].unflatten(1, (1, S))
        w, _ = make(rng, torch.bfloat16, D, 4)
        A = -torch.rand(D, S, device="cuda") - 0.1
        own = [t.contiguous() for t in (x, dt, z, B, C)]
        y, s = gdn.gdn_conv_forward(x, w)
        y2, s2 = gdn.gdn_conv_forward(own[0], w)
        assert torch.equal(y, y2) and torch.equal(s, s2)
        one, two = gdn.gdn_conv_backward(x, w, z), gdn.gdn_conv_backward(own[0], w, own[2])
        assert torch.equal(one[0], two[0]) and torch.equal(one[3], two[3])
        # the same T terms of at most 16, summed in another order where the accesses are narrower
        assert (one[1] - two[1]).abs().max() <= 2 * T * U * T * 16
        f = lambda x, dt, z, B, C: gdn.gdn_ssm_forward(x, dt, A, B, C, z=z, save_states=True)  # noqa: E731
        one, two = f(x, dt, z, B, C), f(*own)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        st = two[2]
        for a, b in zip(gdn.gdn_ssm_backward(x, dt, A, B, C, dt, st, z=z),
                        gdn.gdn_ssm_backward(own[0], own[1], A, own[3], own[4], own[1], st, z=own[2])):
            assert a is None or torch.equal(a, b)
        n1, n2 = gdn.gdn_layer_norm_forward(x, w[:, 0].contiguous()), gdn.gdn_layer_norm_forward(
            own[0], w[:, 0].contiguous())
        for a, b in zip(n1, n2):  # sums over D in another order, then one rounding to bf16
            assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 4 * D * U).all()


def test_offsets_beyond_32_bits():
    """2.3e9 elements a tensor, zero but for the last rows: those give what they give alone."""
    T, D, S, n = 70000, 32768, 16, 64
    rng = np.random.default_rng(31)
    tail, _ = make(rng, torch.bfloat16, n, D)
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    x[T - n:] = tail
    w, _ = make(rng, torch.bfloat16, D, 4)
    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    y, _ = gdn.gdn_conv_forward(x, w, cu)
    assert torch.equal(y[T - n:], gdn.gdn_conv_forward(tail, w, one)[0])
    dx = gdn.gdn_conv_backward(x, w, x, cu)[0]
    assert torch.equal(dx[T - n:], gdn.gdn_conv_backward(tail, w, tail, one)[0])
    del dx
    y, mean, rstd = gdn.gdn_layer_norm_forward(x, w[:, 0].contiguous())
    assert torch.equal(y[T - n:], gdn.gdn_layer_norm_forward(tail, w[:, 0].contiguous())[0])
    del y, mean, rstd
    A = -torch.rand(D, S, device="cuda") - 0.1
    B, _ = make(rng, torch.bfloat16, T, 1, S)
    y, last, _ = gdn.gdn_ssm_forward(x, x, A, B, B, cu)
    y1, last1, _ = gdn.gdn_ssm_forward(tail, tail, A, B[T - n:], B[T - n:], one)
    # N D picks the segment length; the same sums in another grouping
    assert ((y[T - n:].float() - y1.float()).abs() <= 2.0 ** -7 * y1.float().abs() + 1e-4).all()
    assert torch.allclose(last[1], last1[0], rtol=1e-4, atol=1e-5)


def test_rows_behind_the_last_sequence_stay():
    rng = np.random.default_rng(12)
    T, D, S = 90, 48, 16
    cu = torch.tensor([0, 30, 30, 71], dtype=torch.int32, device="cuda")
    x, _ = make(rng, torch.float32, T, D)
    x[71:] = float("nan")  # padding may hold anything
    w, _ = make(rng, torch.float32, D, 4)
    y = torch.full_like(x, 7.0)
    gdn.gdn_conv_forward(x, w, cu, y=y)
    assert (y[71:] == 7).all() and torch.isfinite(y[:71]).all()
    grads = (torch.full_like(x, 7.0), torch.empty(D, 4, device="cuda"), None, torch.empty(3, 3, D, device="cuda"))
    gdn.gdn_conv_backward(x, w, x, cu, grads=grads)
    assert (grads[0][71:] == 7).all() and all(torch.isfinite(t).all() for t in (grads[0], grads[1], grads[3]))
    A = -torch.rand(D, S, device="cuda") - 0.1
    B, _ = make(rng, torch.float32, T, 1, S)
    y = torch.full_like(x, 7.0)
    _, last, st = gdn.gdn_ssm_forward(x, x, A, B, B, cu, z=x, y=y, save_states=True)
    assert (y[71:] == 7).all() and torch.isfinite(y[:71]).all() and torch.isfinite(last).all()
    seven = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    g = (seven(T, D), seven(T, D), seven(D, S), seven(T, 1, S), seven(T, 1, S), None, seven(T, D), None,
         seven(3, D, S))
    gdn.gdn_ssm_backward(x, x, A, B, B, x, st, cu, z=x, grads=g)
    for i in (0, 1, 3, 4, 6):
        assert (g[i][71:] == 7).all() and torch.isfinite(g[i]).all()
    assert torch.isfinite(g[2]).all()


def test_bad_offsets_are_reported_and_stay_in_bounds():
    rng = np.random.default_rng(13)
    T, D, S = 40, 32, 16
    x, _ = make(rng, torch.float32, T, D)
    w, _ = make(rng, torch.float32, D, 3)
    A = -torch.rand(D, S, device="cuda")
    B, _ = make(rng, torch.float32, T, 1, S)
    for bad in ([0, 50], [-3, 10], [0, 30, 20, 40], [0, 2 ** 30, 40]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        st = torch.zeros(4, dtype=torch.int32, device="cuda")
        gdn.gdn_conv_forward(x, w, cu, status=st[0:1])
        gdn.gdn_conv_backward(x, w, x, cu, status=st[1:2])
        _, _, cs = gdn.gdn_ssm_forward(x, x, A, B, B, cu, save_states=True, status=st[2:3])
        gdn.gdn_ssm_backward(x, x, A, B, B, x, torch.zeros_like(cs), cu, status=st[3:4])
        assert st.tolist() == [gdn.GDN_ERR_DEVICE_INPUT] * 4, bad
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_conv_forward(x, w, torch.tensor([0, 4, 40], dtype=torch.int32, device="cuda"), status=st)
    assert st.item() == gdn.GDN_OK


def test_no_tokens_and_no_sequences():
    D, S = 24, 16
    w = torch.randn(D, 4, device="cuda")
    x = torch.empty(0, D, device="cuda")
    B = torch.empty(0, 1, S, device="cuda")
    A = -torch.rand(D, S, device="cuda")
    for N in (0, 3):
        cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
        s, h = torch.randn(N, 3, D, device="cuda"), torch.randn(N, D, S, device="cuda")
        _, so = gdn.gdn_conv_forward(x, w, cu, state_in=s)
        assert torch.equal(so, s)
        g = gdn.gdn_conv_backward(x, w, x, cu, state_in=s, dstate_out=s, bias=w[:, 0].contiguous())
        assert (g[1] == 0).all() and (g[2] == 0).all() and torch.equal(g[3], s)
        _, last, st = gdn.gdn_ssm_forward(x, x, A, B, B, cu, state_in=h, save_states=True)
        assert torch.equal(last, h)
        g = gdn.gdn_ssm_backward(x, x, A, B, B, x, st, cu, dstate_out=h)
        assert (g[2] == 0).all() and torch.equal(g[8], h)
    y, mean, rstd = gdn.gdn_layer_norm_forward(x, w[:, 0].contiguous())
    _, dw, db = gdn.gdn_layer_norm_backward(x, w[:, 0].contiguous(), x, mean, rstd)
    assert y.shape == (0, D) and (dw == 0).all() and (db == 0).all()


def test_repeats_and_batches_give_the_same_bits():
    g, _, dy, do, cu, cu_h = ssm_case(torch.bfloat16, 96, 1, 16, [60, 200, 7])
    first = ssm_run(g, cu, save_states=True)
    grads = ssm_grads(g, dy[0], first[2], cu, do[0])
    for _ in range(3):
        again = ssm_run(g, cu, save_states=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        for a, b in zip(grads, ssm_grads(g, dy[0], again[2], cu, do[0])):
            assert torch.equal(a, b)
    d, cu, _ = conv_case(torch.bfloat16, 64, 4, [60, 200, 7], True, True)
    run = lambda: gdn.gdn_conv_backward(d["x"][0], d["w"][0], d["dy"][0], cu, bias=d["b"][0])  # noqa: E731
    a = run()
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(a, run()))


def test_nan_stays_in_its_sequence_and_channel():
    g, _, _, _, cu, cu_h = ssm_case(torch.float32, 40, 1, 16, [50, 60])
    g["x"][20, 7] = float("nan")
    y, last, _ = ssm_run(g, cu)
    bad = torch.isnan(y)
    assert bad[20:50, 7].all() and bad.sum() == 30 and torch.isnan(last).sum() == 16
    d, cu, _ = conv_case(torch.float32, 40, 4, [50, 60], True, True)
    d["x"][0][20, 7] = float("inf")
    y, _ = gdn.gdn_conv_forward(d["x"][0], d["w"][0], cu, silu=False)
    assert (~torch.isfinite(y)).sum() == 4 and not torch.isfinite(y[20:24, 7]).any()
    x = torch.randn(6, 64, device="cuda")
    x[2, 3] = float("inf")
    y, _, _ = gdn.gdn_layer_norm_forward(x, torch.ones(64, device="cuda"))
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3, 4, 5]]).all()


def test_another_stream_and_captured_graphs():
    """A captured training step replays with other inputs and other lengths; two graphs hold their own
    workspaces; a call on a side stream is ordered by that stream."""
    g, h, dy, do, cu, cu_h = ssm_case(torch.float32, 64, 1, 16, [300, 200, 100])
    d, _, _ = conv_case(torch.float32, 64, 4, [300, 200, 100], True, True)
    w, b = d["w"][0], d["b"][0]

    def step():
        x, _ = gdn.gdn_conv_forward(g["x"], w, cu, bias=b)
        y, last, st = gdn.gdn_ssm_forward(x, g["dt"], g["A"], g["B"], g["C"], cu, D=g["D"], z=g["z"],
                                          dt_bias=g["dt_bias"], save_states=True)
        n, mean, rstd = gdn.gdn_layer_norm_forward(y, b)
        dn = gdn.gdn_layer_norm_backward(y, b, dy[0], mean, rstd)
        ds = gdn.gdn_ssm_backward(x, g["dt"], g["A"], g["B"], g["C"], dn[0], st, cu, D=g["D"], z=g["z"],
                                  dt_bias=g["dt_bias"])
        dc = gdn.gdn_conv_backward(g["x"], w, ds[0], cu, bias=b)
        return [t for t in (n, last, *dn, *ds, *dc) if t is not None]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(eager, o))
    cu.copy_(torch.tensor([0, 10, 10, 600], dtype=torch.int32))
    g["x"].mul_(-0.5)
    other = [t.clone() for t in step()]
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(other, o))
    assert not torch.equal(eager[0], other[0])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_mixer_layer_prefilled_and_decoded_token_by_token(dtype):
    """Norm, convolution and scan over 40 tokens at once, and over 25 with 15 steps on the cached states."""
    t = TYPES[dtype]
    rng = np.random.default_rng(21)
    N, L, D, S = 3, 40, 64, 16
    x = make(rng, t, N, L, D)[0]
    nw, nb = make(rng, t, D)[0], make(rng, t, D)[0]
    w, b = make(rng, t, D, 4)[0], make(rng, t, D)[0]
    dt, B, C = make(rng, t, N, L, D, scale=0.3)[0], make(rng, t, N, L, 1, S)[0], make(rng, t, N, L, 1, S)[0]
    A = -torch.rand(D, S, device="cuda") * 4
    Dp = torch.randn(D, device="cuda")

    def prefill(n):
        cut = lambda a: a[:, :n].reshape(N * n, *a.shape[2:])  # noqa: E731
        cu = torch.arange(N + 1, dtype=torch.int32, device="cuda") * n
        y, _, _ = gdn.gdn_layer_norm_forward(cut(x), nw, bias=nb)
        u, cs = gdn.gdn_conv_forward(y, w, cu, bias=b)
        o, hs, _ = gdn.gdn_ssm_forward(u, cut(dt), A, cut(B), cut(C), cu, D=Dp, z=y)
        return o.view(N, n, D), cs, hs

    whole, cs_w, hs_w = prefill(L)
    part, cs, hs = prefill(25)
    # the prefix does not depend on what follows
    assert torch.equal(whole[:, :25], part)
    for i in range(25, L):
        y, _, _ = gdn.gdn_layer_norm_forward(x[:, i], nw, bias=nb)
        u = gdn.gdn_conv_step(y, w, cs, bias=b)
        o = gdn.gdn_ssm_step(u, dt[:, i], A, B[:, i], C[:, i], hs, D=Dp, z=y)
        # the same formulas in another order of sums: a unit or two of fp32, then one rounding to the type
        e = torch.finfo(t).eps
        assert ((o.float() - whole[:, i].float()).abs() <= e * whole[:, i].float().abs() + 1e-4).all()
    assert torch.equal(cs, cs_w)
    assert torch.allclose(hs, hs_w, rtol=1e-4, atol=1e-4 if t == torch.float32 else 2e-2)


def test_with_the_gated_delta_rule():
    """q, k, v through one convolution, the gated delta rule, and layer norm per head: prefill of 48 tokens, and 32
    with 16 decode steps, agree."""
    rng = np.random.default_rng(22)
    N, L, H, d, C = 2, 48, 2, 32, 16
    t = torch.float32
    qkv = make(rng, t, N, L, 3 * H * d, scale=0.5)[0]
    w = make(rng, t, 3 * H * d, 4)[0]
    nw = make(rng, t, d)[0]
    al = torch.rand(N, L, H, device="cuda") * 0.5 + 0.5
    be = torch.rand(N, L, H, device="cuda")

    def split(u, rows):
        q, k, v = u.view(rows, 3, H, d).unbind(1)
        k = torch.nn.functional.normalize(k, dim=-1)
        return q.contiguous(), k.contiguous(), v.contiguous()

    def prefill(n):
        cu = [n * i for i in range(N + 1)]
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        u, cs = gdn.gdn_conv_forward(qkv[:, :n].reshape(N * n, -1), w, cud)
        cache = gdn.new_cache(N, H, d, d, C, t)
        q, k, v = split(u, N * n)
        o, _ = gdn.gdn_cpr_forward(q, k, v, al[:, :n].reshape(-1, H).contiguous(),
                                   be[:, :n].reshape(-1, H).contiguous(), cud, C, cu_seqlens_host=cu, cache_out=cache)
        return gdn.gdn_layer_norm_forward(o, nw)[0].view(N, n, H, d), cs, cache

    whole, _, _ = prefill(L)
    _, cs, cache = prefill(32)
    for i in range(32, L):
        u = gdn.gdn_conv_step(qkv[:, i], w, cs)
        q, k, v = split(u, N)
        o = gdn.gdn_decode_step(q, k, v, al[:, i].contiguous(), be[:, i].contiguous(), cache, C)
        y = gdn.gdn_layer_norm_forward(o, nw)[0]
        assert torch.allclose(y, whole[:, i], rtol=1e-5, atol=1e-5)
