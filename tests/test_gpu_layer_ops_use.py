"""Calls of the layer operators that their interface allows and ordinary batches do not make.  Tolerances as in
test_gpu_layer_ops (K roundings of 2^-24 on the magnitude sum M of a value's terms, and half a step of the output's type)."""
import numpy as np
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn
from oracle import layer_ops as ops
from test_gpu_layer_ops import SSM_GRADS, TYPES, close, conv_case, make, ssm_case, ssm_grads, ssm_run

pytestmark = pytest.mark.gpu
F32 = torch.float32


def odd(like, shift=1):
    """An output buffer that starts `shift` elements off the alignment of its allocation, filled with sevens."""
    return torch.full((like.numel() + shift,), 7.0, dtype=like.dtype, device="cuda")[shift:].view(like.shape)


def placed(cu_h, first, T):
    """Offsets moved `first` rows down in tensors of T rows."""
    cu_h = cu_h + first
    assert cu_h[-1] < T
    return torch.from_numpy(cu_h.astype(np.int32)).cuda(), cu_h


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,W", [(64, 4), (37, 3), (2, 2)])
def test_conv_of_rows_inside_a_padded_batch(dtype, D, W):
    """Sequences that start behind row 0 and end before the last row: the padding holds NaN and stays as it is."""
    t, first, T = TYPES[dtype], 19, 130
    d, _, cu_h = conv_case(t, D, W, [0, 40, 2, 0, 33, 7], True, True)
    cu, cu_h = placed(cu_h, first, T)
    last, rng = int(cu_h[-1]), np.random.default_rng(1)

    def padded():
        a = make(rng, t, T, D)[0]
        a[:first], a[last:] = float("nan"), float("nan")
        return a, torch.nan_to_num(a, nan=0.0).double().cpu().numpy()

    (x, x64), (dy, dy64) = padded(), padded()
    y = torch.full_like(x, 7.0)
    _, so = gdn.gdn_conv_forward(x, d["w"][0], cu, bias=d["b"][0], state_in=d["s"][0], y=y)
    a = (x64, d["w"][1], cu_h, d["b"][1], d["s"][1], True)
    (wy, ws, _), M = ops.conv(*a), ops.conv(*a, bound=True)[2]
    close("y", y[first:last], wy[first:last], (1.1 * M + np.abs(wy))[first:last], W + 26)
    assert torch.equal(so.double().cpu(), torch.from_numpy(ws))
    grads = (torch.full_like(x, 7.0), torch.empty(D, W, device="cuda"), torch.empty(D, device="cuda"),
             torch.empty(6, W - 1, D, device="cuda"))
    gdn.gdn_conv_backward(x, d["w"][0], dy, cu, bias=d["b"][0], state_in=d["s"][0], dstate_out=d["do"][0], grads=grads)
    a = (x64, d["w"][1], dy64, cu_h, d["b"][1], d["s"][1], True, d["do"][1])
    K = 2 * W + 60 + T
    for name, g, w, m in zip(("dx", "dw", "db", "ds"), grads, ops.conv_backward(*a), ops.conv_backward(*a, bound=True)):
        inside = slice(first, last) if name == "dx" else slice(None)
        close(name, g[inside], w[inside], m[inside], K)
    for out in (y, grads[0]):
        assert (out[:first] == 7).all() and (out[last:] == 7).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,G,S", [(64, 1, 16), (35, 5, 32), (24, 1, 64)])
def test_scan_of_rows_inside_a_padded_batch(dtype, D, G, S):
    t, first, T, lengths = TYPES[dtype], 21, 150, [0, 70, 1, 0, 33, 6]
    g, h, dy, do, _, cu_h = ssm_case(t, D, G, S, lengths)
    cu, cu_h = placed(cu_h, first, T)
    last = int(cu_h[-1])

    def pad(a):
        out = torch.full((T,) + a.shape[1:], float("nan"), dtype=t, device="cuda")
        out[first:last] = a
        return out, torch.nan_to_num(out, nan=0.0).double().cpu().numpy()

    for k in ("x", "dt", "B", "C", "z"):
        g[k], h[k] = pad(g[k])
    dy = pad(dy[0])
    y = torch.full_like(g["x"], 7.0)
    _, hs, states = ssm_run(g, cu, save_states=True, y=y)
    (wy, wl, _), (My, Ml, _) = ops.ssm(h, cu_h), ops.ssm(h, cu_h, bound=True)
    K = 8 * (max(lengths) + 8) + S + 60
    close("y", y[first:last], wy[first:last], My[first:last], K)
    close("state_out", hs, wl, Ml, K)
    like = lambda a: torch.full_like(a, 7.0)  # noqa: E731
    grads = tuple(like(g[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state_in"))
    ssm_grads(g, dy[0], states, cu, do[0], grads=grads)
    want, M = ops.ssm_backward(h, dy[1], cu_h, do[1]), ops.ssm_backward(h, dy[1], cu_h, do[1], bound=True)
    for name, got in zip(SSM_GRADS, grads):
        rows = name in ("dx", "ddt", "dB", "dC", "dz")
        inside = slice(first, last) if rows else slice(None)
        close(name, got[inside], want[name][inside], M[name][inside], K + D + T)
        assert not rows or ((got[:first] == 7).all() and (got[last:] == 7).all()), name
    assert (y[:first] == 7).all() and (y[last:] == 7).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_outputs_at_odd_addresses_get_the_same(dtype):
    """Token outputs need the alignment of one element; inputs are whole vectors."""
    t = TYPES[dtype]
    d, cu, cu_h = conv_case(t, 64, 4, [30, 9], True, True)
    K = 2.0 ** -24 * 39
    run = lambda **kw: gdn.gdn_conv_forward(d["x"][0], d["w"][0], cu, bias=d["b"][0], state_in=d["s"][0], **kw)  # noqa: E731
    y, _ = run()
    assert torch.equal(y, run(y=odd(y))[0])
    back = lambda **kw: gdn.gdn_conv_backward(d["x"][0], d["w"][0], d["dy"][0], cu, bias=d["b"][0], **kw)  # noqa: E731
    one = back()
    two = back(grads=(odd(one[0]), *(torch.empty_like(a) for a in one[1:])))
    assert torch.equal(one[0], two[0]) and torch.equal(one[3], two[3])
    # 39 terms of at most 16 in another order
    assert (one[1] - two[1]).abs().max() <= 2 * K * 39 * 16
    step = lambda **kw: gdn.gdn_conv_step(d["x"][0][:2], d["w"][0], d["s"][0], state_out=torch.empty_like(d["s"][0]), **kw)  # noqa: E731
    assert torch.equal(step(), step(y=odd(step())))
    g, _, dy, do, cu, _ = ssm_case(t, 64, 2, 16, [30, 70])
    y, last, states = ssm_run(g, cu, save_states=True)
    assert torch.equal(y, ssm_run(g, cu, y=odd(y))[0])
    one = ssm_grads(g, dy[0], states, cu, do[0])
    two = ssm_grads(g, dy[0], states, cu, do[0], grads=tuple(
        odd(a) if n in ("dx", "ddt", "dB", "dC", "dz") else torch.empty_like(a) for n, a in zip(SSM_GRADS, one)))
    for n, a, b in zip(SSM_GRADS, one, two):  # ddt_bias: 100 terms in another order
        assert torch.equal(a, b) if n != "ddt_bias" else torch.allclose(a, b, rtol=1e-4, atol=1e-4), n
    x = make(np.random.default_rng(2), t, 9, 64)[0]
    w = make(np.random.default_rng(3), t, 64)[0]
    y, mean, rstd = gdn.gdn_layer_norm_forward(x, w)
    assert ((gdn.gdn_layer_norm_forward(x, w, y=odd(y))[0].float() - y.float()).abs()
            <= 2.0 ** -7 * y.float().abs() * (t != F32) + 1e-5).all()


@pytest.mark.parametrize("xt,wt", [("bf16", "f32"), ("f32", "bf16")])
def test_weights_of_the_other_type(xt, wt):
    xt, wt = TYPES[xt], TYPES[wt]
    for D in (64, 1003, 77, 20001):
        rng = np.random.default_rng([9, D])
        (x, x64), (w, w64), (b, b64), (dy, dy64) = make(rng, xt, 20, D), make(rng, wt, D), make(rng, wt, D), make(rng, xt, 20, D)
        for xs, dys in ((x, dy), (x[:, 1:], dy[:, 1:])):
            a64, g64, n = (x64, dy64, D) if xs is x else (x64[:, 1:], dy64[:, 1:], D - 1)
            y, mean, rstd = gdn.gdn_layer_norm_forward(xs, w[:n], bias=b[:n])
            My, Mx, Mw, Mb = ops.layer_norm_bounds(a64, w64[:n], g64)
            d = 28 + D // 1024
            close("y", y, ops.layer_norm(a64, w64[:n], b64[:n])[0], My + np.abs(b64[:n]), 2 * d + 12)
            got = gdn.gdn_layer_norm_backward(xs, w[:n], dys, mean, rstd)
            for name, g, want, m in zip(("dx", "dw", "db"), got, ops.layer_norm_backward(a64, w64[:n], g64), (Mx, Mw, Mb)):
                close(name, g, want, m, 6 * d + 52)
    for D in (64, 33):
        d, cu, cu_h = conv_case(xt, D, 3, [9, 0, 20], True, True, wtype=wt)
        a = (d["x"][1], d["w"][1], d["dy"][1], cu_h, d["b"][1], d["s"][1], True, d["do"][1])
        got = gdn.gdn_conv_backward(d["x"][0], d["w"][0], d["dy"][0], cu, bias=d["b"][0], state_in=d["s"][0],
                                    dstate_out=d["do"][0])
        for name, g, want, m in zip(("dx", "dw", "db", "ds"), got, ops.conv_backward(*a), ops.conv_backward(*a, bound=True)):
            close(name, g, want, m, 66 + 29)
        y = gdn.gdn_conv_step(d["x"][0][:3], d["w"][0], d["s"][0], bias=d["b"][0])
        a = (d["x"][1][:3], d["w"][1], np.arange(4), d["b"][1], d["s"][1], True)
        close("step", y, ops.conv(*a)[0], 1.1 * ops.conv(*a, bound=True)[2] + np.abs(ops.conv(*a)[0]), 29)


def test_norm_gradients_of_a_dense_and_a_strided_operand():
    """x dense with odd rows, dy a view of wider ones, and the other way round: one access form for both."""
    for t in TYPES.values():
        rng = np.random.default_rng(10)
        R, D = 40, 1003
        (x, x64), (w, w64) = make(rng, t, R, D), make(rng, t, D)
        dy = make(rng, t, R, D + 5)[0][:, 2:2 + D]
        dy64 = dy.double().cpu().numpy()
        for a, a64, b, b64 in ((x, x64, dy, dy64), (dy, dy64, x, x64)):
            _, mean, rstd = gdn.gdn_layer_norm_forward(a, w)
            _, Mx, Mw, Mb = ops.layer_norm_bounds(a64, w64, b64)
            for name, g, want, m in zip(("dx", "dw", "db"), gdn.gdn_layer_norm_backward(a, w, b, mean, rstd),
                                        ops.layer_norm_backward(a64, w64, b64), (Mx, Mw, Mb)):
                close(name, g, want, m, 6 * 28 + 32 + R)


def test_more_sequences_than_a_grid_has_rows():
    """70000 sequences of 0 to 2 tokens: the steps' grid, and the tail of the convolution's."""
    N, D, S = 70000, 8, 16
    rng = np.random.default_rng(11)
    lengths = rng.integers(0, 3, N)
    cu_h = np.concatenate([[0], np.cumsum(lengths)])
    cu, T = torch.from_numpy(cu_h.astype(np.int32)).cuda(), int(cu_h[-1])
    x, dt = make(rng, F32, N, D)[0], make(rng, F32, N, D)[0]
    B = make(rng, F32, N, 1, S)[0]
    A = -torch.rand(D, S, device="cuda") - 0.1
    state = make(rng, F32, N, D, S)[0]
    delta = torch.nn.functional.softplus(dt.double())[:, :, None]
    want = torch.exp(delta * A.double()) * state.double() + delta * x.double()[:, :, None] * B.double()
    wy = (want * B.double()).sum(-1)
    y = gdn.gdn_ssm_step(x, dt, A, B, B, state)
    # 72 + S roundings on magnitudes of at most a few hundred (|x delta B| below 6^3, 16 states times |C| below 6)
    assert torch.allclose(state.double(), want, rtol=1e-4, atol=1e-4) and torch.allclose(y.double(), wy, rtol=1e-4, atol=1e-3)
    w, cs = make(rng, F32, D, 3)[0], make(rng, F32, N, 2, D)[0]
    xt = make(rng, F32, T, D)[0]
    yt, so = gdn.gdn_conv_forward(xt, w, cu, state_in=cs, silu=False)
    lens = torch.from_numpy(lengths).cuda()
    lo = cu[:-1].long()
    full = torch.cat([cs, torch.zeros(N, 2, D, device="cuda")], 1)
    for k in range(2):
        has = lens > k
        full[has, 2 + k] = xt[lo[has] + k]
        pre = (full[has, k:k + 3].double() * w.t().double()).sum(1)
        assert torch.allclose(yt[lo[has] + k].double(), pre, rtol=1e-5, atol=1e-5)
    assert torch.equal(so, torch.stack([full[torch.arange(N), lens], full[torch.arange(N), lens + 1]], 1))
    one, last, _ = gdn.gdn_ssm_forward(xt, xt, A, B[:1].expand(T, 1, S).contiguous(), B[:1].expand(T, 1, S).contiguous(), cu,
                                       state_in=state)
    assert torch.equal(last[lens == 0], state[lens == 0]) and torch.isfinite(one).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,S", [(5, 16), (16, 32), (3, 64)])
def test_a_group_for_every_channel(dtype, D, S):
    g, h, dy, do, cu, cu_h = ssm_case(TYPES[dtype], D, D, S, [40, 0, 65, 3])
    y, last, states = ssm_run(g, cu, save_states=True)
    K = 8 * 73 + S + 60
    (wy, wl, _), (My, Ml, _) = ops.ssm(h, cu_h), ops.ssm(h, cu_h, bound=True)
    close("y", y, wy, My, K)
    close("state_out", last, wl, Ml, K)
    want, M = ops.ssm_backward(h, dy[1], cu_h, do[1]), ops.ssm_backward(h, dy[1], cu_h, do[1], bound=True)
    for name, t in zip(SSM_GRADS, ssm_grads(g, dy[0], states, cu, do[0])):
        close(name, t, want[name], M[name], K + len(wy))


def test_negative_steps_and_growing_states():
    """Without softplus a step may be negative, and A may be positive: growth of up to e^0.02 a token over 200 tokens."""
    D, S, lengths = 40, 16, [200, 70, 0, 5]
    g, h, dy, do, cu, cu_h = ssm_case(F32, D, 1, S, lengths, bias=False, soft=False)
    rng = np.random.default_rng(12)
    for k, v in (("dt", rng.uniform(-0.02, 0.02, h["dt"].shape)), ("A", rng.uniform(-1, 1, (D, S)))):
        g[k] = torch.from_numpy(v.astype(np.float32)).cuda()
        h[k] = v.astype(np.float32).astype(np.float64)
    y, last, states = ssm_run(g, cu, False, save_states=True)
    wy, wl, _ = ops.ssm(h, cu_h)
    # magnitudes: every decay at its largest, e^0.02
    hb = dict(h, A=np.full((D, S), 0.0))
    scale = float(np.exp(0.02 * 200))
    My, Ml, _ = ops.ssm(hb, cu_h, bound=True)
    K = 8 * 208 + S + 60
    close("y", y, wy, scale * My, K)
    close("state_out", last, wl, scale * Ml, K)
    assert np.linalg.norm(last.double().cpu().numpy() - wl) <= 1e-5 * np.linalg.norm(wl)
    want = ops.ssm_backward(h, dy[1], cu_h, do[1])
    for name, t in zip(SSM_GRADS, ssm_grads(g, dy[0], states, cu, do[0], False)):
        if t is not None:
            err = np.linalg.norm(t.double().cpu().numpy() - want[name])
            assert err <= 1e-5 * np.linalg.norm(want[name]), (name, err)


def test_gradients_beyond_32_bits():
    """2.3e9 elements a tensor, zero but for the last rows: those give what they give alone."""
    T, D, S, n = 70000, 32768, 16, 64
    rng = np.random.default_rng(13)
    tail, _ = make(rng, torch.bfloat16, n, D)
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    x[T - n:] = tail
    w = make(rng, torch.bfloat16, D)[0]
    y, mean, rstd = gdn.gdn_layer_norm_forward(x, w)
    del y
    one = gdn.gdn_layer_norm_forward(tail, w)
    dx = gdn.gdn_layer_norm_backward(x, w, x, mean, rstd)[0]
    assert torch.equal(dx[T - n:], gdn.gdn_layer_norm_backward(tail, w, tail, *one[1:])[0])
    del dx, mean, rstd
    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    cu1 = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    A = -torch.rand(D, S, device="cuda") - 0.1
    B = make(rng, torch.bfloat16, T, 1, S)[0]
    _, _, st = gdn.gdn_ssm_forward(x, x, A, B, B, cu, save_states=True, y=torch.empty_like(x))
    grads = gdn.gdn_ssm_backward(x, x, A, B, B, x, st, cu)
    _, _, st1 = gdn.gdn_ssm_forward(tail, tail, A, B[T - n:], B[T - n:], cu1, save_states=True)
    alone = gdn.gdn_ssm_backward(tail, tail, A, B[T - n:], B[T - n:], tail, st1, cu1)
    for k in (0, 1, 3, 4):  # the forward's saved states may come from the other tile: 64 decays and a rounding to bf16
        a, b = grads[k][T - n:].float(), alone[k].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-4 * b.abs().max()).all(), k
    assert torch.allclose(grads[8][1], alone[8][0], rtol=1e-4, atol=1e-4)
