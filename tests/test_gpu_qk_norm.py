"""The norm of queries and keys with the position rotation against its 64-bit definition.

Tolerances: half a step of the output's type, plus K units of 2^-24 on the magnitude M of a value's
terms (|a| + |b| for a turned pair).  Roundings: a row's sum of squares, all positive, 8 per
thread and 5 joins, with the division and eps 16 units, half of that on r, and 2 of the square root: r 10;
two products 2; an angle's sine and cosine 2 + 3.2 (the turns rounded to fp32, times 2 pi); the turn 2.
Outputs 10 + 2 + 5.2 + 2 < K = 24.  Gradients: the gradient turned back 8, r three times 30, its sum 16, products
8: dx K = 64; the weights' gradients 8 + 10 + 4 and one rounding per row of a thread, at most the rows: K = 24 + R.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn
from oracle import block_ops as ops
from test_gpu_layer_ops import TYPES, close, make

pytestmark = pytest.mark.gpu


def case(t, T, Hq, Hk, d, rot, weight=True, wtype=None, seed=0, far=0):
    rng = np.random.default_rng([seed, T, Hq, Hk, d, rot])
    c = dict(q=make(rng, t, T, Hq, d), k=make(rng, t, T, Hk, d, scale=3.0), dq=make(rng, t, T, Hq, d), dk=make(rng, t, T, Hk, d))
    c["qw"], c["kw"] = (make(rng, wtype or t, d), make(rng, wtype or t, d)) if weight else ((None, None), (None, None))
    pos = rng.integers(0, 5000, T).astype(np.int32) + np.int32(far)
    freq = (1e4 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    c["pos"] = (torch.from_numpy(pos).cuda(), pos) if rot else (None, None)
    c["freq"] = (torch.from_numpy(freq).cuda(), freq.astype(np.float64)) if rot else (None, None)
    return c


def check(c, inter=False, l2=False, eps=1e-6, views=None, **kw):
    g = {n: v[0] for n, v in c.items()}
    g.update(views or {})
    args = dict(q_weight=g["qw"], k_weight=g["kw"], positions=g["pos"], inv_freq=g["freq"], interleaved=inter, l2=l2, eps=eps)
    out = gdn.gdn_qk_norm_forward(g["q"], g["k"], **args, **kw)
    grads = gdn.gdn_qk_norm_backward(g["q"], g["k"], g["dq"], g["dk"], **args)
    rot = dict(pos=c["pos"][1], freq=c["freq"][1], inter=inter, l2=l2, eps=eps)
    for i, n in enumerate("qk"):
        x, w, dy = c[n][1], c[n + "w"][1], c["d" + n][1]
        close(n, out[i], ops.head_norm(x, w, **rot), ops.head_norm(x, w, bound=True, **rot), 24)
        dx, dw = ops.head_norm_backward(x, dy, w, **rot)
        Mx, Mw = ops.head_norm_backward(x, dy, w, bound=True, **rot)
        close("d" + n, grads[i], dx, Mx, 64)
        if w is None:
            assert grads[2 + i] is None
        else:
            close("d" + n + " weight", grads[2 + i], dw, Mw, 24 + x.shape[0] * x.shape[1])
    return out, grads


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter", [
    (1, 1, 1, 2, 2, False), (1, 1, 1, 16, 0, False), (3, 2, 1, 64, 64, False), (70, 4, 4, 128, 128, False),
    (33, 7, 3, 90, 40, True), (5, 3, 2, 128, 64, True), (9, 2, 2, 256, 256, False), (65, 1, 2, 254, 254, False),
    (17, 5, 1, 34, 22, False), (40, 16, 2, 96, 24, False), (300, 3, 3, 8, 8, True), (257, 8, 1, 4, 2, False)])
def test_sizes(dtype, T, Hq, Hk, d, rot, inter):
    check(case(TYPES[dtype], T, Hq, Hk, d, rot), inter)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("l2", [False, True])
def test_without_weights_and_at_far_positions(dtype, l2):
    check(case(TYPES[dtype], 40, 4, 2, 64, 64, weight=False, far=2 ** 31 - 6000), l2=l2)
    check(case(TYPES[dtype], 40, 4, 2, 64, 32, far=-(2 ** 31)), l2=l2)
    check(case(TYPES[dtype], 11, 4, 2, 64, 0, weight=False), l2=l2, eps=0.0)


@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f32", "bf16")])
def test_weights_of_the_other_type(dtype, wtype):
    c = case(TYPES[dtype], 21, 3, 2, 72, 16, wtype=TYPES[wtype])
    check(c)
    c["kw"] = (None, None)  # one weight alone
    check(c)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_views_of_one_projection(dtype, shift):
    """q, k and their gradients as slices of wider rows, at any alignment."""
    t, (T, Hq, Hk, d) = TYPES[dtype], (37, 4, 2, 64)
    c = case(t, T, Hq, Hk, d, 32)
    wide = torch.full((T, shift + 2 * (Hq + Hk) * d + 3 * shift), float("nan"), dtype=t, device="cuda")
    views, at = {}, shift
    for n, H in (("q", Hq), ("k", Hk), ("dq", Hq), ("dk", Hk)):
        views[n] = wide[:, at:at + H * d].unflatten(1, (H, d))
        views[n].copy_(c[n][0])
        at += H * d
    out, grads = check(c, views=views)
    one, two = check(c)
    for a, b in zip(out + tuple(grads[:2]), one + tuple(two[:2])):
        assert torch.equal(a, b)


def test_repeats_give_the_same_bits_and_no_tokens_give_zeros():
    c = case(torch.bfloat16, 500, 4, 2, 128, 64)
    a, b = check(c), check(c)
    for x, y in zip(a[0] + tuple(a[1]), b[0] + tuple(b[1])):
        assert torch.equal(x, y)
    c = case(torch.bfloat16, 0, 4, 2, 128, 64)
    (q, k), grads = check(c)
    assert q.shape == (0, 4, 128) and k.shape == (0, 2, 128) and not grads[2].any() and not grads[3].any()


def test_rows_that_are_not_finite_stay_in_their_row():
    c = case(torch.float32, 9, 2, 2, 64, 64)
    q = c["q"][0].clone()
    q[3, 1, 5] = float("inf")
    q[4, 0, 7] = float("nan")
    args = dict(positions=c["pos"][0], inv_freq=c["freq"][0])
    a, b = gdn.gdn_qk_norm_forward(q, c["k"][0], **args), gdn.gdn_qk_norm_forward(c["q"][0], c["k"][0], **args)
    keep = torch.ones(9, 2, dtype=torch.bool, device="cuda")
    keep[3, 1] = keep[4, 0] = False
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1], b[1]) and torch.isnan(a[0][4, 0]).all()


def test_a_graph_replays_other_values_and_positions():
    c = case(torch.bfloat16, 64, 4, 2, 64, 64)
    q, k, pos = c["q"][0].clone(), c["k"][0].clone(), c["pos"][0].clone()
    out = torch.empty_like(q), torch.empty_like(k)
    call = lambda: gdn.gdn_qk_norm_forward(q, k, positions=pos, inv_freq=c["freq"][0], q_out=out[0], k_out=out[1])  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    d = case(torch.bfloat16, 64, 4, 2, 64, 64, seed=5)
    q.copy_(d["q"][0]), k.copy_(d["k"][0]), pos.copy_(d["pos"][0])
    graph.replay()
    want = gdn.gdn_qk_norm_forward(d["q"][0], d["k"][0], positions=d["pos"][0], inv_freq=c["freq"][0])
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_many_tokens():
    """More tokens than a launch has blocks at a time; sums over all of them."""
    t = torch.float32
    T, H, d = 30000, 2, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    q, dq = torch.randn(T, H, d, device="cuda", generator=g), torch.randn(T, H, d, device="cuda", generator=g)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freq = 100.0 ** (-torch.arange(8, device="cuda", dtype=t) / 8)
    w = torch.ones(d, device="cuda")
    args = dict(q_weight=w, k_weight=w, positions=pos, inv_freq=freq)
    y, _ = gdn.gdn_qk_norm_forward(q, q, **args)
    n = lambda v: v.double().cpu().numpy()  # noqa: E731
    kw = dict(pos=pos.cpu().numpy(), freq=n(freq))
    close("q", y, ops.head_norm(n(q), n(w), **kw), ops.head_norm(n(q), n(w), bound=True, **kw), 24)
    got = gdn.gdn_qk_norm_backward(q, q, dq, dq, **args)
    for i, (a, m) in enumerate(zip(ops.head_norm_backward(n(q), n(dq), n(w), **kw), ops.head_norm_backward(n(q), n(dq), n(w), bound=True, **kw))):
        close(str(i), got[2 * i], a, m, 64 if i == 0 else 24 + T)
    assert torch.equal(got[0], got[1]) and torch.equal(got[2], got[3])
