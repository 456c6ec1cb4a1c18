"""The gated feed-forward block against its 64-bit definition.

Tolerances, U = 2^-24.  A product of n bf16 pairs in fp32 on the tensor cores adds 16 at a time, each
time off by at most 4 U of the magnitudes' sum M: e = (n / 4 + 8) U M.  act and act' (silu, gelu) are Lipschitz with
1.13 and 0.8 and evaluated within 12 U; so h is off by 1.13 |u| e_g + |act(g)| e_u + 16 U |h|, and half a step.
The backward reads g and u truncated to 24 bits, off by 2^-15 of their value (r below, in which e_g and e_u are included),
and rounds dg and du to bf16, 2^-8 of their value (up to 128 tokens, to two bf16 terms: 2^-16).  What that leaves in dx and in the weights' gradients is
summed by magnitude, with e of their own product.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn
from oracle import block_ops as ops
from test_gpu_layer_ops import HALF, U, make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def case(T, D, F, seed=0):
    rng = np.random.default_rng([seed, T, D, F])
    return dict(x=make(rng, BF, T, D), wg=make(rng, BF, F, D, scale=D ** -0.5), wu=make(rng, BF, F, D, scale=D ** -0.5),
                dh=make(rng, BF, T, F))


def e_dot(n, M):
    return (n / 4 + 8) * U * M


def near(name, got, want, tol, M=0.0):
    """M: the magnitudes' sum; a sum of which it passes fp32's range may overflow, and is not held to its value."""
    half = HALF[got.dtype] * np.abs(want) * (1 + 2.0 ** -7)
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, name
    bad = ~(np.abs(got - want) <= tol + half + 1e-37) & (M + np.zeros_like(want) < 3.3e38)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], (tol + half)[bad][:4])


def check(c, act="silu", views=None, backward=True, **kw):
    g = {n: v[0] for n, v in c.items()}
    g.update(views or {})
    x, wg, wu, dh = (c[n][1] for n in ("x", "wg", "wu", "dh"))
    T, D = x.shape
    F = wg.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, saved = gdn.gdn_glu_forward(g["x"], g["wg"], g["wu"], act=act, save=backward, status=status)
    G, V = x @ wg.T, x @ wu.T
    f, df = ops.ACT[act]
    eg, eu = (e_dot(D, np.abs(x) @ np.abs(w).T) for w in (wg, wu))
    a = f(G)
    near("h", h, a * V, 1.13 * np.abs(V) * eg + (np.abs(a) + 1.13 * eg) * eu + 16 * U * np.abs(a * V))
    plain, none = gdn.gdn_glu_forward(g["x"], g["wg"], g["wu"], act=act)
    assert torch.equal(plain, h) and none is None
    if not backward:
        return h, None
    grads = gdn.gdn_glu_backward(g["x"], g["wg"], g["wu"], g["dh"], saved, act=act, status=status, **kw)
    rg, ru = eg + 2.0 ** -15 * np.abs(G), eu + 2.0 ** -15 * np.abs(V)
    dg, du = dh * V * df(G), dh * a
    step = 2.0 ** -8 if T > 128 else 2.0 ** -16
    edg = step * np.abs(dg) * 1.01 + np.abs(dh) * (1.13 * ru + 0.8 * rg * (np.abs(V) + ru) + 16 * U * np.abs(V)) * 1.01
    edu = step * np.abs(du) * 1.01 + np.abs(dh) * (1.13 * rg + 12 * U * np.abs(a)) * 1.01
    n = np.abs
    want = ops.glu_backward(x, wg, wu, dh, act)
    near("dx", grads[0], want[0], edg @ n(wg) + edu @ n(wu) + e_dot(2 * F, n(dg) @ n(wg) + n(du) @ n(wu)) * 1.01)
    near("dwg", grads[1], want[1], edg.T @ n(x) + e_dot(T, n(dg).T @ n(x)) * 1.01, n(dg).T @ n(x))
    near("dwu", grads[2], want[2], edu.T @ n(x) + e_dot(T, n(du).T @ n(x)) * 1.01, n(du).T @ n(x))
    assert status.item() == gdn.GDN_OK
    return h, grads


@pytest.mark.parametrize("T,D,F", [(1, 64, 128), (1, 1, 1), (3, 8, 130), (16, 512, 256), (17, 72, 384), (33, 100, 40), (64, 1024, 200),
                                   (65, 64, 128), (128, 520, 512), (129, 200, 300), (256, 1003, 129)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_few_tokens(T, D, F, act):
    check(case(T, D, F), act)


@pytest.mark.parametrize("T,D,F,act", [(257, 64, 128, "silu"), (512, 256, 256, "gelu"), (300, 1003, 777, "gelu"), (700, 72, 1000, "silu"),
                                       (1024, 512, 640, "silu"), (333, 1, 5, "silu"), (2100, 264, 136, "gelu"), (600, 2048, 1032, "silu")])
def test_many_tokens(T, D, F, act):
    check(case(T, D, F), act)


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_ends(T, act):
    """Activations whose squares overflow fp32 keep their slopes, 1 and 0 (dw_up's first column, 1e20 * 1e20 dh, is out of
    range)."""
    c = case(T, 2, 40)
    ends = torch.tensor([1e20, -1e20, 30.0, -30.0, 0.0], dtype=BF).repeat(T // 5).cuda()
    x, wg, wu = (c[n][0].clone() for n in ("x", "wg", "wu"))
    x[:, 0], x[:, 1] = ends, 1.0
    wg[:, 0], wg[:, 1] = 1.0, 0.0
    wu[:, 0] = 0.0
    for n, t in dict(x=x, wg=wg, wu=wu).items():
        c[n] = (t, t.double().cpu().numpy())
    check(c, act)


def test_more_tiles_than_pairs_of_sms():
    check(case(3000, 128, 2000))


def test_long_sums_are_split():
    check(case(9000, 64, 72))


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_views(T, shift):
    """x and dh as slices of wider rows, the weights as halves of one matrix, at any alignment."""
    D, F = 104, 136
    c = case(T, D, F)
    both = torch.full((2 * F, D + 2 * shift), float("nan"), dtype=BF, device="cuda")
    wide = torch.full((T, D + F + 3 * shift), float("nan"), dtype=BF, device="cuda")
    v = dict(wg=both[:F, shift:shift + D], wu=both[F:, shift:shift + D], x=wide[:, shift:shift + D],
             dh=wide[:, D + 2 * shift:D + 2 * shift + F])
    for n, t in v.items():
        t.copy_(c[n][0])
    one, two = check(c, views=v), check(c)
    assert torch.equal(one[0], two[0])
    for a, b in zip(one[1], two[1]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("D,F", [(64, 136), (72, 264), (250, 131)])
def test_outputs_at_odd_addresses_get_the_same(T, D, F):
    """Outputs need the alignment of one element; what lies around them stays as it is."""
    c = case(T, D, F)

    def odd(*shape):
        n = int(np.prod(shape))
        b = torch.full((n + 24,), 7.0, dtype=BF, device="cuda")
        return b, b[11:11 + n].view(shape)

    h, saved = gdn.gdn_glu_forward(c["x"][0], c["wg"][0], c["wu"][0], save=True)
    one = gdn.gdn_glu_backward(c["x"][0], c["wg"][0], c["wu"][0], c["dh"][0], saved)
    bh, vh = odd(T, F)
    gdn.gdn_glu_forward(c["x"][0], c["wg"][0], c["wu"][0], h=vh)
    buffers = [odd(*g.shape) for g in one]
    gdn.gdn_glu_backward(c["x"][0], c["wg"][0], c["wu"][0], c["dh"][0], saved, grads=tuple(v for _, v in buffers))
    for (b, v), want in zip([(bh, vh)] + buffers, (h,) + tuple(one)):
        assert torch.equal(v, want) and (b[:11] == 7).all() and (b[11 + v.numel():] == 7).all()


@pytest.mark.parametrize("T", [7, 400])
def test_weight_gradients_in_fp32(T):
    c = case(T, 200, 72)
    f32 = lambda: torch.empty(72, 200, device="cuda")  # noqa: E731
    check(c, grads=(torch.empty(T, 200, dtype=BF, device="cuda"), f32(), f32()))


def test_no_tokens_and_leading_axes():
    c = case(0, 64, 32)
    _, grads = check(c)
    assert not grads[1].any() and not grads[2].any()
    c = case(12, 64, 32)
    h, saved = gdn.gdn_glu_forward(c["x"][0].view(3, 4, 64), c["wg"][0], c["wu"][0], save=True)
    assert h.shape == (3, 4, 32) and torch.equal(h.view(12, 32), check(c)[0])
    dx = gdn.gdn_glu_backward(c["x"][0].view(3, 4, 64), c["wg"][0], c["wu"][0], c["dh"][0].view(3, 4, 32), saved)[0]
    assert dx.shape == (3, 4, 64)


@pytest.mark.parametrize("T", [3, 300])
def test_extreme_projections(T):
    """Gates far on either side, and rows that are not finite."""
    c = case(T, 64, 64)
    x = c["x"][0].clone()
    x[0] *= 1000
    x[1] *= 1e18
    x[2, 5] = float("nan")
    h, _ = gdn.gdn_glu_forward(x, c["wg"][0], c["wu"][0])
    x64 = x.double().cpu().numpy()
    for r in (0, 1):
        want = ops.glu(x64[r:r + 1], c["wg"][1], c["wu"][1])
        e = e_dot(64, np.abs(x64[r:r + 1]) @ (np.abs(c["wg"][1]) + np.abs(c["wu"][1])).T)
        size = np.abs(x64[r:r + 1] @ c["wu"][1].T) + np.abs(x64[r:r + 1] @ c["wg"][1].T)
        near("h", h[r:r + 1], want, 2.3 * (size + e) * e + 16 * U * np.abs(want))
    assert torch.isnan(h[2]).all()
    assert torch.equal(h[3:], gdn.gdn_glu_forward(c["x"][0], c["wg"][0], c["wu"][0])[0][3:])


@pytest.mark.parametrize("T", [40, 500])
def test_repeats_give_the_same_bits_and_graphs_replay(T):
    c = case(T, 264, 520)
    g = {n: v[0].clone() for n, v in c.items()}
    out = [torch.empty(T, 520, dtype=BF, device="cuda"), torch.empty(6 * T * 520, dtype=torch.uint8, device="cuda")]
    grads = tuple(torch.empty(n, dtype=BF, device="cuda") for n in ((T, 264), (520, 264), (520, 264)))

    def step():
        gdn.gdn_glu_forward(g["x"], g["wg"], g["wu"], h=out[0], saved=out[1])
        gdn.gdn_glu_backward(g["x"], g["wg"], g["wu"], g["dh"], out[1], grads=grads)

    step()
    first = [v.clone() for v in (out[0],) + grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in (out[0],) + grads:
        v.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, (out[0],) + grads))
    d = case(T, 264, 520, seed=3)
    for n in g:
        g[n].copy_(d[n][0])
    graph.replay()
    h, two = check(d)
    assert torch.equal(h, out[0]) and all(torch.equal(a, b) for a, b in zip(two, grads))


def test_fp32_is_refused():
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_glu_forward(x, x, x)
    assert e.value.status == gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("T,D,F,shift", [(1, 1003, 777, 0), (5, 64, 100, 1), (16, 257, 2000, 0), (17, 510, 300, 3), (33, 1, 9, 0), (64, 4097, 72, 0),
                                         (64, 2048, 640, 5), (3, 8, 8, 7), (4, 63, 20000, 0), (40, 127, 10000, 0), (9, 8190, 64, 0)])
def test_few_tokens_of_rows_that_start_anywhere(T, D, F, shift):
    """Neighbours of the operands' rows that are not numbers do not reach the results."""
    c = case(T, D, F)
    views = {}
    for n in ("x", "wg", "wu"):
        rows = c[n][0].shape[0]
        wide = torch.full((rows * (D + shift) + 2 * shift,), float("nan"), dtype=BF, device="cuda")
        views[n] = wide[shift:shift + rows * (D + shift)].view(rows, D + shift)[:, :D]
        views[n].copy_(c[n][0])
    one, two = check(c, views=views, backward=T <= 17), check(c, backward=T <= 17)
    assert torch.equal(one[0], two[0])
