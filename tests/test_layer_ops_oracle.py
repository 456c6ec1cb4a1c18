"""The 64-bit definitions of the layer operators: their gradients against
differences, their forwards against cases worked by hand."""
import numpy as np
import pytest

from oracle import layer_ops as ops

CU = np.array([0, 5, 5, 6, 13])


def _difference(f, a, at, h=1e-5):
    a = a.copy()
    old = a[at]
    a[at] = old + h
    up = f(a)
    a[at] = old - h
    down = f(a)
    return (up - down) / (2 * h)


def _check(f, args, grads, rng, n=6):
    # central differences in 64 bits: truncation h^2 f''' / 6 and rounding 1e-16 / h, both below 1e-8 here
    for name, g in grads.items():
        for _ in range(n):
            at = tuple(rng.integers(0, s) for s in g.shape)
            d = _difference(lambda a: f(dict(args, **{name: a})), args[name], at)
            assert abs(d - g[at]) <= 1e-6 * (1 + abs(d)), (name, at, d, g[at])


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", [True, False])
def test_conv_gradients(W, act):
    rng = np.random.default_rng(W)
    D = 3
    a = dict(x=rng.normal(size=(13, D)), w=rng.normal(size=(D, W)), b=rng.normal(size=D),
             state=rng.normal(size=(4, W - 1, D)))
    dy, do = rng.normal(size=(13, D)), rng.normal(size=(4, W - 1, D))

    def loss(a):
        y, s, _ = ops.conv(a["x"], a["w"], CU, a["b"], a["state"], act)
        return (y * dy).sum() + (s * do).sum()

    dx, dw, db, ds = ops.conv_backward(a["x"], a["w"], dy, CU, a["b"], a["state"], act, do)
    _check(loss, a, dict(x=dx, w=dw, b=db, state=ds), rng)


@pytest.mark.parametrize("soft", [True, False])
def test_ssm_gradients(soft):
    rng = np.random.default_rng(5)
    T, D, G, S = 13, 4, 2, 3
    a = dict(x=rng.normal(size=(T, D)), dt=rng.normal(size=(T, D)) * 0.5 + (0 if soft else 1.0),
             A=-rng.uniform(0.1, 2, (D, S)), B=rng.normal(size=(T, G, S)), C=rng.normal(size=(T, G, S)),
             D=rng.normal(size=D), z=rng.normal(size=(T, D)), dt_bias=rng.normal(size=D) * 0.1,
             state_in=rng.normal(size=(4, D, S)), dt_softplus=soft)
    dy, do = rng.normal(size=(T, D)), rng.normal(size=(4, D, S))

    def loss(a):
        y, last, _ = ops.ssm(a, CU)
        return (y * dy).sum() + (last * do).sum()

    g = ops.ssm_backward(a, dy, CU, do)
    _check(loss, a, dict(x=g["dx"], dt=g["ddt"], A=g["dA"], B=g["dB"], C=g["dC"], D=g["dD"], z=g["dz"],
                         dt_bias=g["ddt_bias"], state_in=g["dstate_in"]), rng)


def test_norm_gradients():
    rng = np.random.default_rng(7)
    a = dict(x=rng.normal(size=(5, 7)) + 3, w=rng.normal(size=7), b=rng.normal(size=7))
    dy = rng.normal(size=(5, 7))
    dx, dw, db = ops.layer_norm_backward(a["x"], a["w"], dy)
    _check(lambda a: (ops.layer_norm(a["x"], a["w"], a["b"])[0] * dy).sum(), a, dict(x=dx, w=dw, b=db), rng)


def test_by_hand():
    # taps 1, 10 on 1, 2, 3 with 5 before the start: 5 + 10, 1 + 20, 2 + 30
    y, s, _ = ops.conv(np.array([[1.], [2.], [3.]]), np.array([[1., 10.]]), [0, 3], None, np.array([[[5.]]]), False)
    assert y[:, 0].tolist() == [15, 21, 32] and s.tolist() == [[[3.0]]]
    # a sequence shorter than the state keeps part of it; an empty one keeps all of it
    _, s, _ = ops.conv(np.array([[7.]]), np.ones((1, 3)), [0, 1, 1], None, np.array([[[1.], [2.]], [[3.], [4.]]]))
    assert s[:, :, 0].tolist() == [[2, 7], [3, 4]]
    # decay 1/2, inputs 1, 1: 1, 1.5; the second sequence starts from its own state 4
    p = dict(x=np.ones((3, 1)), dt=np.ones((3, 1)), A=-np.log(2) * np.ones((1, 1)), B=np.ones((3, 1, 1)),
             C=np.ones((3, 1, 1)), dt_softplus=False, state_in=np.array([[[0.]], [[4.]]]))
    y, last, _ = ops.ssm(p, [0, 2, 3])
    assert np.allclose(y[:, 0], [1, 1.5, 3]) and np.allclose(last[:, 0, 0], [1.5, 3])
    y, mean, rstd = ops.layer_norm(np.array([[1., 3.]]), np.array([2., 1.]), np.array([0., 5.]), eps=3.0)
    assert np.allclose(y, [[-1.0, 5.5]]) and mean[0] == 2 and rstd[0] == 0.5
