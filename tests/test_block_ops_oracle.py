"""The 64-bit definitions of the norm of queries and keys, the gated block and the policy loss: their
gradients against differences, their forwards against cases worked by hand."""
import numpy as np
import pytest

from oracle import block_ops as ops
from test_layer_ops_oracle import _check


@pytest.mark.parametrize("rot,inter,l2", [(0, False, False), (4, False, True), (6, True, False), (8, False, False)])
def test_head_norm_gradients(rot, inter, l2):
    rng = np.random.default_rng(rot)
    a = dict(x=rng.normal(size=(4, 3, 8)), w=rng.normal(size=8))
    dy, pos, freq = rng.normal(size=(4, 3, 8)), np.array([0, 5, -3, 100]), rng.uniform(0.01, 1, rot // 2)
    kw = dict(pos=pos, freq=freq, inter=inter, l2=l2, eps=1e-3)
    dx, dw = ops.head_norm_backward(a["x"], dy, a["w"], **kw)
    _check(lambda a: (ops.head_norm(a["x"], a["w"], **kw) * dy).sum(), a, dict(x=dx, w=dw), rng)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_gradients(act):
    rng = np.random.default_rng(3)
    a = dict(x=rng.normal(size=(5, 4)), wg=rng.normal(size=(6, 4)), wu=rng.normal(size=(6, 4)))
    dh = rng.normal(size=(5, 6))
    dx, dwg, dwu = ops.glu_backward(a["x"], a["wg"], a["wu"], dh, act)
    _check(lambda a: (ops.glu(a["x"], a["wg"], a["wu"], act) * dh).sum(), a, dict(x=dx, wg=dwg, wu=dwu), rng)


@pytest.mark.parametrize("tau,kl", [(1.0, 0.0), (0.7, 0.3)])
def test_policy_gradient(tau, kl):
    rng = np.random.default_rng(4)
    z, y = rng.normal(size=(12, 7)) * 2, rng.integers(0, 7, 12)
    y[3] = -100
    lp = ops.policy(z, y, tau=tau)[1]
    kw = dict(old=lp - np.linspace(-0.5, 0.5, 12), adv=rng.normal(size=12), ref=lp + rng.normal(size=12) * 0.3 if kl else None,
              lo=0.1, hi=0.25, kl=kl, tau=tau)  # ratios away from the borders
    w = rng.normal(size=12)
    dz = ops.policy_backward(z, y, w, **kw)
    _check(lambda a: (ops.policy(a["z"], y, **kw)[0] * w).sum(), dict(z=z), dict(z=dz), rng, n=40)
    assert (dz[3] == 0).all()


def test_by_hand():
    # (3, 4) at unit length is (0.6, 0.8), a quarter turn on (-0.8, 0.6)
    x = np.array([[[3.0, 4.0]]])
    assert np.allclose(ops.head_norm(x, l2=True, eps=0), [0.6, 0.8])
    assert np.allclose(ops.head_norm(x, np.array([1.0, 1.0]), np.array([1]), np.array([np.pi / 2]), l2=True, eps=0), [-0.8, 0.6])
    # mean square 12.5
    assert np.allclose(ops.head_norm(x, eps=0), np.array([3, 4]) / np.sqrt(12.5))
    # pairs (0, 2), (1, 3) and (0, 1), (2, 3) by a half turn of the second pair
    x, f = np.array([[[1.0, 1.0, 1.0, 1.0]]]), np.array([0.0, np.pi])
    assert np.allclose(ops.head_norm(x, None, np.array([1]), f, False, eps=0), [1, -1, 1, -1])
    assert np.allclose(ops.head_norm(x, None, np.array([1]), f, True, eps=0), [1, 1, -1, -1])
    assert np.allclose(ops.glu(np.array([[2.0]]), np.array([[0.5]]), np.array([[3.0]])), 6 / (1 + np.exp(-1)))
    # probabilities 1/4, 3/4; ratio 1.5 held at 1.2 for a positive advantage, not for a negative one
    z, y = np.log(np.array([[1.0, 3.0]] * 2)), np.array([1, 1])
    loss, lp, d, _ = ops.policy(z, y, np.log([0.5, 0.5]), np.array([1.0, -1.0]))
    assert np.allclose(lp, np.log(0.75)) and np.allclose(loss, [-1.2, 1.5]) and np.allclose(d, [0, 1.5])
    loss, _, d, _ = ops.policy(z, y, lp, np.zeros(2), lp + np.log(2), kl=0.5)
    assert np.allclose(loss, 0.5 * (2 - np.log(2) - 1)) and np.allclose(d, -0.5)
