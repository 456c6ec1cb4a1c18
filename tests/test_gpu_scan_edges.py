"""The selective scan on the GPU: batches wide enough for the forward's short tiles, with the states that it saves and the
gradients made from them.

Tolerances as in test_gpu_layer_ops: a term passes at most L decays, each off by 2.5 + 2 units, then the sum over
the states: 8 (L + 8) + S + 60 units on the magnitude sum; dB and dC sum over the channels of a group too, and the parameters'
gradients over the tokens.  In the norm, where roundings add like a random walk, fp32 results are within 1e-5.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn
from oracle import layer_ops as ops
from test_gpu_layer_ops import SSM_GRADS, TYPES, close, ssm_case, ssm_grads, ssm_run

pytestmark = pytest.mark.gpu


def near(name, got, want):
    if got.dtype == torch.float32:
        err = np.linalg.norm(got.double().cpu().numpy() - want)
        assert err <= 1e-5 * np.linalg.norm(want), (name, err / np.linalg.norm(want))


LENGTHS = [65, 130, 0, 1, 64, 33, 2, 31, 32, 5, 0, 8, 7, 9, 16, 40, 3, 128, 1, 1, 63, 10, 0, 4, 20, 12, 6, 97]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("S", [16, 32, 64])
@pytest.mark.parametrize("D,G", [(600, 1), (600, 3), (603, 1)])
def test_saved_states_and_gradients_of_wide_batches(dtype, S, D, G):
    """28 sequences of 600 channels: 16800 pairs, above where the forward takes tiles of 64 tokens."""
    g, h, dy, do, cu, cu_h = ssm_case(TYPES[dtype], D, G, S, LENGTHS)
    y, last, states = ssm_run(g, cu, save_states=True)
    wy, wl, hs = ops.ssm(h, cu_h)
    My, Ml, Mh = ops.ssm(h, cu_h, bound=True)
    K = 8 * (max(LENGTHS) + 8) + S + 60
    close("y", y, wy, My, K)
    close("state_out", last, wl, Ml, K)
    near("state_out", last, wl)
    states64 = states.double().cpu().numpy()
    for n, L in enumerate(LENGTHS):
        for k in range(-(-L // gdn.SSM_CHUNK)):
            lo, t = int(cu_h[n]), int(cu_h[n]) + k * gdn.SSM_CHUNK
            want, M = (hs[t - 1], Mh[t - 1]) if k else (h["state_in"][n], np.abs(h["state_in"][n]))
            got = states64[lo // gdn.SSM_CHUNK + n + k]
            assert (np.abs(got - want) <= K * 2.0 ** -24 * M).all(), (n, k)
    got = ssm_grads(g, dy[0], states, cu, do[0])
    want, M = ops.ssm_backward(h, dy[1], cu_h, do[1]), ops.ssm_backward(h, dy[1], cu_h, do[1], bound=True)
    for name, t in zip(SSM_GRADS, got):
        close(name, t, want[name], M[name], K + (D // G if name in ("dB", "dC") else len(wy)))
        near(name, t, want[name])


def softplus_case(dt):
    """States of single tokens from zero with x = B = 1: the state is the step width itself."""
    N, D = dt.shape
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    A, B = -one(D, 16), one(N, 1, 16)
    state = torch.zeros(N, D, 16, device="cuda")
    gdn.gdn_ssm_step(one(N, D), dt, A, B, B, state)
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    return state, gdn.gdn_ssm_forward(one(N, D), dt, A, B, B, cu)[1]


@pytest.mark.parametrize("D", [4096, 96])
def test_step_widths_are_accurate_relative_to_their_value(D):
    """softplus over [-20, 5], where step widths lie.  In units of 2^-24: e^-|v| is off by 2.5 (2^x in one
    instruction), 0.9 (ln 2 rounded, times |v|) and 1; log1p's polynomial by 0.6 and, relative to its smallest
    value ln 2, 3 of its roundings; the result by 1: 9 in all."""
    dt = torch.linspace(-20, 5, 64 * D, device="cuda").view(64, D)
    v = dt.double().cpu().numpy()
    want = np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))
    for got in softplus_case(dt):
        got = got.double().cpu().numpy()
        assert (got == got[:, :, :1]).all()
        assert np.abs(got[:, :, 0] / want - 1).max() <= 9 * 2.0 ** -24


def test_step_widths_at_the_ends():
    inf, nan = float("inf"), float("nan")
    dt = torch.tensor([[-inf, -3e38, -1e5, -200, -104, -88, 0, 88, 104, 200, 1e5, 3e38, inf, nan]], device="cuda")
    got = softplus_case(dt)[0][0, :, 0].cpu()
    want = torch.tensor([0, 0, 0, 0, 0, 0, np.log(2), 88, 104, 200, 1e5, 3e38, inf, nan], dtype=torch.float32)
    assert torch.equal(got[7:13], want[7:13]) and got[13].isnan()
    assert (got[:6].abs() <= 2.0 ** -126).all() and abs(got[6] - want[6]) <= 9 * 2.0 ** -24
