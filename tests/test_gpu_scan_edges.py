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
