"""The norm of queries and keys, the gated block and the policy loss where a call's form, sizes or values are at an edge."""
import itertools

import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rand(seed, *shape, t=BF, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)


@pytest.mark.parametrize("T", [7, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gated_block_gradients_partly_given(T, dtype):
    """Buffers that the caller leaves out are made in the type of those that are given; the values are the same."""
    D, F = 200, 72
    x, wg, wu, dh = rand(1, T, D), rand(2, F, D, scale=0.1), rand(3, F, D, scale=0.1), rand(4, T, F)
    _, saved = gdn.gdn_glu_forward(x, wg, wu, save=True)
    full = lambda: (torch.empty(T, D, dtype=BF, device="cuda"),) + tuple(torch.empty(F, D, dtype=dtype, device="cuda") for _ in range(2))  # noqa: E731
    want = gdn.gdn_glu_backward(x, wg, wu, dh, saved, grads=full())
    for given in itertools.product([0, 1], repeat=3):
        if not given[1] and not given[2] and dtype is F32:
            continue
        got = gdn.gdn_glu_backward(x, wg, wu, dh, saved, grads=tuple(b if on else None for b, on in zip(full(), given)))
        for a, b in zip(got, want):
            assert a.dtype is b.dtype and torch.equal(a, b), given
