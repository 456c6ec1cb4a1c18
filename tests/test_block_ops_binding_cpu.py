"""What the binding hands to the library for the norm of queries and keys, the gated block and the policy loss, with the library
replaced by a recorder: no GPU is needed, and no address is read."""
import itertools

import pytest
import torch

from gated_deltanet_cpr_delta_b200 import build, gdn

BF, F32 = torch.bfloat16, torch.float32


class Recorder:
    """Stands for the library: sizes are 256, calls are recorded and return GDN_OK."""

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 256
        return lambda *a: self.calls.__setitem__(name, a) or 0


@pytest.fixture
def lib(monkeypatch):
    """CPU tensors pass for tensors on the device that `cpu` names."""
    rec, cpu = Recorder(), torch.device("cpu")
    monkeypatch.setattr(gdn, "load_library", lambda: rec)
    monkeypatch.setattr(gdn, "_gpu", lambda what, t: cpu)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: t.device)
    monkeypatch.setattr(gdn, "_call", lambda dev, what, fn, *args: fn(*args))
    monkeypatch.setattr(gdn, "_glu_scratch", lambda *a: (None, None, 0))
    return rec


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("given", list(itertools.product([0, 1], repeat=3)))
def test_gated_block_gradients_partly_given(lib, dtype, given):
    """Every buffer that the library writes has the type that it is told, whichever of the three the caller brings."""
    x, w, dh = torch.zeros(5, 8, dtype=BF), torch.zeros(6, 8, dtype=BF), torch.zeros(5, 6, dtype=BF)
    mine = (torch.empty(5, 8, dtype=BF), torch.empty(6, 8, dtype=dtype), torch.empty(6, 8, dtype=dtype))
    grads = tuple(g if on else None for g, on in zip(mine, given))
    out = gdn.gdn_glu_backward(x, w, w, dh, torch.zeros(6 * 30, dtype=torch.uint8), grads=grads)
    args = lib.calls["gdn_glu_backward"]
    want = dtype if given[1] or given[2] else BF
    assert args[7] == (gdn.GDN_F32 if want is F32 else gdn.GDN_BF16)
    assert [g.dtype for g in out] == [BF, want, want] and [g.shape for g in out] == [x.shape, w.shape, w.shape]
    assert list(args[4:7]) == [g.data_ptr() for g in out]
    for g, m, on in zip(out, mine, given):
        assert not on or g is m


def test_gated_block_gradients_of_two_types_are_refused(lib):
    x, w, dh = torch.zeros(5, 8, dtype=BF), torch.zeros(6, 8, dtype=BF), torch.zeros(5, 6, dtype=BF)
    for a, b in ((F32, BF), (BF, F32)):
        with pytest.raises(ValueError, match="dw_up"):
            gdn.gdn_glu_backward(x, w, w, dh, torch.zeros(180, dtype=torch.uint8),
                                 grads=(None, torch.empty(6, 8, dtype=a), torch.empty(6, 8, dtype=b)))


def test_a_new_output_has_the_type_that_is_asked_for():
    cpu = torch.device("cpu")
    like = torch.zeros(4, 8, dtype=BF)
    for dtype in (BF, F32):
        t, p = gdn._out("f", "y", None, dtype, (4, 8), cpu, like)
        assert t.dtype is dtype and t.shape == (4, 8) and t.is_contiguous() and p == t.data_ptr()
    # views and other orders of the axes come out dense
    for view in (torch.zeros(4, 16, dtype=BF)[:, :8], torch.zeros(8, 4, dtype=BF).t(), torch.zeros(1, 8, dtype=BF).expand(4, 8)):
        t, _ = gdn._out("f", "y", None, BF, (4, 8), cpu, view)
        assert t.is_contiguous() and t.shape == (4, 8)


BIG = 1 << 36


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory")
def test_temperatures_whose_reciprocal_leaves_the_range_are_refused():
    """2^-100 is the smallest that is taken: a call that passes every check ends with GDN_ERR_CUDA here."""
    build.build()
    lib = gdn.load_library()

    def forward(tau):
        s = gdn.PolicyStruct(BIG, 2 * BIG, 3 * BIG, None, 4 * BIG, 64, 10, 64, 0.2, 0.2, 0.0, tau, gdn.GDN_BF16)
        return lib.gdn_policy_loss_forward(s, 5 * BIG, 6 * BIG, None, None)

    assert [forward(t) for t in (1e-45, 1e-40, 1e-38, 2.0 ** -101, 0.0)] == [gdn.GDN_ERR_INVALID_ARG] * 5
    assert [forward(t) for t in (2.0 ** -100, 1e-6, 1.0, 1e30)] == [gdn.GDN_ERR_CUDA] * 4


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory")
def test_gradients_of_the_norms_outputs_in_fp32():
    """Which types the entry takes, and that the checks go by them: strides, alignment and overlap of 4-byte elements."""
    build.build()
    lib = gdn.load_library()
    A = [(i + 1) << 36 for i in range(12)]

    def call(t=gdn.GDN_BF16, g=gdn.GDN_F32, gq=A[2], ldgq=128, gk=A[3], ldgk=64, dq=A[4], dk=A[5]):
        s = gdn.QkNormStruct(A[0], A[1], None, None, None, None, 128, 64, 10, 4, 2, 32, 0, 0, 0, 1e-6, t, t)
        return lib.gdn_qk_norm_backward_ex(s, g, gq, ldgq, gk, ldgk, dq, dk, None, None, None, 0, None)

    bad, cuda = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_CUDA
    assert call() == cuda and call(g=gdn.GDN_BF16) == cuda and call(gdn.GDN_F32, gdn.GDN_F32) == cuda
    assert call(gdn.GDN_F32, gdn.GDN_BF16) == gdn.GDN_ERR_UNSUPPORTED
    assert call(g=2) == bad and call(g=-1) == bad
    assert call(gq=A[2] + 2) == bad and call(gq=A[2] + 2, g=gdn.GDN_BF16) == cuda and call(gq=A[2] + 4) == cuda
    assert call(ldgq=127) == bad and call(ldgk=63) == bad and call(gq=None) == bad
    size = 10 * 128 * 4
    assert call(dq=A[2] + size - 16) == bad and call(dq=A[2] + size) == cuda
    assert call(dq=A[2] + size // 2, g=gdn.GDN_BF16) == cuda
    assert lib.gdn_qk_norm_backward_ex(None, 0, A[2], 128, A[3], 64, A[4], A[5], None, None, None, 0, None) == bad
    assert lib.gdn_qk_norm_backward(None, A[2], 128, A[3], 64, A[4], A[5], None, None, None, 0, None) == bad
