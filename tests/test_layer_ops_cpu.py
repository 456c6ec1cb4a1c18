"""Refusals and sizes of the layer operators that need no GPU: the C entries
check on the host before anything is enqueued, and the binding before that."""
import ctypes

import pytest
import torch

from gated_deltanet_cpr_delta_b200 import build, gdn

P = ctypes.c_void_p
A0, A1, A2, A3, A4, A5, A6, A7, A8 = ((i + 1) << 32 for i in range(9))  # never dereferenced: checks fail first
BAD, UNSUPPORTED, SCRATCH = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load_library()


def conv_forward(lib, **kw):
    a = dict(x=A0, ldx=64, w=A1, b=None, s=A2, cu=A3, N=2, T=10, D=64, W=4, silu=1, it=1, wt=1, y=A4, so=A5, st=None,
             stream=None)
    a.update(kw)
    return lib.gdn_conv_forward(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), BAD), (dict(T=-1), BAD), (dict(D=0), BAD), (dict(W=0), BAD), (dict(W=5), UNSUPPORTED),
    (dict(W=1), UNSUPPORTED), (dict(it=7), BAD), (dict(wt=3), BAD), (dict(x=None), BAD), (dict(ldx=63), BAD),
    (dict(x=A0 + 1), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(so=None), BAD), (dict(so=A5 + 8), BAD),
    (dict(s=A2 + 2), BAD), (dict(cu=None), BAD), (dict(y=A0), BAD), (dict(y=A0 + 2 * 64 * 9), BAD), (dict(so=A2), BAD),
    (dict(T=2 ** 31), BAD)])
def test_conv_forward_refuses(lib, kw, want):
    assert conv_forward(lib, **kw) == want


def conv_backward(lib, **kw):
    a = dict(x=A0, ldx=64, w=A1, b=None, s=None, dy=A2, ldg=64, do=None, cu=A3, N=2, T=10, D=64, W=4, silu=1, it=1,
             wt=1, dx=A4, dw=A5, db=None, ds=A6, ws=A7, wsb=1 << 30, st=None, stream=None)
    a.update(kw)
    return lib.gdn_conv_backward(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(W=5), UNSUPPORTED), (dict(dy=None), BAD), (dict(ldg=1), BAD), (dict(dx=None), BAD), (dict(dw=None), BAD),
    (dict(ds=None), BAD), (dict(do=A8 + 4), BAD), (dict(dx=A2), BAD), (dict(dx=A0), BAD), (dict(ws=None), SCRATCH),
    (dict(wsb=64), SCRATCH), (dict(ws=A7 + 16), BAD), (dict(do=A6), BAD), (dict(T=2 ** 31 - 1), BAD)])
def test_conv_backward_refuses(lib, kw, want):
    assert conv_backward(lib, **kw) == want


def conv_step(lib, **kw):
    a = dict(x=A0, ldx=64, w=A1, b=None, s=A2, so=A2, N=2, D=64, W=4, silu=1, it=1, wt=1, y=A4, stream=None)
    a.update(kw)
    return lib.gdn_conv_step(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(W=9), UNSUPPORTED), (dict(s=None), BAD), (dict(so=None), BAD), (dict(y=None), BAD), (dict(y=A0), BAD),
    (dict(y=A2), BAD), (dict(so=A2 + 16), BAD), (dict(so=A2 + 6), BAD), (dict(x=None), BAD)])
def test_conv_step_refuses(lib, kw, want):
    assert conv_step(lib, **kw) == want


def ssm_struct(**kw):
    a = dict(x=A0, dt=A1, B=A2, C=A3, z=None, A=A4, D=None, dt_bias=None, cu=A5, ldx=64, lddt=64, ldB=32, ldC=32,
             ldz=0, T=10, N=2, D_=64, G=2, S=16, soft=1, it=1)
    a.update(kw)
    return gdn.SsmStruct(*a.values())


SSM_BAD = [(dict(S=17), UNSUPPORTED), (dict(S=0), BAD), (dict(G=3), BAD), (dict(G=0), BAD), (dict(it=4), BAD),
           (dict(A=None), BAD), (dict(A=A4 + 4), BAD), (dict(x=None), BAD), (dict(dt=None), BAD), (dict(B=None), BAD),
           (dict(C=None), BAD), (dict(ldx=60), BAD), (dict(ldB=31), BAD), (dict(z=A6, ldz=2), BAD),
           (dict(D=A6 + 2), BAD), (dict(T=-1), BAD)]


@pytest.mark.parametrize("kw,want", SSM_BAD + [(dict(cu=None), BAD)])
def test_ssm_forward_refuses(lib, kw, want):
    s = ssm_struct(**kw)
    assert lib.gdn_ssm_forward(s, None, A7, A8, None, None, None) == want


def test_ssm_forward_refuses_buffers(lib):
    f = lambda si=None, y=A7, so=A8, cs=None: lib.gdn_ssm_forward(ssm_struct(), si, y, so, cs, None, None)  # noqa: E731
    assert f(y=None) == BAD and f(so=None) == BAD and f(so=A8 + 8) == BAD and f(cs=A5 + 4) == BAD
    assert f(y=A0) == BAD and f(y=A1 + 128) == BAD and f(si=A8) == BAD and f(y=A2) == BAD and f(y=A3) == BAD
    assert lib.gdn_ssm_forward(None, None, A7, A8, None, None, None) == BAD


@pytest.mark.parametrize("kw,want", SSM_BAD + [(dict(cu=None), BAD)])
def test_ssm_backward_refuses(lib, kw, want):
    o = [(20 + i) << 32 for i in range(12)]
    assert lib.gdn_ssm_backward(ssm_struct(**kw), o[0], 64, o[1], None, o[2], o[3], o[4], o[5], o[6], None, None, None,
                                o[7], o[8], 1 << 30, None, None) == want


def test_ssm_backward_refuses_buffers(lib):
    names = ("dy", "ld", "cs", "do", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "ds", "ws", "n")
    base = {n: (20 + i) << 32 for i, n in enumerate(names)}
    base.update(ld=64, do=None, dD=None, db=None, dz=None, n=1 << 30)
    f = lambda z=False, **kw: lib.gdn_ssm_backward(  # noqa: E731
        ssm_struct(**(dict(z=A6, ldz=64) if z else {})), *dict(base, **kw).values(), None, None)
    for n in ("dy", "cs", "dx", "ddt", "dA", "dB", "dC", "ds"):
        assert f(**{n: None}) == BAD, n
    assert f(z=True) == BAD                                   # dz is needed with z
    assert f(ld=63) == BAD and f(do=A8 + 8) == BAD and f(dx=base["dy"]) == BAD and f(dB=A2) == BAD
    assert f(do=base["ds"]) == BAD
    assert f(ws=None) == SCRATCH and f(n=256) == SCRATCH and f(ws=base["ws"] + 16) == BAD


@pytest.mark.parametrize("kw,want", SSM_BAD[:14] + [(dict(T=3), BAD)])
def test_ssm_step_refuses(lib, kw, want):
    s = ssm_struct(**dict(dict(T=2, N=2), **kw))
    assert lib.gdn_ssm_step(s, A7, A7, A8, None) == want


def test_ssm_step_refuses_buffers(lib):
    f = lambda s=A7, so=A7, y=A8: lib.gdn_ssm_step(ssm_struct(T=2, N=2), s, so, y, None)  # noqa: E731
    assert f(s=None) == BAD and f(so=None) == BAD and f(y=None) == BAD and f(so=A7 + 16) == BAD and f(s=A7 + 4) == BAD
    assert f(y=A0) == BAD


def test_layer_norm_refuses(lib):
    f = lambda x=A0, ld=64, w=A1, b=None, eps=1e-5, R=4, D=64, it=1, wt=1, y=A2, m=A3, r=A4: (  # noqa: E731
        lib.gdn_layer_norm_forward(x, ld, w, b, eps, R, D, it, wt, y, m, r, None))
    for kw in (dict(x=None), dict(ld=63), dict(w=None), dict(b=A5 + 1), dict(eps=-1.0), dict(eps=float("nan")),
               dict(R=-1), dict(D=0), dict(it=2), dict(wt=9), dict(y=None), dict(y=A0 + 64), dict(m=None),
               dict(r=None), dict(R=2 ** 31)):
        assert f(**kw) == BAD, kw
    g = lambda x=A0, ld=64, dy=A1, lg=64, w=A2, m=A3, r=A4, R=4, D=64, dx=A5, dw=A6, db=None, ws=A7, n=1 << 30: (  # noqa: E731
        lib.gdn_layer_norm_backward(x, ld, dy, lg, w, m, r, R, D, 1, 1, dx, dw, db, ws, n, None))
    for kw in (dict(x=None), dict(dy=None), dict(lg=10), dict(w=None), dict(m=None), dict(r=None), dict(dx=None),
               dict(dw=None), dict(dx=A0), dict(dx=A1), dict(R=-1), dict(D=0), dict(ws=A7 + 8)):
        assert g(**kw) == BAD, kw
    assert g(ws=None) == SCRATCH and g(n=8) == SCRATCH


def test_sizes(lib):
    assert gdn.gdn_ssm_num_chunk_states(100, 3) == 100 // gdn.SSM_CHUNK + 3
    with pytest.raises(gdn.GdnError):
        gdn.gdn_ssm_num_chunk_states(-1, 3)
    assert lib.gdn_ssm_backward_workspace_size(10, 1, 64, 3, 16) == 0
    assert lib.gdn_ssm_backward_workspace_size(1000, 1, 64, 1, 16) >= 1000 * 2 * 16 * 4
    assert lib.gdn_conv_backward_workspace_size(100, 1, 64, 5) == 0
    assert lib.gdn_conv_backward_workspace_size(100, 1, 64, 4) > 0
    assert lib.gdn_layer_norm_backward_workspace_size(-1, 4) == 0
    assert lib.gdn_layer_norm_backward_workspace_size(10, 64) >= 10 * 2 * 64 * 4


def test_binding_refuses_before_the_library():
    x, w = torch.zeros(4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_conv_forward(x, w)
    with pytest.raises(ValueError, match="weight"):
        gdn.gdn_conv_forward(x, torch.zeros(7, 4))
    with pytest.raises(ValueError, match="cu_seqlens"):
        gdn.gdn_conv_forward(x, w, torch.zeros(3, dtype=torch.int64))
    B = torch.zeros(4, 1, 16)
    with pytest.raises(ValueError, match="A must have shape"):
        gdn.gdn_ssm_forward(x, x, torch.zeros(8, 8), B, B)
    with pytest.raises(ValueError, match="dt must be"):
        gdn.gdn_ssm_forward(x, x.double(), torch.zeros(8, 16), B, B)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.gdn_ssm_forward(x.t().contiguous().t(), x, torch.zeros(8, 16), B, B)
    with pytest.raises(ValueError, match="overlap"):
        gdn.gdn_ssm_forward(x[:1].expand(4, 8), x, torch.zeros(8, 16), B, B)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_layer_norm_forward(x, torch.zeros(8))
