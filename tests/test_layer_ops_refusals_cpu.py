"""What the layer operators' C entries refuse, on a machine without a GPU: there a call that passes
every check ends with GDN_ERR_CUDA at its first CUDA call, so an accepted call can be told from a
refused one.  No address is dereferenced."""
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import build, gdn

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory")
BAD, UNSUPPORTED, SCRATCH = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE
CUDA = gdn.GDN_ERR_CUDA
A = [(i + 1) << 32 for i in range(64)]  # far apart


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load_library()


def conv_forward(lib, **kw):
    a = dict(x=A[0], ldx=64, w=A[1], b=A[2], s=A[3], cu=A[4], N=2, T=10, D=64, W=4, silu=1, it=1, wt=1, y=A[5], so=A[6],
             st=A[7], stream=None)
    a.update(kw)
    return lib.gdn_conv_forward(*a.values())


def conv_backward(lib, **kw):
    a = dict(x=A[0], ldx=64, w=A[1], b=A[2], s=A[3], dy=A[4], ldg=64, do=A[5], cu=A[6], N=2, T=10, D=64, W=4, silu=1, it=1,
             wt=1, dx=A[7], dw=A[8], db=A[9], ds=A[10], ws=A[11], wsb=1 << 30, st=A[12], stream=None)
    a.update(kw)
    return lib.gdn_conv_backward(*a.values())


def conv_step(lib, **kw):
    a = dict(x=A[0], ldx=64, w=A[1], b=A[2], s=A[3], so=A[3], N=2, D=64, W=4, silu=1, it=1, wt=1, y=A[4], stream=None)
    a.update(kw)
    return lib.gdn_conv_step(*a.values())


def norm_forward(lib, **kw):
    a = dict(x=A[0], ldx=64, w=A[1], b=A[2], eps=1e-5, R=4, D=64, it=1, wt=1, y=A[3], m=A[4], r=A[5], stream=None)
    a.update(kw)
    return lib.gdn_layer_norm_forward(*a.values())


def norm_backward(lib, **kw):
    a = dict(x=A[0], ldx=64, dy=A[1], ldg=64, w=A[2], m=A[3], r=A[4], R=4, D=64, it=1, wt=1, dx=A[5], dw=A[6], db=A[7],
             ws=A[8], wsb=1 << 30, stream=None)
    a.update(kw)
    return lib.gdn_layer_norm_backward(*a.values())


SSM = dict(x=A[0], dt=A[1], B=A[2], C=A[3], z=A[4], A=A[5], D=A[6], dt_bias=A[7], cu=A[8], ldx=64, lddt=64, ldB=32, ldC=32,
           ldz=64, T=10, N=2, D_=64, G=2, S=16, soft=1, it=1)


def ssm_forward(lib, **kw):
    o = dict(si=A[20], y=A[21], so=A[22], cs=A[23], st=A[24], stream=None)
    s = gdn.SsmStruct(*dict(SSM, **{k: v for k, v in kw.items() if k in SSM}).values())
    return lib.gdn_ssm_forward(s, *dict(o, **{k: v for k, v in kw.items() if k in o}).values())


def ssm_backward(lib, **kw):
    o = dict(dy=A[20], ldg=64, cs=A[21], do=A[22], dx=A[23], ddt=A[24], dA=A[25], dB=A[26], dC=A[27], dD=A[28], dz=A[29],
             db=A[30], ds=A[31], ws=A[32], wsb=1 << 30, st=A[33], stream=None)
    s = gdn.SsmStruct(*dict(SSM, **{k: v for k, v in kw.items() if k in SSM}).values())
    return lib.gdn_ssm_backward(s, *dict(o, **{k: v for k, v in kw.items() if k in o}).values())


def ssm_step(lib, **kw):
    o = dict(s=A[20], so=A[20], y=A[21], stream=None)
    s = gdn.SsmStruct(*dict(SSM, T=2, **{k: v for k, v in kw.items() if k in SSM}).values())
    return lib.gdn_ssm_step(s, *dict(o, **{k: v for k, v in kw.items() if k in o}).values())


CALLS = [conv_forward, conv_backward, conv_step, norm_forward, norm_backward, ssm_forward, ssm_backward, ssm_step]


@pytest.mark.parametrize("call", CALLS)
def test_a_valid_call_without_a_gpu_is_a_cuda_error(lib, call):
    assert call(lib) == CUDA
