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


# bytes of each tensor of the calls above (bf16 tokens, parameters as the call has them)
TOK, BC = 10 * 64 * 2, 10 * 2 * 16 * 2
OVERLAPS = {
    conv_forward: (dict(x=TOK, w=64 * 4 * 2, b=128, s=2 * 3 * 64 * 2, cu=12), dict(y=TOK, so=2 * 3 * 64 * 2, st=4)),
    conv_backward: (dict(x=TOK, w=64 * 4 * 2, b=128, s=2 * 3 * 64 * 2, cu=12, dy=TOK, do=2 * 3 * 64 * 4),
                    dict(dx=TOK, dw=64 * 4 * 4, db=256, ds=2 * 3 * 64 * 4, ws=2 * 5 * 64 * 4, st=4)),
    conv_step: (dict(x=2 * 64 * 2, w=64 * 4 * 2, b=128), dict(y=2 * 64 * 2, so=2 * 3 * 64 * 2)),
    norm_forward: (dict(x=4 * 64 * 2, w=128, b=128), dict(y=4 * 64 * 2, m=16, r=16)),
    norm_backward: (dict(x=4 * 64 * 2, dy=4 * 64 * 2, w=128, m=16, r=16), dict(dx=4 * 64 * 2, dw=256, db=256, ws=4 * 2 * 64 * 4)),
    ssm_forward: (dict(x=TOK, dt=TOK, B=BC, C=BC, z=TOK, A=4096, D=256, dt_bias=256, cu=12, si=8192),
                  dict(y=TOK, so=8192, cs=2 * 4096, st=4)),
    ssm_backward: (dict(x=TOK, dt=TOK, B=BC, C=BC, z=TOK, A=4096, D=256, dt_bias=256, cu=12, dy=TOK, cs=8192, do=8192),
                   dict(dx=TOK, ddt=TOK, dA=4096, dB=BC, dC=BC, dD=256, dz=TOK, db=256, ds=8192, ws=8192 + 1024 + 2560, st=4)),
    ssm_step: (dict(x=256, dt=256, B=128, C=128, z=256, A=4096, D=256, dt_bias=256), dict(y=256, so=8192)),
}
PAIRS = [(call, o, i) for call, (ins, outs) in OVERLAPS.items() for n, o in enumerate(outs)
         for i in list(ins) + list(outs)[n + 1:]]
BIG = A[60]


def place(call, name):
    """(the tensor's bytes, the alignment that it needs)"""
    ins, outs = OVERLAPS[call]
    return dict(ins, **outs)[name]


@pytest.mark.parametrize("call,out,other", PAIRS, ids=[f"{c.__name__}-{o}-{i}" for c, o, i in PAIRS])
def test_outputs_that_overlap_are_refused(lib, call, out, other):
    """The last 16 bytes (4 of a short tensor) of either inside the other; just behind it is accepted."""
    step = 256 if "ws" in (out, other) else 16 if place(call, out) >= 16 and place(call, other) >= 16 else 4
    kw = {"s": BIG + (1 << 30)} if call is conv_step else {"s": BIG + (2 << 30)} if call is ssm_step else {}
    n = place(call, other) // step * step
    assert call(lib, **dict(kw, **{other: BIG, out: BIG + max(0, n - step)})) == BAD
    n = place(call, out) // step * step
    assert call(lib, **dict(kw, **{out: BIG, other: BIG + max(0, n - step)})) == BAD
    n = -(-place(call, other) // 256) * 256
    assert call(lib, **dict(kw, **{other: BIG, out: BIG + n})) == CUDA


def test_states_of_the_steps(lib):
    for call, n in ((conv_step, 2 * 3 * 64 * 2), (ssm_step, 8192)):
        assert call(lib, s=BIG, so=BIG) == CUDA and call(lib, s=BIG, so=BIG + n) == CUDA
        assert call(lib, s=BIG, so=BIG + n - 16) == BAD and call(lib, s=BIG + n - 16, so=BIG) == BAD
        assert call(lib, s=BIG, so=BIG, y=BIG) == BAD and call(lib, s=BIG, so=A[40], y=BIG + n - 16) == BAD
        assert call(lib, s=BIG, so=A[40], y=A[40] + n - 16) == BAD


def test_outputs_between_the_rows_of_an_input(lib):
    """Rows 4096 elements apart leave room for another tensor; a row's own bytes do not."""
    wide = dict(x=BIG, ldx=4096)
    assert conv_forward(lib, so=BIG + 128, **wide) == CUDA and conv_forward(lib, y=BIG + 8192 + 128, **wide) == CUDA
    assert conv_forward(lib, y=BIG + 8192 - 16, **wide) == BAD and conv_forward(lib, y=BIG + 8192 * 9 + 112, **wide) == BAD
    assert conv_forward(lib, y=BIG + 8192 * 9 + 128, **wide) == CUDA
    assert conv_forward(lib, y=BIG + 8192 - TOK, **wide) == CUDA and conv_forward(lib, y=BIG - TOK, **wide) == CUDA


def test_the_workspace_is_what_the_call_needs(lib):
    """A workspace with bytes to spare may hold other tensors behind the bytes that the call asks for."""
    n = lib.gdn_conv_backward_workspace_size(10, 2, 64, 4)
    assert conv_backward(lib, ws=BIG, wsb=1 << 30, dx=BIG + n) == CUDA
    assert conv_backward(lib, ws=BIG, wsb=1 << 30, dx=BIG + n - 256) == BAD
    n = lib.gdn_ssm_backward_workspace_size(10, 2, 64, 2, 16)
    assert ssm_backward(lib, ws=BIG, wsb=1 << 30, ds=BIG + n) == CUDA
    assert ssm_backward(lib, ws=BIG, wsb=1 << 30, ds=BIG + n - 256) == BAD
    n = lib.gdn_layer_norm_backward_workspace_size(4, 64)
    assert norm_backward(lib, ws=BIG, wsb=1 << 30, dx=BIG + n) == CUDA
    assert norm_backward(lib, ws=BIG, wsb=1 << 30, dx=BIG + n - 256) == BAD


# alignment that each address needs (bf16 tokens and weights): what the kernels read in one access
ALIGNMENT = [(conv_forward, dict(cu=4, st=4, x=2, w=2, b=2, y=2, s=16, so=16)),
             (conv_backward, dict(cu=4, st=4, x=2, dy=2, w=2, b=2, dx=2, s=16, do=16, dw=16, db=16, ds=16, ws=256)),
             (conv_step, dict(x=2, w=2, b=2, y=2, so=16)),
             (norm_forward, dict(x=2, w=2, b=2, y=2, m=4, r=4)),
             (norm_backward, dict(x=2, dy=2, w=2, m=4, r=4, dx=2, dw=4, db=4, ws=256)),
             (ssm_forward, dict(x=2, dt=2, B=2, C=2, z=2, A=16, D=4, dt_bias=4, cu=4, si=16, y=2, so=16, cs=16, st=4)),
             (ssm_backward, dict(x=2, dt=2, B=2, C=2, z=2, A=16, D=4, dt_bias=4, cu=4, dy=2, cs=16, do=16, dx=2, ddt=2, dA=4,
                                 dB=2, dC=2, dD=4, dz=2, db=4, ds=16, ws=256, st=4)),
             (ssm_step, dict(x=2, dt=2, B=2, C=2, z=2, A=16, D=4, dt_bias=4, y=2, so=16))]


@pytest.mark.parametrize("call,name,n", [(c, k, n) for c, a in ALIGNMENT for k, n in a.items()],
                         ids=[f"{c.__name__}-{k}" for c, a in ALIGNMENT for k in a])
def test_misaligned_addresses_are_refused(lib, call, name, n):
    assert call(lib, **{name: BIG + n // 2}) == BAD
    assert call(lib, **{name: BIG + n}) == CUDA


@pytest.mark.parametrize("call,name,ld", [(norm_forward, "D", ("ldx",)), (norm_backward, "D", ("ldx", "ldg")),
                                          (ssm_forward, "D_", ("ldx", "lddt", "ldz")), (ssm_backward, "D_", ("ldx", "lddt", "ldz", "ldg")),
                                          (ssm_step, "D_", ("ldx", "lddt", "ldz"))])
def test_widths_beyond_the_counters_are_refused(lib, call, name, ld):
    """The kernels count columns, and a block's worth beyond the last, in 32 bits."""
    far = {k: (i + 1) << 50 for i, k in enumerate(dict(OVERLAPS[call][0], **OVERLAPS[call][1]))}
    far.update({"s": 60 << 50} if call is ssm_step else {}, **({"wsb": 1 << 50} if "ws" in far else {}))
    for width, want in ((2 ** 31 - 4098, CUDA), (2 ** 31 - 4096, BAD), (2 ** 31 - 2, BAD)):
        assert call(lib, **dict(far, **{name: width, **{k: width for k in ld}})) == want, width
