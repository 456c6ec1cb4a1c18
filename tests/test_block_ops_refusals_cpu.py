"""What the C entries of the norm of queries and keys, the gated block and the policy loss refuse, on a machine without a
GPU: there a call that passes every check ends with GDN_ERR_CUDA at its first CUDA call, so an accepted call can be told
from a refused one.  No address is dereferenced.  And what the binding refuses before that."""
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import build, gdn

BAD, UNSUPPORTED, SCRATCH, OK = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE, gdn.GDN_OK
CUDA = gdn.GDN_ERR_CUDA
A = [(i + 1) << 36 for i in range(64)]  # far apart
BIG = A[60]
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load_library()


def run(fn, struct, args, rest, kw):
    s = struct(*dict(args, **{k: v for k, v in kw.items() if k in args}).values())
    return fn(s, *dict(rest, **{k: v for k, v in kw.items() if k in rest}).values())


# 10 tokens, 4 + 2 heads of 32, 16 dimensions rotated, bf16
QK = dict(q=A[0], k=A[1], qw=A[2], kw=A[3], pos=A[4], freq=A[5], ldq=128, ldk=64, T=10, Hq=4, Hk=2, d=32, rot=16, inter=0, unit=0,
          eps=1e-6, it=1, wt=1)
# 10 rows, width 64, inner 32, bf16
GLU = dict(x=A[0], wg=A[1], wu=A[2], ldx=64, ldg=64, ldu=64, R=10, D=64, F=32, act=0, it=1)
# 10 rows of 64 logits, bf16
POL = dict(z=A[0], y=A[1], old=A[2], ref=A[3], adv=A[4], ldz=64, R=10, V=64, lo=0.2, hi=0.2, kl=0.1, tau=1.0, it=1)


def qk_forward(lib, **kw):
    return run(lib.gdn_qk_norm_forward, gdn.QkNormStruct, QK, dict(oq=A[10], ok=A[11], stream=None), kw)


def qk_backward(lib, **kw):
    return run(lib.gdn_qk_norm_backward, gdn.QkNormStruct, QK,
               dict(gq=A[12], ldgq=128, gk=A[13], ldgk=64, dq=A[14], dk=A[15], dqw=A[16], dkw=A[17], ws=A[18], wsb=1 << 30,
                    stream=None), kw)


def glu_forward(lib, **kw):
    return run(lib.gdn_glu_forward, gdn.GluStruct, GLU, dict(h=A[10], sv=A[11], ws=None, wsb=0, st=A[12], stream=None), kw)


def glu_backward(lib, **kw):
    return run(lib.gdn_glu_backward, gdn.GluStruct, GLU,
               dict(dh=A[13], ldh=32, sv=A[11], dx=A[14], dwg=A[15], dwu=A[16], dwt=1, ws=A[17], wsb=1 << 40, st=A[12],
                    stream=None), kw)


def pol_forward(lib, **kw):
    return run(lib.gdn_policy_loss_forward, gdn.PolicyStruct, POL, dict(loss=A[10], lp=A[11], st=A[12], stream=None), kw)


def pol_backward(lib, **kw):
    return run(lib.gdn_policy_loss_backward, gdn.PolicyStruct, POL,
               dict(w=A[13], dz=A[14], loss=A[10], lp=A[11], st=A[12], stream=None), kw)


CALLS = [qk_forward, qk_backward, glu_forward, glu_backward, pol_forward, pol_backward]


@no_gpu
@pytest.mark.parametrize("call", CALLS)
def test_a_valid_call_without_a_gpu_is_a_cuda_error(lib, call):
    assert call(lib) == CUDA


@pytest.mark.parametrize("call", [qk_forward, qk_backward])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), BAD), (dict(T=2 ** 31), BAD), (dict(Hq=0), BAD), (dict(Hk=0), BAD), (dict(d=0), BAD), (dict(d=31), UNSUPPORTED),
    (dict(d=258, ldq=2000, ldk=2000), UNSUPPORTED), (dict(rot=15), UNSUPPORTED), (dict(rot=34), BAD), (dict(rot=-2), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(it=2), BAD), (dict(wt=5), BAD), (dict(q=None), BAD), (dict(k=None), BAD),
    (dict(ldq=127), BAD), (dict(ldk=63), BAD), (dict(pos=None), BAD), (dict(freq=None), BAD), (dict(q=A[0] + 1), BAD),
    (dict(pos=A[4] + 2), BAD), (dict(freq=A[5] + 2), BAD), (dict(qw=A[2] + 1), BAD), (dict(Hq=2 ** 27), BAD)])
def test_qk_norm_refuses(lib, call, kw, want):
    assert call(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(gq=None), BAD), (dict(gk=None), BAD), (dict(ldgq=100), BAD), (dict(dq=None), BAD), (dict(dk=None), BAD), (dict(qw=None), BAD),
    (dict(kw=None), BAD), (dict(ws=None), SCRATCH), (dict(wsb=64), SCRATCH), (dict(ws=A[18] + 16), BAD), (dict(dqw=A[16] + 2), BAD)])
def test_qk_norm_backward_refuses(lib, kw, want):
    assert qk_backward(lib, **kw) == want


@no_gpu
def test_qk_norm_accepts_what_is_not_needed(lib):
    assert qk_forward(lib, rot=0, pos=None, freq=None) == CUDA and qk_forward(lib, qw=None, kw=None) == CUDA
    assert qk_backward(lib, dqw=None, dkw=None, ws=None, wsb=0) == CUDA and qk_backward(lib, qw=None, dqw=None) == CUDA
    assert qk_forward(lib, T=0, q=None, k=None, pos=None, oq=None, ok=None) == OK


@pytest.mark.parametrize("call", [glu_forward, glu_backward])
@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), BAD), (dict(R=2 ** 31), BAD), (dict(D=0), BAD), (dict(F=0), BAD), (dict(act=2), BAD), (dict(act=-1), BAD), (dict(it=9), BAD),
    (dict(it=0), UNSUPPORTED), (dict(x=None), BAD), (dict(wg=None), BAD), (dict(wu=None), BAD), (dict(ldx=63), BAD), (dict(ldg=60), BAD),
    (dict(ldu=1), BAD), (dict(x=A[0] + 1), BAD), (dict(wg=A[1] + 1), BAD), (dict(st=A[12] + 2), BAD), (dict(sv=A[11] + 8), BAD),
    (dict(F=2 ** 31 - 1), BAD), (dict(ldg=2 ** 32), BAD)])
def test_glu_refuses(lib, call, kw, want):
    assert call(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), BAD), (dict(h=A[10] + 1), BAD), (dict(x=A[0] + 2), SCRATCH), (dict(ldg=67), SCRATCH), (dict(D=63, ldx=63), SCRATCH),
    (dict(x=A[0] + 2, ws=A[20], wsb=1000), SCRATCH), (dict(x=A[0] + 2, ws=A[20] + 16, wsb=1 << 20), BAD)])
def test_glu_forward_refuses(lib, kw, want):
    assert glu_forward(lib, **kw) == want


@no_gpu
def test_glu_forward_needs_a_workspace_for_rows_off_their_alignment_only(lib):
    size = lambda **kw: lib.gdn_glu_forward_workspace_size(gdn.GluStruct(*dict(GLU, **kw).values()))  # noqa: E731
    assert size() == 0 and size(ldx=72) == 0 and size(D=63, ldx=64, ldg=64, ldu=64) == 0
    assert size(x=A[0] + 2) == 10 * 64 * 2 and size(wg=A[1] + 2) == 32 * 64 * 2
    assert size(D=63, ldx=63, ldg=63, ldu=63) == 10 * 64 * 2 + 2 * 32 * 64 * 2
    assert glu_forward(lib, x=A[0] + 2, ws=A[20], wsb=1280) == CUDA
    assert lib.gdn_glu_saved_size(10, 32) == 1920 and lib.gdn_glu_saved_size(-1, 32) == -1 and lib.gdn_glu_saved_size(1, 0) == -1
    assert glu_forward(lib, R=0, x=None, h=None, sv=None) == OK and glu_forward(lib, sv=None) == CUDA


@pytest.mark.parametrize("kw,want", [
    (dict(dh=None), BAD), (dict(ldh=31), BAD), (dict(sv=None), BAD), (dict(dx=None), BAD), (dict(dwg=None), BAD), (dict(dwu=None), BAD),
    (dict(dwt=2), BAD), (dict(dwt=0, dwg=A[15] + 2), BAD), (dict(dwg=A[15] + 1), BAD)])
def test_glu_backward_refuses(lib, kw, want):
    assert glu_backward(lib, **kw) == want


@pytest.mark.parametrize("call", [pol_forward, pol_backward])
@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), BAD), (dict(R=2 ** 31), BAD), (dict(V=0), BAD), (dict(it=4), BAD), (dict(z=None), BAD), (dict(ldz=63), BAD), (dict(y=None), BAD),
    (dict(y=A[1] + 4), BAD), (dict(old=None), BAD), (dict(adv=None), BAD), (dict(tau=0.0), BAD), (dict(tau=-1.0), BAD),
    (dict(tau=float("inf")), BAD), (dict(tau=float("nan")), BAD), (dict(lo=-0.1), BAD), (dict(lo=1.5), BAD), (dict(hi=-0.1), BAD),
    (dict(kl=float("nan")), BAD), (dict(old=A[2] + 2), BAD), (dict(st=A[12] + 2), BAD), (dict(z=A[0] + 1), BAD),
    (dict(V=2 ** 31 - 1, ldz=2 ** 31 - 1), BAD)])
def test_policy_refuses(lib, call, kw, want):
    assert call(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [(dict(loss=None), BAD), (dict(lp=None), BAD), (dict(old=None, adv=None, ref=None), BAD),
                                     (dict(old=None, adv=None, loss=None), BAD), (dict(lp=A[11] + 2), BAD)])
def test_policy_forward_refuses(lib, kw, want):
    assert pol_forward(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [(dict(w=None), BAD), (dict(dz=None), BAD), (dict(old=None, adv=None, ref=None), BAD), (dict(w=A[13] + 1), BAD),
                                     (dict(dz=A[14] + 1), BAD), (dict(dz=A[0], ldz=72), BAD), (dict(dz=A[0] + 128), BAD)])
def test_policy_backward_refuses(lib, kw, want):
    assert pol_backward(lib, **kw) == want


@no_gpu
def test_policy_accepts(lib):
    assert pol_forward(lib, old=None, adv=None, ref=None, loss=None) == CUDA and pol_forward(lib, ref=None, st=None) == CUDA
    assert pol_backward(lib, dz=A[0]) == CUDA and pol_backward(lib, loss=None, lp=None) == CUDA
    assert pol_backward(lib, dz=A[0], R=1, ldz=100) == CUDA
    assert pol_forward(lib, R=0, z=None, y=None, lp=None) == OK


# bytes of each tensor of the calls above
Q, K = 10 * 128 * 2, 10 * 64 * 2
OVERLAPS = {
    qk_forward: (dict(q=Q, k=K, qw=64, kw=64, pos=40, freq=32), dict(oq=Q, ok=K)),
    qk_backward: (dict(q=Q, k=K, qw=64, kw=64, pos=40, freq=32, gq=Q, gk=K), dict(dq=Q, dk=K, dqw=128, dkw=128, ws=1024 * 2 * 32 * 4)),
    glu_forward: (dict(x=1280, wg=4096, wu=4096), dict(h=640, sv=1920, st=4)),
    glu_backward: (dict(x=1280, wg=4096, wu=4096, dh=640, sv=1920), dict(dx=1280, dwg=4096, dwu=4096, st=4)),
    pol_forward: (dict(z=1280, y=80, old=40, ref=40, adv=40), dict(loss=40, lp=40, st=4)),
    pol_backward: (dict(y=80, old=40, ref=40, adv=40, w=40), dict(dz=1280, loss=40, lp=40, st=4)),
}
PAIRS = [(call, o, i) for call, (ins, outs) in OVERLAPS.items() for n, o in enumerate(outs) for i in list(ins) + list(outs)[n + 1:]]


@no_gpu
@pytest.mark.parametrize("call,out,other", PAIRS, ids=[f"{c.__name__}-{o}-{i}" for c, o, i in PAIRS])
def test_outputs_that_overlap_are_refused(lib, call, out, other):
    """The last bytes of either inside the other; just behind it is accepted."""
    ins, outs = OVERLAPS[call]
    size = dict(ins, **outs)
    step = 256 if "ws" in (out, other) else 16 if size[out] >= 16 and size[other] >= 16 else 4
    kw = {} if "sv" in (out, other) or "sv" not in size else {"sv": A[40]}
    n = size[other] // step * step
    assert call(lib, **dict(kw, **{other: BIG, out: BIG + max(0, n - step)})) == BAD
    n = size[out] // step * step
    assert call(lib, **dict(kw, **{out: BIG, other: BIG + max(0, n - step)})) == BAD
    n = -(-size[other] // 256) * 256
    assert call(lib, **dict(kw, **{other: BIG, out: BIG + n})) == CUDA


def test_the_binding_refuses_before_the_library():
    cpu = torch.zeros(4, 2, 8)
    for fn, args in ((gdn.gdn_qk_norm_forward, (cpu, cpu)), (gdn.gdn_glu_forward, (cpu[0], cpu[0], cpu[0])),
                     (gdn.gdn_policy_loss_forward, (cpu[0], torch.zeros(2, dtype=torch.int64))),
                     (gdn.gdn_qk_norm_backward, (cpu, cpu, cpu, cpu)),
                     (gdn.gdn_glu_backward, (cpu[0], cpu[0], cpu[0], cpu[0], cpu[0]))):
        with pytest.raises(ValueError, match="CUDA device"):
            fn(*args)
    with pytest.raises(ValueError, match="CUDA device"):
        gdn.gdn_policy_loss_backward(cpu[0], torch.zeros(2, dtype=torch.int64), cpu[0, 0], old_logprob=None, advantages=None)
